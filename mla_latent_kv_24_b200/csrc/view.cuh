// Which cached tokens a query sees, for the decodes whose queries do not simply see every token up
// to their own position.
//
// Window: query j of request b (length L, position p = L - s_q + j) sees the tokens t <= p with
//   t < sinks or t > p - window.
// Tree: the last n = n_nodes[b] of the L cached tokens are drafted nodes; node j sees every token
//   of the context (t < L - n) and the nodes whose bits its 64-bit mask sets.
//
// A plan row's work items cover "virtual" tokens: the pages a row has to read, in order and without
// the pages between the sinks and the window.  Virtual token v is token v below `gap_at` and
// v + gap above it; both are multiples of the page size, so a page is never cut.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MLA_HD __host__ __device__ __forceinline__
#else
#define MLA_HD inline
#endif

namespace mla {

enum ViewKind { VIEW_CAUSAL = 0, VIEW_WINDOW = 1, VIEW_TREE = 2 };

struct View {
    int kind;
    int sinks, window;               // VIEW_WINDOW
    const int *n_nodes;              // VIEW_TREE: [batch]
    const int *depths;               // VIEW_TREE: [batch, s_q]
    const unsigned long long *mask;  // VIEW_TREE: [batch, s_q]
};

// Tokens [0, gap_at) and [gap_at + gap, end), as virtual tokens [0, len).
struct Span {
    int gap_at, gap, len;
};

// The pages of the queries at positions p0..p1 of one request: the sinks' and from the first page
// of p0's window on.  Without a page between the two there is no gap.
MLA_HD Span window_span(int sinks, int window, int p0, int p1, int page) {
    const int end = p1 + 1;
    const int lo = p0 - window + 1 > 0 ? p0 - window + 1 : 0;
    const int s = sinks < end ? sinks : end;
    const int gap_at = (s + page - 1) / page * page;
    const int first = lo / page * page;
    if (first <= gap_at) return Span{0, 0, end};
    return Span{gap_at, first - gap_at, end - (first - gap_at)};
}

// Virtual length of plan row (b, j), 0 for a row with nothing to do, -1 for lengths that cannot be.
// With plan_sq = 1 and n_q > 1 one row stands for all n_q queries of its request.
MLA_HD int view_row_len(int kind, int sinks, int window, int L, int n, int plan_sq, int n_q, int j,
                                            int page, int max_len) {
    if (L > max_len) return -1;
    if (kind == VIEW_TREE) {
        if (n < 0 || n > n_q || L < n) return -1;
        return j < n ? L : 0;
    }
    if (L < n_q) return -1;
    if (kind == VIEW_CAUSAL) return L - plan_sq + j + 1;
    const int p0 = plan_sq == 1 ? L - n_q : L - n_q + j, p1 = plan_sq == 1 ? L - 1 : p0;
    return window_span(sinks, window, p0, p1, page).len;
}

// One work item's view: of one query, or (window only) of all queries of a request together.
struct ItemView {
    Span span;
    int lo, sinks, end;              // window: tokens [lo, end) and [0, sinks)
    unsigned long long mask;         // tree: bit i = token ctx + i
    int ctx;
    bool tree;
    int whole0, whole1;              // virtual tokens [whole0, whole1) are all seen; multiples of 64

    MLA_HD int token(int v) const { return v < span.gap_at ? v : v + span.gap; }

    // Bit i: token t0 + i is seen, i < 64.
    MLA_HD unsigned long long seen64(int t0) const {
        if (tree) {
            const int d = ctx - t0;   // place of node 0
            if (d >= 64) return ~0ull;
            if (d >= 0) return (d ? (~0ull >> (64 - d)) : 0ull) | (mask << d);
            return d > -64 ? mask >> -d : 0ull;
        }
        return (below(sinks - t0) | ~below(lo - t0)) & below(end - t0);
    }
    MLA_HD bool seen(int t) const {
        if (tree) return t < ctx || (t - ctx < 64 && ((mask >> (t - ctx)) & 1ull));
        return t < end && (t < sinks || t >= lo);
    }

  private:
    // Bits 0..n-1.
    static MLA_HD unsigned long long below(int n) {
        return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
    }
};

// `n_q` queries per request (tree: node slots).  `j` < 0: all queries of the request together.
// Only for requests whose lengths the plan accepted.
MLA_HD ItemView item_view(const View &v, const int *seq_lens, int b, int j, int n_q, int page) {
    ItemView iv;
    const int L = seq_lens[b];
    iv.tree = v.kind == VIEW_TREE;
    if (iv.tree) {
        const int n = v.n_nodes[b];
        iv.span = Span{0, 0, L};
        iv.ctx = L - n;
        iv.mask = v.mask[(size_t)b * n_q + j];
        if (n < 64) iv.mask &= (1ull << n) - 1ull;
        iv.lo = 0, iv.sinks = 0, iv.end = L;
        iv.whole0 = 0;
        iv.whole1 = iv.ctx / 64 * 64;
    } else {
        const int p0 = j < 0 ? L - n_q : L - n_q + j, p1 = j < 0 ? L - 1 : p0;
        iv.span = window_span(v.sinks, v.window, p0, p1, page);
        iv.lo = p0 - v.window + 1 > 0 ? p0 - v.window + 1 : 0;
        iv.sinks = v.sinks;
        iv.end = p1 + 1;
        iv.ctx = 0, iv.mask = 0;
        // The window's whole pages; the sinks' pages are few.  (Pages other than 64 tokens: not used.)
        iv.whole0 = (iv.lo + 63) / 64 * 64 - iv.span.gap;
        iv.whole1 = iv.end / 64 * 64 - iv.span.gap;
    }
    return iv;
}

}  // namespace mla
