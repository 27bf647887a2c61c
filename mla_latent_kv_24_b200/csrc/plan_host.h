// Host side of the split-KV plan (the device side is plan_block.cuh).  Both follow one rule:
// row (b, j) has len = seq_lens[b] - s_q + j + 1 tokens (or those of its window or tree, view.cuh),
// cut into ceil(len / chunk) chunks.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace mla {

// Chunks of all rows; len(r) = tokens of row r (a row without tokens has none).
template <typename Len>
inline long long plan_count_rows(int rows, const Len &len, long long chunk) {
    long long n = 0;
    for (int r = 0; r < rows; ++r) n += ((long long)len(r) + chunk - 1) / chunk;
    return n;
}

// Chunk length (a multiple of `granule` tokens) that spreads all rows' tokens over about
// `units` concurrently running workers: the smallest such length whose chunk count fits in
// one wave of `units` when that is possible (more chunks than workers would leave a second,
// mostly idle wave).  Otherwise (more rows than workers) workers take several chunks each, and
// three quarters of the even split of all tokens: the smaller chunks balance the workers'
// totals better (a ragged batch of 128 rows on 74 tcgen05 workers: 275 -> 264 us; half the
// even split paid more in per-chunk overhead than it gained).
template <typename Len>
inline int plan_chunk_rows(int rows, const Len &len, int units, int granule) {
    long long total = 0, longest = 1;
    for (int r = 0; r < rows; ++r) {
        total += len(r);
        longest = std::max<long long>(longest, len(r));
    }
    units = std::max(1, units);
    auto round_up = [&](long long c) { return std::max<long long>(granule, (c + granule - 1) / granule * granule); };
    long long lo = round_up((total + units - 1) / units);
    long long hi = round_up(longest);
    if (lo >= hi) return (int)std::min<long long>(lo, 1 << 30);
    if (plan_count_rows(rows, len, std::min<long long>(hi, 1 << 30)) > units)
        return (int)std::min<long long>(round_up(lo * 3 / 4), 1 << 30);
    while (lo < hi) {  // smallest multiple of granule in [lo, hi] with count <= units
        const long long mid = round_up((lo + hi) / 2 - granule + 1);
        const long long m = mid < lo ? lo : mid;
        if (plan_count_rows(rows, len, m) <= units)
            hi = m;
        else
            lo = m + granule;
    }
    return (int)std::min<long long>(lo, 1 << 30);
}

// Chunk length for a view's rows on the persistent tcgen05 decode: of several candidates the one whose
// snake-dealt items (plan_block.cuh: full chunks, then the rows' last chunks by length, longest first) give
// the shortest longest worker.  A request has `rows(b)` rows of about `len(b)` tokens.  In steps of
// `granule` tokens (1.9 us): an item costs its steps and ITEM_STEPS more (its queries' load, the drain of O,
// the pipeline's refill), and the merge of its partial MERGE_STEPS over all workers (512 KiB written and
// read).  Rows that the three-quarter rule above leaves unequal gain most: 64 ragged windows, two queries
// each, 71 -> 57 steps; 24 trees of up to 13 nodes on 1,024 to 32,768 tokens, 265 -> 242.
template <typename Rows, typename Len>
inline int plan_chunk_balanced(int batch, const Rows &rows, const Len &len_of, int units, int granule) {
    constexpr float ITEM_STEPS = 3.7f, MERGE_STEPS = 0.055f;
    constexpr int BUCKETS = 64, MAX_UNITS = 256, KEPT = 512;
    int kept[KEPT];   // the first requests' lengths: every candidate asks for them
    for (int b = 0; b < std::min(batch, KEPT); ++b) kept[b] = rows(b) > 0 ? len_of(b) : 0;
    auto len = [&](int b) { return b < KEPT ? kept[b] : len_of(b); };
    units = std::max(1, std::min(units, MAX_UNITS));
    auto round_up = [&](long long c) {
        return (int)std::min<long long>(std::max<long long>(granule, (c + granule - 1) / granule * granule), 1 << 30);
    };
    int longest = 1;
    long long total = 0;
    for (int b = 0; b < batch; ++b) {
        if (rows(b) <= 0) continue;
        longest = std::max(longest, len(b));
        total += (long long)rows(b) * len(b);
    }
    int best = round_up(longest), tried[16], n_tried = 0;
    float best_cost = -1.f;
    auto consider = [&](long long candidate) {
        const int chunk = round_up(candidate);
        for (int i = 0; i < n_tried; ++i)
            if (tried[i] == chunk) return;
        tried[n_tried++] = chunk;
        long long full = 0, items = 0;
        int hist[BUCKETS] = {};   // the rows' last chunks by length
        const float per_token = (float)BUCKETS / (float)chunk;
        for (int b = 0; b < batch; ++b) {
            const int n = rows(b), l = n > 0 ? len(b) : 0, whole = l / chunk, tail = l - whole * chunk;
            if (l <= 0) continue;
            full += (long long)n * whole;
            items += (long long)n * (whole + (tail > 0));
            if (tail) hist[std::min(BUCKETS - 1, (int)((float)tail * per_token))] += n;
        }
        // Equal items in whole rounds load every worker alike; the rest go on in snake order.
        float load[MAX_UNITS] = {}, all = 0.f;
        int at = 0, turn = 0;
        auto deal = [&](long long n, float cost) {
            all += cost * (float)(n / units);
            for (int i = (int)(n % units); i > 0; --i) {
                load[turn ? units - 1 - at : at] += cost;
                if (++at == units) at = 0, turn ^= 1;
            }
        };
        deal(full, (float)(chunk / granule) + ITEM_STEPS);
        for (int k = BUCKETS - 1; k >= 0; --k)
            if (hist[k]) {
                const float steps = ((float)k + 0.5f) * (float)chunk / (float)(BUCKETS * granule);
                deal(hist[k], std::max(1.f, (float)(int)(steps + 0.999f)) + ITEM_STEPS);
            }
        float worst = 0.f;
        for (int u = 0; u < units; ++u) worst = std::max(worst, load[u]);
        const float cost = all + worst + MERGE_STEPS * (float)items;
        if (best_cost < 0.f || cost < best_cost) best_cost = cost, best = chunk;
    };
    for (int k = 1; k <= 6; ++k) consider((longest + k - 1) / k);
    for (int k = 1; k <= 8; k *= 2) consider((total + (long long)units * k - 1) / ((long long)units * k));
    return best;
}

// The kernels around a view's tcgen05 decode (head_gemm.cu, or absorb.cu and combine.cu), by its rows and chunks.
//
// Above 16 rows, where the mma.sync form leaves its single wave (24 rows: 1.7 us a call less; 96: 4; the
// kernel alone at 512 rows: 35 and 48).
inline bool absorb_tc_pays(int rows) { return rows > 16; }
// One 16-row tile merges faster in clusters of four CTAs a head (launch_combine_mma; a window's call of 8 rows 29 us
// against 43, of 16 rows 34 and 37).  Above that a cluster takes its rows one pass after another, and this kernel a
// row's chunks: rows^2 / 6 chunks in all are where the two meet (17 rows of 4.4 chunks 55 us in clusters, 65 here; 20
// of 3.7: 57 and 62; 24 of 3.1: 65 and 64; 24 of one: 43 and 35; 32: 74 and 64; 40: 91 and 78).
inline bool project_tc_pays(int rows, long long n_work) { return rows > 16 && 6 * n_work <= (long long)rows * rows; }

// Causal rows: r = (b, j).
inline int plan_chunk(const int32_t *lens, int batch, int s_q, int units, int granule) {
    return plan_chunk_rows(batch * s_q, [=](int r) { return lens[r / s_q] - s_q + r % s_q + 1; }, units, granule);
}
inline long long plan_count(const int32_t *lens, int batch, int s_q, int chunk) {
    return plan_count_rows(batch * s_q, [=](int r) { return lens[r / s_q] - s_q + r % s_q + 1; }, chunk);
}

}  // namespace mla
