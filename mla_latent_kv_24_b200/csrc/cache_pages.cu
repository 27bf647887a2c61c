// Pages of the caches: reserving, forking, releasing, and moving a tree's accepted rows together.
//
// The pool's whole state is page_refs [n_pages]: how many page-table entries name each page.  A page
// with no entry is free, and allocation takes the lowest free ids in the order of the requests, so
// neither the pages a call hands out nor the state it leaves depends on the order of atomics, and
// freeing is a decrement.  The price is that an allocating call reads the counts up to the last page
// it takes (4 bytes a page: 40,000 pages are 160 KB); one block does it, 16,384 pages at a time.
//
// Rows of the caches are copied with 16-byte accesses (2 or 4 bytes where a row's size asks for it).
// All of it is bound by launches and latency, except forks over many layers, which are bound by the
// copied bytes.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "kernels.h"

namespace mla {
namespace {

constexpr int PT = 1024;        // threads of the allocating block
constexpr int PER = 16;         // counts a thread reads per tile
constexpr int CAP = PAGES_MAX_REQS;

// Exclusive prefix of v over the block; *total gets the sum.  All PT threads call it.
__device__ __forceinline__ int block_prefix(int v, int *total) {
    __shared__ int warp_sum[PT / 32 + 1];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
    }
    __syncthreads();   // the previous call's readers are done
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int w = warp_sum[lane];
        int wi = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, wi, off);
            if (lane >= off) wi += x;
        }
        warp_sum[lane] = wi - w;
        if (lane == 31) warp_sum[PT / 32] = wi;
    }
    __syncthreads();
    *total = warp_sum[PT / 32];
    return warp_sum[warp] + incl - v;
}

// Bit i: page base + i is free, i < PER.
__device__ __forceinline__ uint32_t free_bits(const int *refs, int n_pages, int base) {
    uint32_t m = 0;
    if (base + PER <= n_pages) {
        const int4 *p = reinterpret_cast<const int4 *>(refs + base);
        int4 v[PER / 4];
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) v[i] = p[i];
#pragma unroll
        for (int i = 0; i < PER / 4; ++i)
            m |= ((uint32_t)(v[i].x == 0) | (uint32_t)(v[i].y == 0) << 1 | (uint32_t)(v[i].z == 0) << 2 |
                  (uint32_t)(v[i].w == 0) << 3)
                 << 4 * i;
    } else {
        for (int i = 0; base + i < n_pages; ++i) m |= (uint32_t)(refs[base + i] == 0) << i;   // < PER of them
    }
    return m;
}

// Hands the `wanted` lowest free pages to take(rank, page), rank 0 first, and marks them held.
// False, with nothing changed, if there are fewer.  All PT threads call it.
// first_tile: this thread's free_bits() of the first pages, which the caller loads ahead of its own chain.
template <typename Take>
__device__ __forceinline__ bool allocate(int *refs, int n_pages, int wanted, uint32_t first_tile, const Take &take) {
    if (wanted == 0) return true;
    int first_total;
    const int first_rank = block_prefix(__popc(first_tile), &first_total);
    int have = first_total;
    for (int base = PT * PER; base < n_pages && have < wanted; base += PT * PER) {
        const int at = base + (int)threadIdx.x * PER;
        int total;
        block_prefix(__popc(at < n_pages ? free_bits(refs, n_pages, at) : 0u), &total);
        have += total;
    }
    if (have < wanted) return false;
    int before = 0;
    for (int base = 0; before < wanted; base += PT * PER) {
        const int at = base + (int)threadIdx.x * PER;
        uint32_t m = first_tile;
        int rank = first_rank, total = first_total;
        if (base) {
            m = at < n_pages ? free_bits(refs, n_pages, at) : 0u;
            rank = before + block_prefix(__popc(m), &total);
        }
        for (; m && rank < wanted; m &= m - 1, ++rank) {
            const int page = at + __ffs(m) - 1;
            refs[page] = 1;
            take(rank, page);
        }
        before += total;
    }
    return true;
}

struct RowSets {
    PageRows r[2];
    int n;
};

struct Pool {
    int *seq_lens, *page_table, *refs;
    int batch, max_pages, n_pages, page;
    int *err;
    __device__ __forceinline__ int pages_of(int len) const { return len / page + (len % page != 0); }
    __device__ __forceinline__ bool fits(int len) const { return len >= 0 && len <= (long long)max_pages * page; }
    __device__ __forceinline__ int *entry(int b, int k) const { return page_table + (size_t)b * max_pages + k; }
};

__device__ __forceinline__ uint32_t first_bits(const Pool &p) {
    const int at = (int)threadIdx.x * PER;
    return at < p.n_pages ? free_bits(p.refs, p.n_pages, at) : 0u;
}

// ------------------------------------------------------------------------------------- reserve
__global__ void __launch_bounds__(PT) reserve_kernel(Pool p, const int *__restrict__ new_lens) {
    step_begin();
    __shared__ int off[CAP + 1];
    const uint32_t tile = first_bits(p);
    const int per = ceil_div(p.batch, PT), b0 = min(p.batch, (int)threadIdx.x * per), b1 = min(p.batch, b0 + per);
    int mine = 0, bad = 0;
    for (int b = b0; b < b1; ++b) {
        const int L = p.seq_lens[b], n = new_lens[b];
        if (L < 0 || n < L || !p.fits(n)) {
            bad = 1;
            off[b] = 0;
        } else {
            off[b] = p.pages_of(n) - p.pages_of(L);
            mine += off[b];
        }
    }
    bad = __syncthreads_or(bad);
    int total;
    int at = block_prefix(mine, &total);
    for (int b = b0; b < b1; ++b) {
        const int n = off[b];
        off[b] = at;
        at += n;
    }
    if (threadIdx.x == 0) off[p.batch] = total;
    __syncthreads();
    if (bad) {
        if (threadIdx.x == 0) report(p.err, MLA_ERR_DEVICE_BOUNDS);
        return;
    }
    const bool ok = allocate(p.refs, p.n_pages, total, tile, [&](int rank, int pg) {
        int lo = 0, hi = p.batch - 1;   // the last request that starts at or before `rank`
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (off[mid] <= rank) lo = mid;
            else hi = mid - 1;
        }
        *p.entry(lo, p.pages_of(p.seq_lens[lo]) + rank - off[lo]) = pg;
    });
    if (!ok) {
        if (threadIdx.x == 0) report(p.err, MLA_ERR_NO_PAGES);
        return;
    }
    __syncthreads();   // the lengths are read above
    for (int b = b0; b < b1; ++b) p.seq_lens[b] = new_lens[b];
}

// ------------------------------------------------------------------------------------- fork
// Checks and new pages.  Claims the destinations (which must be empty, each named once) by a compare
// and swap of their length, so that a destination named twice is found whatever the order.  A call
// that is carried out leaves -1 - length in every destination, which tells the copying blocks the length.
// A destination of a refused call keeps its own, which may be anything, such a mark too; so a refused call also
// leaves its number in a word of its own.  (Numbers FORK_WORDS apart share a word, which names one of them;
// a captured call keeps its number, and clears what an earlier replay left.)
//
// A fork takes a page for its source's partly filled last page.  Where the source has dropped that page, the
// copying blocks give it back.  If the pool is short of pages for that, the sources' entries are read here, and
// those forks take none: reading them always would put a load into the chain of every call (forks of one request 10.7 -> 11.9 us).
constexpr int FORK_WORDS = 4096;
__device__ unsigned long long g_fork_refused[FORK_WORDS];

__global__ void __launch_bounds__(PT) fork_plan_kernel(Pool p, const int *__restrict__ src, const int *__restrict__ dst,
                                                       int n, unsigned long long call) {
    step_begin();
    unsigned long long left = 0;
    if (threadIdx.x == 0) left = g_fork_refused[call % FORK_WORDS];
    __shared__ int len[CAP];   // the source's length; -1 - length where its partial last page is known to be dropped
    const uint32_t tile = first_bits(p);
    const int per = ceil_div(n, PT), i0 = min(n, (int)threadIdx.x * per), i1 = min(n, i0 + per);
    int parts = 0, bad = 0;
    for (int i = i0; i < i1; ++i) {
        const int s = src[i], d = dst[i];
        len[i] = 0;
        if (s < 0 || s >= p.batch || d < 0 || d >= p.batch) {
            bad = 1;
            continue;
        }
        len[i] = p.seq_lens[s];
        if (!p.fits(len[i])) bad = 1;
        parts += len[i] % p.page > 0;
    }
    bad = __syncthreads_or(bad);   // every source is read before any destination is written
    int n_claimed = 0;
    if (!bad)
        for (int i = i0; i < i1; ++i, ++n_claimed)
            if (atomicCAS(p.seq_lens + dst[i], 0, -1 - i) != 0) {
                bad = 1;
                break;
            }
    bad = __syncthreads_or(bad);
    // No destination has pages of its own, so its row holds nothing that is still needed.
    // The rank-th page goes to the rank-th fork with a partial page (a dropped one has a negative length): each
    // thread's forks are consecutive, so a rank names a thread's first rank and a count from there.
    __shared__ int first_rank[PT + 1];
    auto hand_out = [&](int mine) {
        int total;
        const int rank0 = block_prefix(mine, &total);
        first_rank[threadIdx.x] = rank0;
        if (threadIdx.x == PT - 1) first_rank[PT] = total;
        __syncthreads();
        return allocate(p.refs, p.n_pages, total, tile, [&](int rank, int pg) {
            int lo = 0, hi = PT - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (first_rank[mid] <= rank) lo = mid;
                else hi = mid - 1;
            }
            int skip = rank - first_rank[lo], i = min(n, lo * per);
            for (;; ++i)
                if (len[i] % p.page > 0 && skip-- == 0) break;
            *p.entry(dst[i], len[i] / p.page) = pg;
        });
    };
    bool ok = !bad;
    if (ok) {
        ok = hand_out(parts);
        if (!ok) {
            int none = 0;   // forks that need no page after all
            for (int i = i0; i < i1; ++i) {
                const int L = len[i];
                if (L % p.page == 0 || *p.entry(src[i], L / p.page) >= 0) continue;
                len[i] = -1 - L;
                ++none;
            }
            if (__syncthreads_or(none)) ok = hand_out(parts - none);
            __syncthreads();   // the searches have read the lengths
            for (int i = i0; i < i1; ++i)
                if (len[i] < 0) {
                    len[i] = -1 - len[i];
                    if (ok) *p.entry(dst[i], len[i] / p.page) = -1;
                }
        }
    }
    __syncthreads();
    for (int i = i0; i < i0 + n_claimed; ++i) p.seq_lens[dst[i]] = ok ? -1 - len[i] : 0;
    if (threadIdx.x == 0) {
        if (!ok) report(p.err, bad ? MLA_ERR_DEVICE_BOUNDS : MLA_ERR_NO_PAGES);
        if (!ok || left == call) g_fork_refused[call % FORK_WORDS] = ok ? 0 : call;
    }
}

// Copies bytes [from, to) of a span with the block's threads.
template <typename V>
__device__ __forceinline__ void copy_span(char *dst, const char *src, size_t bytes) {
    const size_t n = bytes / sizeof(V);
    constexpr int U = 4;
    const size_t stride = (size_t)blockDim.x;
    size_t i = threadIdx.x;
    for (; i + (U - 1) * stride < n; i += U * stride) {
        V v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = reinterpret_cast<const V *>(src)[i + u * stride];
#pragma unroll
        for (int u = 0; u < U; ++u) reinterpret_cast<V *>(dst)[i + u * stride] = v[u];
    }
    for (; i < n; i += stride) reinterpret_cast<V *>(dst)[i] = reinterpret_cast<const V *>(src)[i];
}

// One cluster per fork shares the full pages and copies the partial page's rows, then gives the
// destination its length.  A piece of rows goes to one block, or in parts to several when there are
// fewer pieces than blocks.
__global__ void __launch_bounds__(256) fork_copy_kernel(Pool p, const int *__restrict__ src, const int *__restrict__ dst,
                                                        RowSets sets, unsigned long long call) {
    step_begin();
    const int rank = blockIdx.x, blocks = gridDim.x;              // the cluster spans the grid's x
    const unsigned long long refused = g_fork_refused[call % FORK_WORDS];
    const int s = src[blockIdx.y], d = dst[blockIdx.y];
    if (refused == call || s < 0 || s >= p.batch || d < 0 || d >= p.batch) return;   // the whole cluster
    const int L = -1 - p.seq_lens[d];
    if (L < 0 || (L > 0 && L != p.seq_lens[s])) return;   // not a mark of this call: nothing to index by
    if (L > 0) {
        const int full = L / p.page, rem = L % p.page;
        for (int k = rank * (int)blockDim.x + (int)threadIdx.x; k < full; k += blocks * (int)blockDim.x) {
            const int pg = *p.entry(s, k);
            *p.entry(d, k) = pg;
            if (pg >= p.n_pages) report(p.err, MLA_ERR_DEVICE_BOUNDS);
            else if (pg >= 0) atomicAdd(p.refs + pg, 1);          // a dropped page (< 0) has no holder to add
        }
        const int from = rem ? *p.entry(s, full) : -1, to = rem ? *p.entry(d, full) : -1;
        if (rem && from < 0) {   // dropped in the source: so it is in the copy, and a page taken for it is free again
            cooperative_groups::this_cluster().sync();   // every block has read the entries
            if (rank == 0 && threadIdx.x == 0 && to >= 0 && to < p.n_pages) {
                *p.entry(d, full) = -1;
                p.refs[to] = 0;
            }
        } else if (rem) {   // reported with and without caches to copy in
            if (from >= p.n_pages || to < 0 || to >= p.n_pages) {
                if (threadIdx.x == 0) report(p.err, MLA_ERR_DEVICE_BOUNDS);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (i >= sets.n) break;
                    const PageRows &r = sets.r[i];
                    const int units = r.n_layers * r.pieces, parts = units >= blocks ? 1 : ceil_div(blocks, units);
                    const size_t bytes = (size_t)rem * r.row_bytes;
                    const size_t part = ((bytes + parts - 1) / parts + 15) / 16 * 16;
                    for (int w = rank; w < units * parts; w += blocks) {
                        const size_t at = (size_t)(w % parts) * part;
                        if (at >= bytes) continue;
                        const size_t n = bytes - at < part ? bytes - at : part;
                        char *to_p = r.at(w / parts, to) + at;
                        const char *from_p = r.at(w / parts, from) + at;
                        if (r.vec == 16) copy_span<uint4>(to_p, from_p, n);
                        else if (r.vec == 4) copy_span<uint32_t>(to_p, from_p, n);
                        else copy_span<uint16_t>(to_p, from_p, n);
                    }
                }
            }
        }
    }
    cooperative_groups::this_cluster().sync();   // every block has read the mark
    if (rank == 0 && threadIdx.x == 0) p.seq_lens[d] = L;
}

// ------------------------------------------------------------------------------------- release
// Drops a page-table entry: the exchange hands an entry that several threads drop to one of them.
__device__ __forceinline__ void drop_entry(const Pool &p, int *entry) {
    const int pg = atomicExch(entry, -1);
    if (pg < 0) return;   // dropped before
    if (pg >= p.n_pages) {
        report(p.err, MLA_ERR_DEVICE_BOUNDS);
        return;
    }
    if (atomicSub(p.refs + pg, 1) <= 0) {   // nobody held it
        atomicAdd(p.refs + pg, 1);
        report(p.err, MLA_ERR_DEVICE_BOUNDS);
    }
}

__global__ void __launch_bounds__(256) release_kernel(Pool p, const int *__restrict__ req, const int *__restrict__ first,
                                                      const int *__restrict__ last) {
    step_begin();
    const int b = req[blockIdx.x];
    if (b < 0 || b >= p.batch) {
        if (threadIdx.x == 0) report(p.err, MLA_ERR_DEVICE_BOUNDS);
        return;
    }
    const int L = p.seq_lens[b];
    if (!p.fits(L)) {
        if (threadIdx.x == 0) report(p.err, MLA_ERR_DEVICE_BOUNDS);
        return;
    }
    int k0 = 0, k1 = p.pages_of(L);
    if (first) {
        k0 = max(0, first[blockIdx.x]);
        k1 = min(k1, last[blockIdx.x]);
    }
    for (int k = k0 + (int)threadIdx.x; k < k1; k += blockDim.x) drop_entry(p, p.entry(b, k));
    if (!first) {
        __syncthreads();
        if (threadIdx.x == 0) p.seq_lens[b] = 0;
    }
}

// ------------------------------------------------------------------------------------- accept
// Whether the accepted path of a request of length L is one: rows it has, node indices that rise and exist, in
// pages of the pool.  The same answer in every block of a call.  All threads of the block call it.
__device__ __forceinline__ bool path_ok(const Pool &p, int b, int L, int ctx, int n, const int *acc, int n_acc,
                                        int max_nodes) {
    int bad = 0;
    if (n < 0 || n > max_nodes || n_acc < 0 || n_acc > n || !p.fits(L) || ctx < 0 || (long long)ctx + n > L)
        bad = 1;
    else
        for (int k = threadIdx.x; k < n_acc; k += blockDim.x) {
            if (acc[k] >= n || acc[k] < k || (k && acc[k] <= acc[k - 1])) {   // indices that rise have acc[k] >= k
                bad = 1;
                break;
            }
            const int from = *p.entry(b, (ctx + acc[k]) / p.page), to = *p.entry(b, (ctx + k) / p.page);
            if (from < 0 || from >= p.n_pages || to < 0 || to >= p.n_pages) bad = 1;
        }
    return !__syncthreads_or(bad);
}

// Row acc[k] of the nodes moves to row k.  The indices rise, so acc[k] >= k: a thread that takes one
// column of every row in order never reads a row that it has overwritten, and needs no buffer.
struct Moves {
    int from_page[MLA_MAX_TREE_NODES], from_row[MLA_MAX_TREE_NODES], to_page[MLA_MAX_TREE_NODES], to_row[MLA_MAX_TREE_NODES];
};
template <typename V>
__device__ __forceinline__ void move_rows(const PageRows &rows, const Moves &m, int k_first, int n_acc, int rank, int blocks) {
    const int cols = rows.row_bytes / (int)sizeof(V);
    const long long n = (long long)rows.n_layers * rows.pieces * cols;
    constexpr int U = 8;
    for (long long id = (long long)rank * blockDim.x + threadIdx.x; id < n; id += (long long)blocks * blockDim.x) {
        const int unit = (int)(id / cols), c = (int)(id % cols);
        for (int k0 = k_first; k0 < n_acc; k0 += U) {
            V v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k0 + u < n_acc)
                    v[u] = reinterpret_cast<const V *>(rows.at(unit, m.from_page[k0 + u]) +
                                                       (size_t)m.from_row[k0 + u] * rows.row_bytes)[c];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k0 + u < n_acc)
                    reinterpret_cast<V *>(rows.at(unit, m.to_page[k0 + u]) + (size_t)m.to_row[k0 + u] * rows.row_bytes)[c] = v[u];
        }
    }
}

// One cluster per request: moves the rows of every layer, then trims the request.
// 288 is the largest block of which an SM's registers hold four with the eight loads a thread has in flight
// (56 each).  64 requests, latent rows of 8 / 27 / 60 / 128 layers, accept and a reserve: 192 threads 6.8 / 9.8 /
// 11.9 / 18.1 us, 256: 7.0 / 8.2 / 13.1 / 18.5, 288: 6.8 / 8.6 / 11.5 / 17.0, 320: 6.6 / 8.8 / 12.1 / 18.4; one pass of
// up to 1,024 threads instead of several: 6.6 / 8.2 / 14.0 / 19.5.
constexpr int ACCEPT_THREADS = 288;

__global__ void __launch_bounds__(ACCEPT_THREADS, 4) accept_kernel(Pool p, const int *__restrict__ ctx_lens,
                                                     const int *__restrict__ n_nodes, const int *__restrict__ accepted,
                                                     const int *__restrict__ n_accepted, int max_nodes, RowSets sets) {
    step_begin();
    const int rank = blockIdx.x, blocks = gridDim.x, b = blockIdx.y;
    const int ctx = ctx_lens[b], n = n_nodes[b], n_acc = n_accepted[b];
    const int *acc = accepted + (size_t)b * max_nodes;
    if (n == 0 && n_acc == 0) return;   // takes no part (the whole cluster)
    const int L = p.seq_lens[b];
    const bool ok = path_ok(p, b, L, ctx, n, acc, n_acc, max_nodes);
    __shared__ Moves m;
    __shared__ int n_move;
    if (threadIdx.x == 0) n_move = 0;
    __syncthreads();
    if (ok) {
        // Rows that stay are the first ones (acc[k] = k only while every node so far is accepted).
        if (threadIdx.x < n_acc) {
            const int k = threadIdx.x, t0 = ctx + acc[k], t1 = ctx + k;
            m.from_page[k] = *p.entry(b, t0 / p.page), m.from_row[k] = t0 % p.page;
            m.to_page[k] = *p.entry(b, t1 / p.page), m.to_row[k] = t1 % p.page;
            if (acc[k] != k) atomicAdd(&n_move, 1);
        }
        __syncthreads();
        if (n_move)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i >= sets.n) break;
                const PageRows &r = sets.r[i];
                if (r.vec == 16) move_rows<uint4>(r, m, n_acc - n_move, n_acc, rank, blocks);
                else if (r.vec == 4) move_rows<uint32_t>(r, m, n_acc - n_move, n_acc, rank, blocks);
                else move_rows<uint16_t>(r, m, n_acc - n_move, n_acc, rank, blocks);
            }
    }
    cooperative_groups::this_cluster().sync();   // every block has read the page table
    if (rank) return;
    if (!ok) {
        if (threadIdx.x == 0) report(p.err, MLA_ERR_DEVICE_BOUNDS);
        return;
    }
    if (p.refs)
        for (int k = p.pages_of(ctx + n_acc) + (int)threadIdx.x; k < p.pages_of(L); k += blockDim.x)
            drop_entry(p, p.entry(b, k));
    if (threadIdx.x == 0) p.seq_lens[b] = ctx + n_acc;
}

Pool pool_of(const PagePool &a) {
    return Pool{a.seq_lens, a.page_table, a.refs, a.batch, a.max_pages, a.n_pages, a.page, a.err};
}

// Launches one cluster of `blocks` blocks for each of `n` requests.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), int blocks, int threads, int n, cudaStream_t st, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, n);
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

RowSets sets_of(const PageRows *rows, int n) {
    RowSets s{};
    for (s.n = 0; s.n < n; ++s.n) s.r[s.n] = rows[s.n];
    return s;
}

}  // namespace

cudaError_t launch_cache_reserve(const PagePool &a, const int *new_lens, cudaStream_t st) {
    MLA_STEP_LAUNCH(reserve_kernel, dim3(1), dim3(PT), 0, st, pool_of(a), new_lens);
    return cudaGetLastError();
}

cudaError_t launch_cache_fork(const PagePool &a, const int *src, const int *dst, int n_fork, const PageRows *rows, int n_rows,
                              cudaStream_t st) {
    static std::atomic<unsigned long long> calls{0};
    const Pool p = pool_of(a);
    const unsigned long long call = calls.fetch_add(1, std::memory_order_relaxed) + 1;   // never 0
    MLA_STEP_LAUNCH(fork_plan_kernel, dim3(1), dim3(PT), 0, st, p, src, dst, n_fork, call);
    return launch_clusters(fork_copy_kernel, 8, 256, n_fork, st, p, src, dst, sets_of(rows, n_rows), call);
}

cudaError_t launch_cache_release(const PagePool &a, const int *req, const int *first, const int *last, int n_req,
                                 cudaStream_t st) {
    MLA_STEP_LAUNCH(release_kernel, dim3(n_req), dim3(256), 0, st, pool_of(a), req, first, last);
    return cudaGetLastError();
}

cudaError_t launch_cache_accept(const PagePool &a, const int *ctx, const int *n_nodes, const int *accepted,
                                const int *n_accepted, int max_nodes, const PageRows *rows, int n_rows, cudaStream_t st) {
    // Blocks enough for one pass over the columns of all rows, up to the portable cluster's eight.
    long long cols = 1;
    for (int i = 0; i < n_rows; ++i)
        cols = std::max(cols, (long long)rows[i].n_layers * rows[i].pieces * (rows[i].row_bytes / rows[i].vec));
    constexpr int T = ACCEPT_THREADS;
    const int blocks = cols > 4 * T ? 8 : cols > 2 * T ? 4 : cols > T ? 2 : 1;
    return launch_clusters(accept_kernel, blocks, T, a.batch, st, pool_of(a), ctx, n_nodes, accepted, n_accepted, max_nodes,
                           sets_of(rows, n_rows));
}

}  // namespace mla
