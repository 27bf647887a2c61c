// The per-head products around a tree's or window's decode on the 5th-generation tensor cores, for
// batches with many query rows (bf16, d_nope = d_v = 128, d_c = 512, d_rope = 64):
//
//   absorption   q_lat[rows, 512] = q_nope[rows, 128] W_UK[w]                       (K = 128)
//   projection   out[rows, 128]   = (merged O)[rows, 512] W_UV[w]^T                 (K = 512)
//
// for each of the H heads.  A decode over a tree of 64 nodes and 8 requests has 512 rows, so that a head's
// products are 128-row tiles of tcgen05.mma (one CTA, cta_group::1); on mma.sync they ran at
// 180-215 TFLOP/s and took a tenth of the call.  Both are bound by memory here: 147 KB of q_abs written
// and 256 KB of partials read per row, against 17 and 34 MFLOP.  For 512 rows of one chunk the absorption takes 35 us
// (3.3 TB/s), the projection 49 (3.4 TB/s); for 128 rows of two chunks 14 and 21.
//
// Every wait is bounded.  A wait that runs out records MLA_ERR_TIMEOUT and ends the CTA's work: nothing more is
// issued or stored, copies in flight get time to land, and the tensor memory is freed.  The next kernel may launch only once a CTA holds its tensor memory: CTAs of two kernels share an
// SM's 512 columns, and one that waits for its predecessor must not hold what the predecessor still needs.
#include <math.h>

#include "plan_block.cuh"
#include "rope_rows.cuh"
#include "tc_decode.h"
#include "tc_ptx.cuh"
#include "tensor_map.h"
#include "warp_mma.cuh"

namespace mla {
namespace {

constexpr int D_C = 512, D_N = 128, D_R = 64, D_QK = 192, D_OUT = 576, D_V = 128;
constexpr int TM = 128;                        // rows of a tile
constexpr uint32_t BLK = TM * 128;             // 128 rows x 64 bf16, 128-byte swizzled

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
    // At once: until the permit is given up, the SM's other CTAs wait for it with their own allocation.
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// The CTA's tensor memory and barriers: set up by all threads, which then may let the next kernel launch.
struct Setup {
    uint32_t base, tmem;
    uint8_t *sbase;
};
template <int NBAR>
__device__ __forceinline__ Setup set_up(uint8_t *raw_smem, uint32_t bar_off, uint32_t cols) {
    Setup s;
    const uint32_t raw = tc::smem_addr(raw_smem);
    s.base = (raw + 1023u) & ~1023u;
    s.sbase = raw_smem + (s.base - raw);
    if (threadIdx.x == 0) {
        for (int i = 0; i < NBAR; ++i) tc::mbar_init(s.base + bar_off + 8 * i, 1);
        tc::fence_mbar_init();
    }
    if (threadIdx.x < 32) tmem_alloc(s.base + bar_off + 8 * NBAR, cols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    s.tmem = *reinterpret_cast<volatile uint32_t *>(s.sbase + bar_off + 8 * NBAR);
    return s;
}

// --------------------------------------------------------------------------- absorption
// One CTA: 128 rows x 256 latent columns of one head.  q_nope comes as two K-major blocks, W_UK as four
// N-major ones ([128 k][64 n]); eight MMAs M128 N256 K16; the tile leaves through shared memory as whole
// 512-byte row pieces.
constexpr uint32_t AB_A = 0, AB_B = 2 * BLK, AB_BAR = 6 * BLK;
constexpr uint32_t AB_SMEM = 1024 + AB_BAR + 32;
constexpr int AB_OUT_LD = 256 + 8;             // staged output row, in bf16
static_assert(TM * AB_OUT_LD * 2 <= AB_BAR, "the output is staged over the operands");
constexpr uint32_t AB_IDESC = tc::idesc_bf16_f32(TM, 256, false, true);

__global__ void __launch_bounds__(256) absorb_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                        const __grid_constant__ CUtensorMap tm_w,
                                                        const __nv_bfloat16 *q, const int *seq_lens, int rows, int s_q,
                                                        int H, int hpw, float base, __nv_bfloat16 *__restrict__ q_abs,
                                                        PlanArgs plan, WaitRule wr) {
    extern __shared__ uint8_t hsm[];
    const int h = blockIdx.x, n0 = blockIdx.y * 256, row0 = blockIdx.z * TM;
    if (h >= H) {
        step_begin();
        rope_or_plan_block(((h - H) * gridDim.z + blockIdx.z) * gridDim.y + blockIdx.y, q, seq_lens, rows, s_q, H, base,
                           q_abs, plan, reinterpret_cast<int *>(hsm), 4096);
        return;
    }
    const Setup s = set_up<2>(hsm, AB_BAR, 256);
    step_allow_next();
    step_wait_prev();   // queries may come from the kernel before, and q_abs is workspace that it may still read
    const uint32_t full = s.base + AB_BAR, done = full + 8;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    bool ok = true;
    if (threadIdx.x == 0) {
        tc::mbar_arrive_expect_tx(full, 6 * BLK);
        for (int i = 0; i < 2; ++i) tc::tma_load_3d(s.base + AB_A + BLK * i, &tm_q, 64 * i, h, row0, full);
        for (int i = 0; i < 4; ++i) tc::tma_load_2d(s.base + AB_B + BLK * i, &tm_w, n0 + 64 * i, (h / hpw) * D_N, full);
        ok = tc::mbar_wait_spin(full, 0, wr.limit_ns);
        if (ok) {
            tc::fence_after_sync();
            const uint64_t a = tc::sdesc_sw128(s.base + AB_A, 16, 1024), b = tc::sdesc_sw128(s.base + AB_B, BLK, 1024);
#pragma unroll
            for (int k = 0; k < D_N / 16; ++k)
                mma(s.tmem, tc::sdesc_add(a, (k / 4) * BLK + 32 * (k % 4)), tc::sdesc_add(b, 2048 * k), AB_IDESC, k > 0);
            if (wr.withhold != 0) commit(done);
        }
    }
    __syncwarp();
    // The operand wait comes before this one: twice the limit for the threads that wait from the start.
    if (ok) ok = tc::mbar_wait(done, 0, 2 * wr.limit_ns);
    if (__syncthreads_or(!ok)) {   // else every thread has passed the wait: the operands are read
        if (threadIdx.x == 0) report(plan.err, MLA_ERR_TIMEOUT);
        tc::drain_copies();
        tc::fence_before_sync();
        __syncthreads();
        if (warp == 0) {
            tc::fence_after_sync();
            tmem_free(s.tmem, 256);
        }
        return;
    }
    tc::fence_after_sync();
    __nv_bfloat16 *stage = reinterpret_cast<__nv_bfloat16 *>(s.sbase);
    const int r = 32 * (warp % 4) + lane;          // TMEM lane = row; warps 4-7 take the second 128 columns
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float v[64];
        const int col = 128 * (warp / 4) + 64 * c;
        tc::tmem_ld64(s.tmem + col + ((uint32_t)(32 * (warp % 4)) << 16), v);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(stage + r * AB_OUT_LD + col + 8 * i) =
                make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                           pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tmem_free(s.tmem, 256);
    }
    for (int i = warp; i < TM; i += 8) {
        const int row = row0 + i;
        if (row < rows)
            *reinterpret_cast<uint4 *>(q_abs + ((size_t)row * H + h) * D_OUT + n0 + 8 * lane) =
                *reinterpret_cast<const uint4 *>(stage + i * AB_OUT_LD + 8 * lane);
    }
}

// --------------------------------------------------------------------------- projection
// One CTA: 128 rows of one head, eight K blocks of 64 latent columns through two stages.  The threads merge
// the rows' chunk partials of a block (a row with one chunk, the usual case, is only scaled by 1 / l) and
// write them as two bf16 values hi + lo, K-major and swizzled as a tensor copy would, so that the product
// sees 16 bits of the merged latent; the W_UV block comes by TMA.  One thread issues the block's eight MMAs
// (hi and lo, M128 N128 K16) while the others merge the next one, whose partials are already in flight: two blocks of
// a row's only chunk, or a block of its first two.  Those registers leave room for one CTA on an SM; with half of them
// and two CTAs, 128 rows of two chunks took 31 us instead of 21, and calls of 128 to 300 rows 1 to 2 us more.
constexpr uint32_t PJ_STAGE = 3 * BLK;         // hi | lo | W_UV
constexpr uint32_t PJ_INFO = 2 * PJ_STAGE;     // int k0[128], k1[128]; float w0[128], m[128], inv[128]
constexpr uint32_t PJ_BAR = PJ_INFO + 5 * 4 * TM;
constexpr uint32_t PJ_SMEM = 1024 + PJ_BAR + 64;
constexpr uint32_t PJ_IDESC = tc::idesc_bf16_f32(TM, D_V, false, false);
constexpr int KB = D_C / 64;
enum { P_FULL = 0, P_EMPTY = 2, P_COUNT = 4 };

constexpr int PJ_THREADS = 512;

__global__ void __launch_bounds__(PJ_THREADS, 1) project_tc_kernel(const __grid_constant__ CUtensorMap tm_w,
                                                            const float *__restrict__ part_o,
                                                            const float *__restrict__ part_ml,
                                                            const int *__restrict__ row_first, int rows, int H, int hpw,
                                                            __nv_bfloat16 *__restrict__ out, bool keep_empty, int *err,
                                                            WaitRule wr) {
    extern __shared__ uint8_t hsm[];
    const Setup s = set_up<P_COUNT>(hsm, PJ_BAR, 128);
    step_allow_next();
    auto bar = [&](int i) { return s.base + PJ_BAR + 8u * i; };
    const int h = blockIdx.x, row0 = blockIdx.y * TM, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    auto load_w = [&](int kb) {
        tc::mbar_arrive_expect_tx(bar(P_FULL + (kb & 1)), BLK);
        tc::tma_load_2d(s.base + PJ_STAGE * (kb & 1) + 2 * BLK, &tm_w, 64 * kb, (h / hpw) * D_V, bar(P_FULL + (kb & 1)));
    };
    if (tid == 128) load_w(0), load_w(1);   // streams in while the decode finishes, which has waited for all before the call
    int *k0s = reinterpret_cast<int *>(s.sbase + PJ_INFO), *k1s = k0s + TM;
    float *w0s = reinterpret_cast<float *>(k1s + TM), *ms = w0s + TM, *invs = ms + TM;
    const float2 *ml = reinterpret_cast<const float2 *>(part_ml);
    step_wait_prev();
    if (tid < TM) {   // this row's chunks, merged maximum and 1 / sum
        const int row = row0 + tid;
        int k0 = 0, k1 = 0;
        if (row < rows) k0 = row_first[row], k1 = row_first[row + 1];
        float2 first = make_float2(-INFINITY, 0.f);
        if (k0 < k1) first = ml[(size_t)k0 * H + h];
        float M = first.x, den = first.y;
        for (int k = k0 + 1; k < k1; ++k) {
            const float2 v = ml[(size_t)k * H + h];
            const float Mn = fmaxf(M, v.x);
            if (Mn == -INFINITY) continue;   // nothing seen so far
            den = den * expf(M - Mn) + v.y * expf(v.x - Mn);
            M = Mn;
        }
        const float inv = den > 0.f ? 1.f / den : 0.f;
        k0s[tid] = k0, k1s[tid] = k1, ms[tid] = M, invs[tid] = inv;
        w0s[tid] = first.x == -INFINITY ? 0.f : expf(first.x - M) * inv;
    }
    __syncthreads();
    // A thread has columns 4 c4..4 c4 + 3 of a block, rows r0, r0 + 32, ...: a warp reads two rows' 256 bytes.
    constexpr int NR = TM * 16 / PJ_THREADS, RS = TM / NR;
    const int c4 = tid % 16, r0 = tid / 16;
    const float4 *src[NR];
    float w0[NR], w1[NR];
    uint32_t held = 0;   // bit i: row i has a chunk, bit NR + i: a second one
    int most = 0;        // chunks of this thread's row with the most
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = r0 + RS * i, k = k0s[r];
        src[i] = reinterpret_cast<const float4 *>(part_o + ((size_t)k * KB * H + h) * 64) + c4;
        w0[i] = w0s[r];
        held |= (uint32_t)(k < k1s[r]) << i;
        w1[i] = 0.f;
        if (k + 1 < k1s[r]) {
            held |= 1u << (NR + i);
            const float m1 = ml[(size_t)(k + 1) * H + h].x;
            w1[i] = m1 == -INFINITY ? 0.f : expf(m1 - ms[r]) * invs[r];
        }
        most = max(most, k1s[r] - k);
    }
    const size_t step = (size_t)H * 16;   // float4s from one block of 64 columns to the next
    float4 x[NR], x1[NR];
    auto load = [&](float4 (&v)[NR], int e, int kb) {   // block kb of every row's chunk e, 0 or 1
#pragma unroll
        for (int i = 0; i < NR; ++i)
            v[i] = (held >> (NR * e + i)) & 1u ? __ldcs(src[i] + (KB * e + kb) * step) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    bool ok = true;
    // Block kb, whose first chunks are in v; refill() fetches what v is to hold next.  A thread whose wait has run out
    // waits no more, issues nothing more, and meets the others at the end.
    auto block = [&](int kb, float4 (&v)[NR], auto merge, auto refill) {
        const int st = kb & 1;
        uint8_t *hi = s.sbase + PJ_STAGE * st, *lo = hi + BLK;
        if (kb >= 2 && ok) ok = tc::mbar_wait(bar(P_EMPTY + st), ((kb >> 1) - 1) & 1, wr.limit_ns);
#pragma unroll
        for (int i = 0; i < NR; ++i) v[i].x *= w0[i], v[i].y *= w0[i], v[i].z *= w0[i], v[i].w *= w0[i];
        merge();
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = r0 + RS * i;
            const uint32_t h0 = pack_bf16(v[i].x, v[i].y), h1 = pack_bf16(v[i].z, v[i].w);
            const uint32_t l0 = pack_bf16(v[i].x - __uint_as_float(h0 << 16), v[i].y - __uint_as_float(h0 & 0xffff0000u));
            const uint32_t l1 = pack_bf16(v[i].z - __uint_as_float(h1 << 16), v[i].w - __uint_as_float(h1 & 0xffff0000u));
            const uint32_t at = 128 * r + (((c4 / 2) ^ (r & 7)) << 4) + 8 * (c4 & 1);
            *reinterpret_cast<uint2 *>(hi + at) = make_uint2(h0, h1);
            *reinterpret_cast<uint2 *>(lo + at) = make_uint2(l0, l1);
        }
        refill();
        tc::fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            if (ok) ok = tc::mbar_wait_spin(bar(P_FULL + st), (kb >> 1) & 1, wr.limit_ns);
            if (ok) {
                tc::fence_after_sync();
                const uint64_t ah = tc::sdesc_sw128(s.base + PJ_STAGE * st, 16, 1024);
                const uint64_t b = tc::sdesc_add(ah, 2 * BLK);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mma(s.tmem, tc::sdesc_add(ah, 32 * k), tc::sdesc_add(b, 32 * k), PJ_IDESC, kb > 0 || k > 0);
                    mma(s.tmem, tc::sdesc_add(ah, BLK + 32 * k), tc::sdesc_add(b, 32 * k), PJ_IDESC, true);
                }
                if (kb != wr.withhold) commit(bar(P_EMPTY + st));
            }
        } else if (tid == 128 && kb >= 1 && kb + 1 < KB) {
            // The W_UV block after this one takes the place of the one before it.
            if (ok) ok = tc::mbar_wait(bar(P_EMPTY + (st ^ 1)), ((kb - 1) >> 1) & 1, wr.limit_ns);
            if (ok) load_w(kb + 1);
        }
        __syncwarp();
    };
    // Chunks from the e0-th on, the e-th of every row together, into x.
    auto merge_from = [&](int e0, int kb) {
        for (int e = e0; e < most; ++e) {
            float4 y[NR];
            float wk[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int r = r0 + RS * i, k = k0s[r] + e;
                y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                wk[i] = -INFINITY;
                if (k < k1s[r]) {
                    wk[i] = ml[(size_t)k * H + h].x;
                    y[i] = __ldcs(src[i] + e * (KB * step) + kb * step);
                }
            }
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int r = r0 + RS * i;
                const float w = wk[i] == -INFINITY ? 0.f : expf(wk[i] - ms[r]) * invs[r];
                x[i].x += w * y[i].x, x[i].y += w * y[i].y, x[i].z += w * y[i].z, x[i].w += w * y[i].w;
            }
        }
    };
    load(x, 0, 0);
    if (__syncthreads_or(most > 1)) {   // two chunks of every row in flight
        load(x1, 1, 0);
#pragma unroll 1
        for (int kb = 0; kb < KB; ++kb)
            block(kb, x,
                  [&] {
#pragma unroll
                      for (int i = 0; i < NR; ++i)
                          x[i].x += w1[i] * x1[i].x, x[i].y += w1[i] * x1[i].y, x[i].z += w1[i] * x1[i].z, x[i].w += w1[i] * x1[i].w;
                      merge_from(2, kb);
                  },
                  [&] { if (kb + 1 < KB) load(x, 0, kb + 1), load(x1, 1, kb + 1); });
    } else {   // two blocks of every row's only chunk in flight
        load(x1, 0, 1);
#pragma unroll 1
        for (int kb = 0; kb < KB; kb += 2) {
            block(kb, x, [] {}, [&] { if (kb + 2 < KB) load(x, 0, kb + 2); });
            block(kb + 1, x1, [] {}, [&] { if (kb + 3 < KB) load(x1, 0, kb + 3); });
        }
    }
    if (ok) ok = tc::mbar_wait(bar(P_EMPTY + 1), ((KB - 1) >> 1) & 1, wr.limit_ns);
    if (__syncthreads_or(!ok)) {
        if (tid == 0) report(err, MLA_ERR_TIMEOUT);
        tc::drain_copies();
        tc::fence_before_sync();
        __syncthreads();
        if (warp == 0) {
            tc::fence_after_sync();
            tmem_free(s.tmem, 128);
        }
        return;
    }
    tc::fence_after_sync();
    const int row = row0 + 32 * (warp % 4) + lane, col = 32 * (warp / 4);
    float v[32];
    tc::tmem_ld32(s.tmem + col + ((uint32_t)(32 * (warp % 4)) << 16), v);
    tc::tmem_wait_ld();
    if (row < rows && !(keep_empty && k0s[row - row0] == k1s[row - row0])) {
        uint4 *dst = reinterpret_cast<uint4 *>(out + ((size_t)row * H + h) * D_V + col);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tmem_free(s.tmem, 128);
    }
}

// --------------------------------------------------------------------------- tensor maps
// Boxes of 64 columns x 128 rows, 128-byte swizzle: of a row-major matrix [rows, cols], or with heads > 0 of
// one head of [rows, heads, cols].
bool encode_box(CUtensorMap *m, const void *ptr, uint64_t cols, uint64_t rows, uint64_t heads) {
    const cuuint64_t d2[2] = {cols, rows}, s2[1] = {cols * 2};
    const cuuint64_t d3[3] = {cols, heads, rows}, s3[2] = {cols * 2, cols * heads * 2};
    const cuuint32_t b2[2] = {64, TM}, b3[3] = {64, 1, TM};
    return heads ? encode_bf16_map(m, ptr, 3, d3, s3, b3) : encode_bf16_map(m, ptr, 2, d2, s2, b2);
}

}  // namespace

cudaError_t launch_absorb_tc(const Dims &d, const void *q, const void *W_uk, const int *seq_lens, int batch, int s_q,
                             void *q_abs, const PlanArgs &plan, cudaStream_t st) {
    const int rows = batch * s_q, z = ceil_div(rows, TM);
    if (z > 65535) return cudaErrorInvalidValue;
    CUtensorMap tm_q, tm_w;
    if (!encode_box(&tm_q, q, D_QK, rows, d.H) || !encode_box(&tm_w, W_uk, D_C, (uint64_t)d.n_groups() * D_N, 0))
        return cudaErrorInvalidValue;
    const long long per = 2ll * z;
    dim3 grid(d.H + (unsigned)((rope_blocks(rows) + per) / per), 2, z);   // + the plan's and the RoPE blocks
    cudaError_t e = raise_smem_limit((const void *)absorb_tc_kernel, AB_SMEM);
    if (e != cudaSuccess) return e;
    MLA_STEP_LAUNCH(absorb_tc_kernel, grid, dim3(256), AB_SMEM, st, tm_q, tm_w, (const __nv_bfloat16 *)q, seq_lens, rows,
                    s_q, d.H, d.hpw, d.base, (__nv_bfloat16 *)q_abs, plan, tc_wait_rule());
    return cudaGetLastError();
}

cudaError_t launch_project_tc(const Dims &d, const float *part_o, const float *part_ml, const int *row_first, int rows,
                              const void *W_uv, void *out, int *err, cudaStream_t st, bool keep_empty) {
    if (ceil_div(rows, TM) > 65535) return cudaErrorInvalidValue;
    CUtensorMap tm_w;
    if (!encode_box(&tm_w, W_uv, D_C, (uint64_t)d.n_groups() * D_V, 0)) return cudaErrorInvalidValue;
    cudaError_t e = raise_smem_limit((const void *)project_tc_kernel, PJ_SMEM);
    if (e != cudaSuccess) return e;
    MLA_STEP_LAUNCH(project_tc_kernel, dim3(d.H, ceil_div(rows, TM)), dim3(PJ_THREADS), PJ_SMEM, st, tm_w, part_o, part_ml,
                    row_first, rows, d.H, d.hpw, (__nv_bfloat16 *)out, keep_empty, err, tc_wait_rule());
    return cudaGetLastError();
}

}  // namespace mla
