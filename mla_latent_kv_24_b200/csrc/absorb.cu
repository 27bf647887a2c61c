// Query preparation.
//
// q absorption ("How to upgrade GQA models to MLA ...", stage "Decompression Multiplex": by
// associativity W_UK folds into the query, which then lives in latent space):
//     q_lat[row, h, :] = W_UK[w(h)]^T q_nope[row, h, :]                (d_c)
// followed by RoPE of the query's RoPE part at its position p = seq_lens[b] - s_q + j.
// Output q_abs[row, h, :] = [q_lat | RoPE(q_rope, p)], in the storage dtype (bf16 rounding
// once, fp32 accumulation).
//
// One CTA handles one head and up to RB query rows, so each W_UK row is read once per RB
// rows; every thread owns two latent columns.  The CTAs past the last head are the plan's: the first
// builds it, which saves a launch (float32 trees of the tiny shape: 23.4 -> 21.3 us a call).
//
// Queries, lengths and a tree's arrays may come from the kernel right before the call, so the kernels here read
// nothing before they have waited for it.
#include "kernels.h"
#include "plan_block.cuh"
#include "rope_rows.cuh"

namespace mla {
namespace {

constexpr int RB = 16;

template <typename T>
__global__ void __launch_bounds__(256) q_absorb_kernel(const T *q, const T *W_uk, const int *seq_lens, int rows, int s_q,
                                                       int H, int hpw, int d_c, int d_r, int d_n, float base,
                                                       T *__restrict__ q_abs, PlanArgs plan) {
    step_allow_next();
    step_wait_prev();
    __shared__ float qn[RB][128];
    if (blockIdx.x == H) {
        static_assert(sizeof(qn) >= sizeof(int) * (2 * 512 + 1), "the plan's scratch");
        if (grid_tile() == 0) plan_block<256>(plan, reinterpret_cast<int *>(qn), 512);
        return;
    }
    const int h = blockIdx.x, w = h / hpw;
    const int row0 = grid_tile() * RB;
    const int nr = min(RB, rows - row0);
    if (nr <= 0) return;
    const int d_qk = d_n + d_r, d_out = d_c + d_r;
    for (int i = threadIdx.x; i < RB * d_n; i += blockDim.x) {
        int r = i / d_n, k = i % d_n;
        qn[r][k] = r < nr ? to_f32(q[((size_t)(row0 + r) * H + h) * d_qk + k]) : 0.f;
    }
    __syncthreads();
    const T *Wk = W_uk + (size_t)w * d_n * d_c;
    // RoPE part: pair i of the query's RoPE vector turns by p * base^(-2i/d_r).
    auto angle = [&](int i, float *cs, float *sn) {
        const int row = row0 + i / (d_r / 2);
        rope_cos_sin(query_pos(plan.view, seq_lens, row / s_q, row % s_q, s_q), i % (d_r / 2), d_r, base, cs, sn);
    };
    const int pairs = nr * (d_r / 2);
    float cs = 0.f, sn = 0.f;
    if ((int)threadIdx.x < pairs) angle(threadIdx.x, &cs, &sn);
    for (int c = threadIdx.x; c < d_c; c += blockDim.x) {
        float acc[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) acc[r] = 0.f;
        for (int k = 0; k < d_n; ++k) {
            const float wv = to_f32(Wk[(size_t)k * d_c + c]);
#pragma unroll
            for (int r = 0; r < RB; ++r) acc[r] += qn[r][k] * wv;
        }
        for (int r = 0; r < nr; ++r) q_abs[((size_t)(row0 + r) * H + h) * d_out + c] = from_f32<T>(acc[r]);
    }
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
        const int r = i / (d_r / 2), pi = i % (d_r / 2), row = row0 + r;
        if (i != (int)threadIdx.x) angle(i, &cs, &sn);
        const T *src = q + ((size_t)row * H + h) * d_qk + d_n + 2 * pi;
        const float x0 = to_f32(src[0]), x1 = to_f32(src[1]);
        T *dst = q_abs + ((size_t)row * H + h) * d_out + d_c + 2 * pi;
        dst[0] = from_f32<T>(x0 * cs - x1 * sn);
        dst[1] = from_f32<T>(x0 * sn + x1 * cs);
    }
}

// GQA path: the no-position part is used as is; only the RoPE part turns.  A warp takes RH heads of a
// row: each lane forms one pair's angle, sine and cosine (in double) once for all of them.  (One angle
// per head and pair took 16 us for 64 rows, this 11; RH = 1, 2, 4, 8 come within 1 us of a call.)
// The last block builds the split plan instead.
constexpr int RH = 2;

template <typename T>
__global__ void __launch_bounds__(256) q_rope_kernel(const T *q, const int *seq_lens, int rows, int s_q, int H,
                                                     int d_r, int d_n, float base, T *__restrict__ q_rot, PlanArgs plan) {
    step_begin();
    if (blockIdx.x == gridDim.x - 1) {
        __shared__ int scratch[2 * 512 + 1];
        plan_block<256>(plan, scratch, 512);
        return;
    }
    const int d_qk = d_n + d_r, groups = ceil_div(H, RH), lane = threadIdx.x % 32;
    const long long n = (long long)rows * groups;
    const long long stride = (long long)(gridDim.x - 1) * (blockDim.x / 32);
    struct alignas(2 * sizeof(T)) Pair {
        T a, b;
    };
    const int quads = d_n * (int)sizeof(T) / 16;   // 16-byte pieces of a head's no-position part
    for (long long u = (long long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; u < n; u += stride) {
        const int row = (int)(u / groups), h0 = (int)(u % groups) * RH, nh = min(H - h0, RH);
        const int b = row / s_q, j = row % s_q, p = seq_lens[b] - s_q + j;
        const T *src = q + ((size_t)row * H + h0) * d_qk;
        T *dst = q_rot + ((size_t)row * H + h0) * d_qk;
        const bool turns = 2 * lane < d_r;
        auto piece = [&](auto *base, int i) {
            return reinterpret_cast<uint4 *>(const_cast<T *>(base) + (size_t)(i / quads) * d_qk) + i % quads;
        };
        Pair x[RH];
        uint4 first;
#pragma unroll
        for (int h = 0; h < RH; ++h)
            if (turns && h < nh) x[h] = *reinterpret_cast<const Pair *>(src + (size_t)h * d_qk + d_n + 2 * lane);
        if (lane < nh * quads) first = *piece(src, lane);
        float cs = 0.f, sn = 0.f;
        if (turns) rope_cos_sin(p, lane, d_r, base, &cs, &sn);
        if (lane < nh * quads) *piece(dst, lane) = first;
#pragma unroll 4
        for (int i = lane + 32; i < nh * quads; i += 32) *piece(dst, i) = *piece(src, i);
#pragma unroll
        for (int h = 0; h < RH; ++h)
            if (turns && h < nh) {
                const float x0 = to_f32(x[h].a), x1 = to_f32(x[h].b);
                // rounds once to the storage type, that of the QK^T operands
                *reinterpret_cast<Pair *>(dst + (size_t)h * d_qk + d_n + 2 * lane) =
                    Pair{from_f32<T>(x0 * cs - x1 * sn), from_f32<T>(x0 * sn + x1 * cs)};
            }
    }
}

}  // namespace

cudaError_t launch_q_absorb(const Dims &d, const void *q, const void *W_uk, const int *seq_lens, int batch,
                            int s_q, void *q_abs, const PlanArgs &plan, cudaStream_t st) {
    const int rows = batch * s_q;
    const dim3 grid = tile_grid(d.H + 1, ceil_div(rows, RB));
    if (d.bf16)
        MLA_STEP_LAUNCH(q_absorb_kernel<__nv_bfloat16>, dim3(grid), dim3(256), 0, st, (const __nv_bfloat16 *)q,
                        (const __nv_bfloat16 *)W_uk, seq_lens, rows, s_q, d.H, d.hpw, d.d_c, d.d_r, d.d_n, d.base,
                        (__nv_bfloat16 *)q_abs, plan);
    else
        MLA_STEP_LAUNCH(q_absorb_kernel<float>, dim3(grid), dim3(256), 0, st, (const float *)q, (const float *)W_uk,
                        seq_lens, rows, s_q, d.H, d.hpw, d.d_c, d.d_r, d.d_n, d.base, (float *)q_abs, plan);
    return cudaGetLastError();
}

cudaError_t launch_q_rope(const Dims &d, const void *q, const int *seq_lens, int batch, int s_q, void *q_rot,
                          const PlanArgs &plan, cudaStream_t st) {
    const int rows = batch * s_q;
    const size_t n = (size_t)rows * ceil_div(d.H, RH);
    const int blocks = (int)std::min<size_t>((n + 7) / 8, 4096) + 1;   // + the plan block
    if (d.bf16)
        MLA_STEP_LAUNCH(q_rope_kernel<__nv_bfloat16>, dim3(blocks), dim3(256), 0, st, (const __nv_bfloat16 *)q,
                        seq_lens, rows, s_q, d.H, d.d_r, d.d_n, d.base, (__nv_bfloat16 *)q_rot, plan);
    else
        MLA_STEP_LAUNCH(q_rope_kernel<float>, dim3(blocks), dim3(256), 0, st, (const float *)q, seq_lens, rows, s_q,
                        d.H, d.d_r, d.d_n, d.base, (float *)q_rot, plan);
    return cudaGetLastError();
}

}  // namespace mla

// ---------------------------------------------------------------------------------------
// Tensor-core q absorption for the DeepSeek-V2 shape (bf16, d_nope = 128, d_c = 512,
// d_rope = 64).  Per head it is the GEMM q_lat[rows, 512] = q_nope[rows, 128] W_UK[w]
// ([128, 512], row k = nope dim), with mma.sync m16n8k16: the W_UK tile [128 k][n] and the q tile are
// staged in padded shared memory by cp.async, B fragments come through ldmatrix.trans.  Every W_UK
// element is read once per head (16.8 MB in total for H = 128), the bound of this step for a few rows;
// for many it is the 147 KB written per row.
//
// Two forms.  Up to 16 rows one CTA computes 16 rows x 128 columns of one head, so that a decode step's
// whole grid (4 column tiles per head) is one wave of CTAs.  More rows: a CTA keeps its W_UK tile (128
// columns) and walks 64-row tiles of the batch, the next tile's queries arriving while this one is
// multiplied, and stores whole 256-byte row pieces through shared memory.  (With 64 x 64 tiles of their
// own, 4-byte stores and an angle per head: 82 us for 512 rows, 29 for 128; now 48 and 19.)
//
// The extra columns of blocks build the split plan (their first block) and turn the queries' RoPE part
// (rope_rows.cuh), so that each pair's double-precision angle is formed once for 16 heads and more.
// ---------------------------------------------------------------------------------------
#include "warp_mma.cuh"

namespace mla {
namespace {

constexpr int AB_K = 128, AB_LD = AB_K + 8, AB_N = 128, AB_LDB = AB_N + 8;
constexpr int D_C = 512, D_N = 128, D_R = 64, D_QK = 192, D_OUT = 576;

// One warp's 16 x (8 NT) product of the staged tiles.
template <int NT>
__device__ __forceinline__ void absorb_mma(float (*acc)[4], const __nv_bfloat16 *As, const __nv_bfloat16 *Bs, int m0, int n0,
                                           int lane) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < AB_K; kk += 16) {
        uint32_t a[4];
        ldmatrix_x4(a[0], a[1], a[2], a[3], As + (m0 + (lane % 8) + 8 * ((lane / 8) % 2)) * AB_LD + kk + 8 * (lane / 16));
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
            // B stored [k][n]: .trans gives the k-major fragments of two n8 tiles
            uint32_t b0, b1, b2, b3;
            const int kr = kk + (lane % 8) + 8 * ((lane / 8) % 2);
            const int nc = n0 + j * 8 + 8 * (lane / 16);
            ldmatrix_x4_trans(b0, b1, b2, b3, Bs + kr * AB_LDB + nc);
            mma_bf16(acc[j], a, b0, b1);
            mma_bf16(acc[j + 1], a, b2, b3);
        }
    }
}

__device__ __forceinline__ void absorb_load_w(__nv_bfloat16 *Bs, const __nv_bfloat16 *Wk, int n0) {
    for (int c = threadIdx.x; c < AB_K * AB_N / 8; c += 256) {   // 16-byte chunks of the W_UK tile
        const int k = c / (AB_N / 8), n = (c % (AB_N / 8)) * 8;
        cp_async16(Bs + k * AB_LDB + n, Wk + (size_t)k * D_C + n0 + n, true);
    }
}
template <int TM>
__device__ __forceinline__ void absorb_load_q(__nv_bfloat16 *As, const __nv_bfloat16 *q, int row0, int rows, int H, int h) {
    for (int c = threadIdx.x; c < TM * AB_K / 8; c += 256) {
        const int r = c / (AB_K / 8), k = (c % (AB_K / 8)) * 8, row = row0 + r;
        cp_async16(As + r * AB_LD + k, q + ((size_t)(row < rows ? row : 0) * H + h) * D_QK + k, row < rows);
    }
}

// Up to 16 rows: grid (H + extra, 4).
__global__ void __launch_bounds__(256) q_absorb_mma_kernel(const __nv_bfloat16 *q, const __nv_bfloat16 *W_uk,
                                                           const int *seq_lens, int rows, int s_q, int H, int hpw,
                                                           float base, __nv_bfloat16 *__restrict__ q_abs, PlanArgs plan) {
    step_allow_next();
    __shared__ __align__(16) __nv_bfloat16 As[16 * AB_LD];          // [rows][128 k]
    __shared__ __align__(16) __nv_bfloat16 Bs[AB_K * AB_LDB];       // [128 k][128 n]
    const int h = blockIdx.x, n0 = blockIdx.y * AB_N;
    const __nv_bfloat16 *Wk = W_uk + (size_t)(h / hpw) * D_N * D_C;
    step_wait_prev();
    if (h >= H) {
        rope_or_plan_block((h - H) * gridDim.y + blockIdx.y, q, seq_lens, rows, s_q, H, base, q_abs, plan,
                           reinterpret_cast<int *>(Bs), ((int)sizeof(Bs) / 4 - 1) / 2);
        return;
    }
    absorb_load_w(Bs, Wk, n0);
    absorb_load_q<16>(As, q, 0, rows, H, h);
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float acc[2][4];
    absorb_mma<2>(acc, As, Bs, 0, 16 * warp, lane);
    const int gid = lane / 4, t4 = lane % 4;
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
        const int row = gid + 8 * hr;
        if (row >= rows) continue;
        __nv_bfloat16 *dst = q_abs + ((size_t)row * H + h) * D_OUT + n0 + 16 * warp;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<uint32_t *>(dst + j * 8 + 2 * t4) = pack_bf16(acc[j][2 * hr], acc[j][2 * hr + 1]);
    }
}

// More rows: grid (H + extra, 4, z); a CTA takes the 64-row tiles blockIdx.z, blockIdx.z + z, ...
constexpr int ABR = 64;
constexpr size_t AB_ROWS_SMEM = sizeof(__nv_bfloat16) * (AB_K * AB_LDB + 2 * ABR * AB_LD);

__global__ void __launch_bounds__(256, 3) q_absorb_rows_kernel(const __nv_bfloat16 *q, const __nv_bfloat16 *W_uk,
                                                               const int *seq_lens, int rows, int s_q, int H, int hpw,
                                                               float base, __nv_bfloat16 *__restrict__ q_abs,
                                                               PlanArgs plan) {
    step_allow_next();
    extern __shared__ __align__(16) uint8_t absm[];
    __nv_bfloat16 *Bs = reinterpret_cast<__nv_bfloat16 *>(absm);    // [128 k][128 n]
    __nv_bfloat16 *As = Bs + AB_K * AB_LDB;                         // [2][64 rows][128 k]; a tile's output too
    const int h = blockIdx.x, n0 = blockIdx.y * AB_N;
    const __nv_bfloat16 *Wk = W_uk + (size_t)(h / hpw) * D_N * D_C;
    step_wait_prev();
    if (h >= H) {
        rope_or_plan_block(((h - H) * gridDim.z + blockIdx.z) * gridDim.y + blockIdx.y, q, seq_lens, rows, s_q, H, base,
                           q_abs, plan, reinterpret_cast<int *>(Bs), (AB_K * AB_LDB / 2 - 1) / 2);
        return;
    }
    const int tiles = ceil_div(rows, ABR), warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int gid = lane / 4, t4 = lane % 4, m0 = 16 * (warp % 4), c0 = 64 * (warp / 4);
    absorb_load_w(Bs, Wk, n0);
    absorb_load_q<ABR>(As, q, blockIdx.z * ABR, rows, H, h);
    cp_async_commit();
    int buf = 0;
    for (int t = blockIdx.z; t < tiles; t += gridDim.z, buf ^= 1) {
        __nv_bfloat16 *A = As + buf * ABR * AB_LD;
        if (t + (int)gridDim.z < tiles) {
            absorb_load_q<ABR>(As + (buf ^ 1) * ABR * AB_LD, q, (t + gridDim.z) * ABR, rows, H, h);
            cp_async_commit();
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncthreads();
        float acc[8][4];
        absorb_mma<8>(acc, A, Bs, m0, c0, lane);
        __syncthreads();   // the queries are read: their tile takes the output
#pragma unroll
        for (int hr = 0; hr < 2; ++hr)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint32_t *>(A + (m0 + gid + 8 * hr) * AB_LD + c0 + 8 * j + 2 * t4) =
                    pack_bf16(acc[j][2 * hr], acc[j][2 * hr + 1]);
        __syncthreads();
        for (int c = threadIdx.x; c < ABR * AB_N / 8; c += 256) {
            const int r = c / (AB_N / 8), n = (c % (AB_N / 8)) * 8, row = t * ABR + r;
            if (row < rows)
                *reinterpret_cast<uint4 *>(q_abs + ((size_t)row * H + h) * D_OUT + n0 + n) =
                    *reinterpret_cast<const uint4 *>(A + r * AB_LD + n);
        }
        __syncthreads();   // the tile after next arrives here
    }
}

}  // namespace

bool q_absorb_mma_ok(const Dims &d) { return d.bf16 && d.d_n == 128 && d.d_c == 512 && d.d_r == 64; }

cudaError_t launch_q_absorb_mma(const Dims &d, const void *q, const void *W_uk, const int *seq_lens, int batch,
                                int s_q, void *q_abs, const PlanArgs &plan, cudaStream_t st) {
    const int rows = batch * s_q;
    constexpr int Y = D_C / AB_N;
    if (rows <= 16) {
        dim3 grid(d.H + ceil_div(1 + rope_blocks(rows), Y), Y, 1);
        MLA_STEP_LAUNCH(q_absorb_mma_kernel, grid, dim3(256), 0, st, (const __nv_bfloat16 *)q,
                        (const __nv_bfloat16 *)W_uk, seq_lens, rows, s_q, d.H, d.hpw, d.base, (__nv_bfloat16 *)q_abs,
                        plan);
    } else {
        // Two tiles per CTA: enough to hide the queries' loads, short enough to share the SMs evenly.
        const int z = std::min(ceil_div(ceil_div(rows, ABR), 2), 65535);
        const long long per = (long long)Y * z;
        dim3 grid(d.H + (unsigned)((rope_blocks(rows) + per) / per), Y, z);   // + the plan's and the RoPE blocks
        cudaError_t e = raise_smem_limit((const void *)q_absorb_rows_kernel, AB_ROWS_SMEM);
        if (e != cudaSuccess) return e;
        MLA_STEP_LAUNCH(q_absorb_rows_kernel, grid, dim3(256), AB_ROWS_SMEM, st, (const __nv_bfloat16 *)q,
                        (const __nv_bfloat16 *)W_uk, seq_lens, rows, s_q, d.H, d.hpw, d.base, (__nv_bfloat16 *)q_abs,
                        plan);
    }
    return cudaGetLastError();
}

}  // namespace mla
