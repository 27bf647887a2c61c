// Query positions, and the RoPE part of the absorbed query for the DeepSeek-V2 shape (d_nope = 128,
// d_rope = 64, d_c = 512), as blocks of the absorption's kernels.
#pragma once

#include "plan_block.cuh"
#include "warp_mma.cuh"

namespace mla {

// Position of query j of request b: the s_q queries are the request's last tokens, and a tree's
// node sits at its depth behind the context.
__device__ __forceinline__ int query_pos(const View &v, const int *seq_lens, int b, int j, int s_q) {
    if (v.kind == VIEW_TREE) return seq_lens[b] - v.n_nodes[b] + v.depths[(size_t)b * s_q + j];
    return seq_lens[b] - s_q + j;
}

constexpr int ROPE_D_QK = 192, ROPE_D_OUT = 576;

// Warps that share a row's heads: eight for few rows, down to one, so that the blocks stay about as many as
// half the SMs (each holds the shared memory of the kernel that it is part of).
__host__ __device__ __forceinline__ int rope_warps(int rows) { return rows <= 64 ? 8 : rows <= 128 ? 4 : rows <= 256 ? 2 : 1; }
__host__ __device__ __forceinline__ int rope_blocks(int rows) { return ceil_div(rows * rope_warps(rows), 8); }

// A block past the heads' ones, `id` counting them: the first builds the split plan, the next
// rope_blocks(rows) turn the RoPE part of the queries.  A warp takes every rope_warps()-th head of a row, so
// that each pair's double-precision angle is formed once for 16 heads and more.  256 threads; `scratch`
// has 2 cap + 1 ints.  After step_wait_prev().
__device__ __forceinline__ void rope_or_plan_block(int id, const __nv_bfloat16 *q, const int *seq_lens, int rows, int s_q,
                                                   int H, float base, __nv_bfloat16 *__restrict__ q_abs,
                                                   const PlanArgs &plan, int *scratch, int cap) {
    if (id == 0) {
        plan_block<256>(plan, scratch, cap);
        return;
    }
    const int wpr = rope_warps(rows), u = (id - 1) * 8 + (int)threadIdx.x / 32, lane = threadIdx.x % 32;
    const int row = u / wpr, first = u % wpr;
    if (row >= rows) return;
    constexpr int U = 16;
    const int b = row / s_q, j = row % s_q;
    const __nv_bfloat16 *src = q + (size_t)row * H * ROPE_D_QK + 128 + 2 * lane;
    __nv_bfloat16 *dst = q_abs + (size_t)row * H * ROPE_D_OUT + 512 + 2 * lane;
    uint32_t x[U];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = h0 + wpr * i;
            x[i] = h < H ? *reinterpret_cast<const uint32_t *>(src + (size_t)h * ROPE_D_QK) : 0u;
        }
    };
    load(first);
    float cs, sn;
    rope_cos_sin(query_pos(plan.view, seq_lens, b, j, s_q), lane, 64, base, &cs, &sn);
    for (int h0 = first; h0 < H; h0 += U * wpr) {
        uint32_t y[U];   // rounds once to bf16, the type of the QK^T operands, as the absorbed part does
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const float x0 = __uint_as_float(x[i] << 16), x1 = __uint_as_float(x[i] & 0xffff0000u);
            y[i] = pack_bf16(x0 * cs - x1 * sn, x0 * sn + x1 * cs);
        }
        load(h0 + U * wpr);
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (h0 + wpr * i < H) *reinterpret_cast<uint32_t *>(dst + (size_t)(h0 + wpr * i) * ROPE_D_OUT) = y[i];
    }
}

}  // namespace mla
