// Shared device helpers for libmla kernels (sm_100a).
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <mutex>
#include <utility>

#include "mla.h"
#include "view.cuh"

namespace mla {

// ---------------------------------------------------------------------------------------
// Device error word: kernels never trap; they record the first error code and skip the
// offending access.  The host reads and clears it in mla_get_device_status().
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void report(int *err, int code) {
    if (err) atomicCAS(err, 0, code);
}

// ---------------------------------------------------------------------------------------
// Storage types.
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// RoPE angle for pair i of a d-wide vector at position pos: pos * base^(-2i/d), with the
// product and the trigonometry in double precision so that large positions (2^17) keep
// full single-precision accuracy after rounding.
__device__ __forceinline__ void rope_cos_sin(int pos, int i, int d, float base, float *c, float *s) {
    double theta = pow((double)base, -2.0 * (double)i / (double)d);
    double ang = (double)pos * theta;
    double sd, cd;
    sincos(ang, &sd, &cd);
    *c = (float)cd;
    *s = (float)sd;
}

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Row tiles over a grid's y and z, which hold 65,535 each: 2^20 rows in tiles of eight are twice that.  A few
// blocks past the last tile may come with it.
inline dim3 tile_grid(unsigned x, int tiles) {
    const int z = ceil_div(tiles, 65535);
    return dim3(x, ceil_div(tiles, z), z);
}
__device__ __forceinline__ int grid_tile() { return (int)(blockIdx.z * gridDim.y + blockIdx.y); }

// ---------------------------------------------------------------------------------------
// Programmatic dependent launch.  The kernels of a call are launched with programmatic stream
// serialisation, so a kernel's CTAs may be launched while the previous kernel of the stream is
// still running: the caller's own kernel too, when that one lets its dependents launch before its
// last stores, and without that as soon as its last block has ended, when its writes need not be visible
// yet.  So no kernel reads or writes global memory before step_wait_prev(), which waits
// until the previous kernel has completed and its writes are visible (griddepcontrol.wait).  Every
// kernel waits in at least one thread of each grid, so a kernel that has completed has seen all its
// predecessors complete, and execution and memory order stay those of a plain stream.
//
// step_allow_next() lets the next kernel launch (griddepcontrol.launch_dependents), so that its
// launch latency, its barriers and its tensor-memory allocation overlap this kernel.  Both do nothing
// in a kernel launched without the attribute.  step_begin() is the two in a row, for kernels that do
// nothing ahead.
//
// The one exception: the kernels that merge and multiply by W_UV load it ahead of their wait.  Every
// decode kernel waits before it lets them launch, so the call's first kernel, and with it all that came
// before the call, has completed by then.  (Fetching the other kernels' weights into L2 ahead gained nothing
// measurable, behind other kernels or in a row of calls.)
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void step_allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void step_wait_prev() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void step_begin() {
    step_wait_prev();
    step_allow_next();
}

// ---------------------------------------------------------------------------------------
// Split-KV plan.  Row r = (b, j) has len_r = seq_lens[b] - s_q + j + 1 visible tokens and
// is cut into ceil(len_r / chunk) chunks of `chunk` tokens (the last one ragged).  Work item
// k covers tokens [t0, t1) of one row; partial results are stored at index k.
// ---------------------------------------------------------------------------------------
struct WorkItem {
    int row;     // b * s_q + j
    int t0, t1;  // token range
    int split;   // chunk index inside the row
};

// Inputs and outputs of the device-side plan builder (plan_block.cuh).
struct PlanArgs {
    const int *seq_lens;
    int batch, s_q, max_pages, page, chunk, n_expected;   // s_q: plan rows per request
    WorkItem *items;     // [n_expected]
    int *row_first;      // [batch * s_q + 1]
    int *err;
    int *order;          // optional: [n_expected] take order of the items (see plan_block), then
                         // [batch * s_q + 1] scratch
    View view;           // which tokens the rows see (default: causal)
    int n_q;             // window and tree views: queries per request
};

struct Plan {
    const WorkItem *items;  // [n_work]
    const int *row_first;   // [rows + 1] first work item of each row (prefix sums)
    int n_work;
    int rows;
    int chunk;
    const int *order;       // nullptr, or the order in which a persistent decode takes the items
};

}  // namespace mla

namespace mla {
// Launches `kernel` on `st` with programmatic stream serialisation (the kernel must call
// step_begin() or step_wait_prev(), as above).  Host only.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_step(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                               Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// One statement: launch with launch_step() and return its error, if any, from the caller.
#define MLA_STEP_LAUNCH(kernel, grid, block, smem, st, ...)                                       \
    do {                                                                                          \
        const cudaError_t e_launch_ = ::mla::launch_step(kernel, grid, block, smem, st, __VA_ARGS__); \
        if (e_launch_ != cudaSuccess) return e_launch_;                                           \
    } while (0)

// Raises a kernel's dynamic shared-memory limit on the current device once, to the largest size
// asked so far; later launches that need no more skip the driver call (it costs microseconds of
// host time per launch).  Host only; thread-safe.
inline cudaError_t raise_smem_limit(const void *kernel, size_t bytes) {
    struct Entry {
        const void *kernel;
        int device;
        size_t bytes;
    };
    static std::mutex mu;
    static Entry table[256];
    static int n = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    Entry *hit = nullptr;
    for (int i = 0; i < n; ++i)
        if (table[i].kernel == kernel && table[i].device == dev) hit = &table[i];
    if (hit && hit->bytes >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    if (hit)
        hit->bytes = bytes;
    else if (n < 256)
        table[n++] = Entry{kernel, dev, bytes};
    return cudaSuccess;
}
}  // namespace mla
