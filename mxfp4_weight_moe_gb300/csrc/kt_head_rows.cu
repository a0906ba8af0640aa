// kt_head_rows.cu -- per-head RMS norm and position rotation of query and key
// heads, to dense outputs or into the pages of a key/value cache, values copied
// along.  One launch per call; the operator is bound by memory traffic (large
// steps) or by launch latency (decode steps).
#include <type_traits>

#include "kt_head_rows_dev.cuh"
#include "kt_internal.h"

namespace kt {

// Four heads a group and six blocks of 128 threads on an SM: measured on 8192 tokens of 64 + 8 heads of 128 (302 MB of
// rows) with norms, 54.1 us (49.9 us, 6.1 TB/s, with the rows marked to leave L2); two heads 58 to 62 us, three 56.3,
// six 56.7, fewer blocks 57.6.  (With norms, six blocks cost 44 bytes of spills a thread.)
constexpr int kRowBlocks = 6, kRowHeads = 4;

template <typename T, int VEC, int R, int NORM, bool STREAM>
__global__ void __launch_bounds__(kRowThreads, kRowBlocks) head_rows_kernel(const HeadRowsParams p) {
    griddep_wait();
    griddep_launch_dependents();
    head_rows_block<T, VEC, R, NORM, STREAM>(p, blockIdx.x);
}

template <typename T, int VEC, int R, bool STREAM>
static cudaError_t launch_rows(HeadRowsParams& p, cudaStream_t s) {
    const dim3 grid(plan_head_rows<VEC, R>(p));
    count_launches(1);
    const bool norm = p.seg[0].weight != nullptr || p.seg[1].weight != nullptr;
    return launch_chained(!norm            ? head_rows_kernel<T, VEC, R, kNoNorm, STREAM>
                          : p.weight_f32   ? head_rows_kernel<T, VEC, R, kWeightsF32, STREAM>
                                           : head_rows_kernel<T, VEC, R, kWeightsTyped, STREAM>,
                          grid, dim3(kRowThreads), 0, s, static_cast<const HeadRowsParams&>(p));
}

template <typename T>
static cudaError_t launch_typed(HeadRowsParams& p, bool wide, cudaStream_t s) {
    const long long rows = static_cast<long long>(p.tokens) * (p.seg[0].heads + p.seg[1].heads + p.seg[2].heads);
    if (!wide) return launch_rows<T, 4, 1, false>(p, s);
    // few rows: one per group, so that they spread over the GPU; many: several, for the loads in flight
    if (rows < 16384) return launch_rows<T, 8, 1, false>(p, s);
    // Rows that pass through L2 (in and out, 128 MB of it) are marked to leave it first: 8192 tokens of 64 + 8 heads of
    // 128 in 49.4 us against 54.1.  What fits stays as it is: the projection has left it there, and attention reads it
    // next (2000 such tokens read and written in place of themselves: 11.4 us against 13.8 marked).
    if (rows * p.head_dim * 4 > (128ll << 20)) return launch_rows<T, 8, kRowHeads, true>(p, s);
    return launch_rows<T, 8, kRowHeads, false>(p, s);
}

cudaError_t launch_head_rows(HeadRowsParams& p, int dtype, bool wide, cudaStream_t s) {
    return dtype == KT_DTYPE_BF16 ? launch_typed<__nv_bfloat16>(p, wide, s) : launch_typed<__half>(p, wide, s);
}

}  // namespace kt
