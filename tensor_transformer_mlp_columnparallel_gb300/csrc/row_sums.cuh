// Sums over a row by the threads of a group.
#pragma once
#include "row_ring.cuh"

namespace tpmlp {
namespace {

// Sums (maxima) of V numbers over a group of NT threads (a power of two up to
// 1024), in every one of them. red: where the CTA's warps put theirs; not the
// place that the sum before used, so that one barrier is enough.
template <int NT, int V, typename Op>
__device__ __forceinline__ void group_reduce(float (&v)[V], int group, float (*red)[V], Op op) {
    const uint32_t lanes = group_lanes<NT>();
#pragma unroll
    for (int off = NT < 32 ? NT / 2 : 16; off > 0; off >>= 1)
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = op(v[k], __shfl_xor_sync(lanes, v[k], off));
    if constexpr (NT > 32) {
        constexpr int WARPS = NT / 32;
        const int lane = threadIdx.x & 31, warp = (threadIdx.x / 32) & (WARPS - 1);
        red += group * WARPS;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < V; ++k) red[warp][k] = v[k];
        group_sync<NT>(group);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = red[lane & (WARPS - 1)][k];
#pragma unroll
        for (int off = WARPS / 2; off > 0; off >>= 1)
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = op(v[k], __shfl_xor_sync(0xffffffffu, v[k], off));
    }
}
struct Add {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return max_nan(a, b); }
};

}  // namespace
}  // namespace tpmlp
