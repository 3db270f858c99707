// What the split linear layers' backward does besides its products:
//   dZ = dY act'(Z),  db = sum_n dZ
// in one pass over dY and Z, which memory bounds: a thread has one access's
// columns of a chunk of rows, writes dZ and keeps the columns' sums (of dZ
// before it is rounded) in fp32; a second launch adds the chunks in order.
#include <cuda_bf16.h>

#include "access.cuh"
#include "ptx.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int COLS = 128;   // threads (accesses) of a CTA

struct DactParams {
    DactArgs a;
    int S;
};

template <typename T> __device__ __forceinline__ float slope(int act, float z);
template <> __device__ __forceinline__ float slope<float>(int act, float z) { return act_grad(act, z); }
template <> __device__ __forceinline__ float slope<__nv_bfloat16>(int act, float z) {
    return act_grad_bf16(act, z);
}

template <typename T, int B, int ACT>
__global__ void __launch_bounds__(COLS) dact_kernel(const DactParams p) {
    using A = Access<T, B>;
    using Word = typename A::Word;
    const DactArgs& a = p.a;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t at = (int64_t)blockIdx.x * COLS + threadIdx.x;
    if (at >= a.F / A::N) return;
    const int64_t lo = a.N * blockIdx.y / p.S, hi = a.N * (blockIdx.y + 1) / p.S;
    float sum[A::N];
#pragma unroll
    for (int j = 0; j < A::N; ++j) sum[j] = 0.f;
#pragma unroll 4
    for (int64_t row = lo; row < hi; ++row) {
        float g[A::N], z[A::N];
        A::unpack(reinterpret_cast<const Word*>(static_cast<const T*>(a.dY) + row * a.lddy)[at], g);
        A::unpack(reinterpret_cast<const Word*>(static_cast<const T*>(a.Z) + row * a.ldz)[at], z);
#pragma unroll
        for (int j = 0; j < A::N; ++j) {
            g[j] *= slope<T>(ACT, z[j]);
            sum[j] += g[j];
        }
        const Word w = A::pack(g);
        reinterpret_cast<Word*>(static_cast<T*>(a.dZ) + row * a.F)[at] = w;
        if (a.rest) {
            A::unpack(w, z);
#pragma unroll
            for (int j = 0; j < A::N; ++j) g[j] -= z[j];
            reinterpret_cast<Word*>(static_cast<T*>(a.dZ) + (a.N + row) * a.F)[at] = A::pack(g);
        }
    }
    if (a.db[0] != nullptr) {
        float* out = a.part + (int64_t)blockIdx.y * a.F + at * A::N;
#pragma unroll
        for (int j = 0; j < A::N; ++j) out[j] = sum[j];
    }
}

// 32 columns to a CTA, eight threads to a column's chunks.
template <typename T>
__global__ void __launch_bounds__(256) dact_sums_kernel(const DactParams p) {
    __shared__ float red[8][33];
    const DactArgs& a = p.a;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    const int lo = p.S * grp / 8, hi = p.S * (grp + 1) / 8;
    float s = 0.f;
    if (c < a.F) {
#pragma unroll 8
        for (int k = lo; k < hi; ++k) s += a.part[(int64_t)k * a.F + c];
    }
    red[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && c < a.F) {
        for (int k = 1; k < 8; ++k) s += red[k][lane];
        const int64_t Fs = a.F / a.T;
        T* out = static_cast<T*>(a.db[c / Fs]) + c % Fs;
        if constexpr (sizeof(T) == 4)
            *out = s;
        else
            *out = __float2bfloat16_rn(s);
    }
}

int64_t chunks(int64_t N, int64_t F) {
    const int64_t blocks = (F + 1023) / 1024;
    int64_t S = 16LL * 152 / blocks;
    if (S > (N + 7) / 8) S = (N + 7) / 8;
    return S < 1 ? 1 : S > 1024 ? 1024 : S;
}

template <typename... P, typename... A>
tpmlp_status launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return TPMLP_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

template <typename T, int B>
tpmlp_status dact(int act, const DactParams& p, cudaStream_t s) {
    LaunchScope ls("linear_dact", s);
    const int64_t accesses = p.a.F / (B / (int)sizeof(T));
    const dim3 grid((unsigned)((accesses + COLS - 1) / COLS), (unsigned)p.S);
    tpmlp_status st;
    switch (act) {
        case TPMLP_ACT_RELU: st = launch(dact_kernel<T, B, TPMLP_ACT_RELU>, grid, COLS, s, p); break;
        case TPMLP_ACT_GELU_ERF: st = launch(dact_kernel<T, B, TPMLP_ACT_GELU_ERF>, grid, COLS, s, p); break;
        case TPMLP_ACT_GELU_SIGMOID: st = launch(dact_kernel<T, B, TPMLP_ACT_GELU_SIGMOID>, grid, COLS, s, p); break;
        default: st = launch(dact_kernel<T, B, TPMLP_ACT_GELU_TANH>, grid, COLS, s, p); break;
    }
    if (st != TPMLP_OK || p.a.db[0] == nullptr) return st;
    return launch(dact_sums_kernel<T>, dim3((unsigned)((p.a.F + 31) / 32)), 256, s, p);
}

}  // namespace

size_t dact_part_bytes(int64_t N, int64_t F) {
    return ((size_t)chunks(N, F) * (size_t)F * sizeof(float) + 255) & ~(size_t)255;
}

tpmlp_status run_dact(int f32, int act, const DactArgs& a, cudaStream_t s) {
    const DactParams p{a, (int)chunks(a.N, a.F)};
    if (!f32) return dact<__nv_bfloat16, 16>(act, p, s);   // 16-byte rows: the bf16 path's rule
    const bool wide = a.F % 4 == 0 && access_fits(a.dY, a.lddy * 4, 16) && access_fits(a.Z, a.ldz * 4, 16) &&
                      access_fits(a.dZ, a.F * 4, 16);
    return wide ? dact<float, 16>(act, p, s) : dact<float, 4>(act, p, s);
}

}  // namespace tpmlp
