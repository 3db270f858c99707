// Layer norm over rows, forward and backward.
//
//   mean = sum x / D,  var = sum (x - mean)^2 / D,  rstd = 1 / sqrt(var + eps)
//   h = (x - mean) rstd,  y = h w + b
//   u = dy w,  dx = rstd (u - sum u / D - h (sum u h) / D) + dresidual
//   dw = sum_n dy h,  db = sum_n dy
//
// Memory bounds both: a row's elements are read once and written once. The
// variance is taken around the row's own mean (a second pass over the elements
// a thread holds), never as a difference of squares. The fp32 mean m of a row
// far from zero is off by its sum's rounding, which is not small next to the
// row's spread; what it is off by, d = sum (x - m) / D, is known to many digits
// (x - m is exact where x and m are near), so every use of the mean is
// (x - m) - d. A row whose mean is within its spread takes d = 0: its m is
// better than such a d, which would hold m's own digits cut to those of x (bf16
// rows around zero, the mean's relative error 2e-6 instead of 4e-8).
#include <cuda_bf16.h>

#include "access.cuh"
#include "ptx.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int HELD_WORDS = 32;   // 32-bit registers of a row that a thread holds
constexpr int WIDEST = 1024;     // threads of the widest row

template <int NT> __device__ __forceinline__ float2 row_sum2(float a, float b, float2* red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, off);
        b += __shfl_xor_sync(0xffffffffu, b, off);
    }
    if constexpr (NT > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        __syncthreads();   // red may hold an earlier sum
        if (lane == 0) red[warp] = make_float2(a, b);
        __syncthreads();
        const float2 p = lane < NT / 32 ? red[lane] : make_float2(0.f, 0.f);
        a = p.x;
        b = p.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, off);
            b += __shfl_xor_sync(0xffffffffu, b, off);
        }
    }
    return make_float2(a, b);
}

template <int NT> __device__ __forceinline__ float row_max(float a, float2* red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, off));
    if constexpr (NT > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        __syncthreads();
        if (lane == 0) red[warp].x = a;
        __syncthreads();
        a = lane < NT / 32 ? red[lane].x : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, off));
    }
    return a;
}

// A row's statistics: x scaled by `scale` (1 but for rows whose squares
// overflow) has mean m + d and reciprocal deviation r.
struct RowStats {
    float scale, m, d, r;
    __device__ __forceinline__ float normal(float x) const { return (x * scale - m - d) * r; }
};

// each(f) calls f for every element of the row that this thread looks after.
template <int NT, typename Each>
__device__ __forceinline__ RowStats row_stats(int64_t D, float eps, float2* red, Each each) {
    const float inv = 1.f / (float)D;
    RowStats s{1.f, 0.f, 0.f, 0.f};
    float var = 0.f;
    auto take = [&]() {
        float a = 0.f;
        each([&](float x) { a += x * s.scale; });
        s.m = row_sum2<NT>(a, 0.f, red).x * inv;
        float c = 0.f, q = 0.f;
        each([&](float x) {
            const float t = x * s.scale - s.m;
            c += t;
            q = fmaf(t, t, q);
        });
        const float2 t = row_sum2<NT>(c, q, red);
        var = t.y * inv;
        s.d = s.m * s.m > var ? t.x * inv : 0.f;
        var = fmaxf(fmaf(-s.d, s.d, var), 0.f);
        if (t.y != t.y) var = t.y;   // (the maximum would drop a NaN)
    };
    take();
    if (!(var < INFINITY)) {   // the same for every thread of the row
        float big = 0.f;
        each([&](float x) { big = max_nan(big, fabsf(x)); });
        big = row_max<NT>(big, red);
        if (big < INFINITY) {   // finite elements: their squares overflowed
            s.scale = 0x1p-100f;
            take();
        }
    }
    s.r = 1.f / sqrtf(fmaf(eps * s.scale, s.scale, var));
    return s;
}

struct NormArgs {
    int64_t N, D;
    const void* x;
    int64_t ldx;
    const void* w;   // NULL: ones
    const void* b;   // NULL: zeros
    float eps;
    void* y;
    int64_t ldy;
    float* mean;     // NULL: not wanted
    float* rstd;
};

// A row in the registers of NT threads (a warp: four rows to a CTA), every
// access of B bytes. One reading of the row whatever D, up to 32 words a thread.
template <typename T, typename W, int B, int NT>
__global__ void __launch_bounds__(NT < 128 ? 128 : NT) layernorm_kernel(const NormArgs a) {
    using A = Access<T, B>;
    using Word = typename A::Word;
    constexpr int R = B >= 4 ? HELD_WORDS * 4 / B : HELD_WORDS;
    constexpr int ROWS = NT < 128 ? 128 / NT : 1;
    __shared__ float2 red[32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / NT : 0);
    if (row >= a.N) return;   // a whole warp
    const int t = ROWS > 1 ? threadIdx.x % NT : threadIdx.x;
    const int accesses = (int)(a.D / A::N);
    const Word* x = reinterpret_cast<const Word*>(static_cast<const T*>(a.x) + row * a.ldx);
    Word* y = reinterpret_cast<Word*>(static_cast<T*>(a.y) + row * a.ldy);
    Word held[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (t + i * NT < accesses) held[i] = x[t + i * NT];
    const RowStats s = row_stats<NT>(a.D, a.eps, red, [&](auto f) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (t + i * NT < accesses) {
                float v[A::N];
                A::unpack(held[i], v);
#pragma unroll
                for (int j = 0; j < A::N; ++j) f(v[j]);
            }
    });
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int at = t + i * NT;
        if (at < accesses) {
            float v[A::N], w[A::N], b[A::N];
            A::unpack(held[i], v);
            if (a.w) load_params<W, A::N>(static_cast<const W*>(a.w) + at * A::N, w);
            if (a.b) load_params<W, A::N>(static_cast<const W*>(a.b) + at * A::N, b);
#pragma unroll
            for (int j = 0; j < A::N; ++j) v[j] = fmaf(s.normal(v[j]), a.w ? w[j] : 1.f, a.b ? b[j] : 0.f);
            y[at] = A::pack(v);
        }
    }
    if (t == 0) {
        if (a.mean) a.mean[row] = (s.m + s.d) / s.scale;
        if (a.rstd) a.rstd[row] = s.r * s.scale;
    }
}

// A row of any length, read three times (from L2 but for the first).
template <typename T, typename W, int B>
__global__ void __launch_bounds__(WIDEST) layernorm_long_kernel(const NormArgs a) {
    using A = Access<T, B>;
    using Word = typename A::Word;
    __shared__ float2 red[32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const int64_t accesses = a.D / A::N;
    const Word* x = reinterpret_cast<const Word*>(static_cast<const T*>(a.x) + row * a.ldx);
    Word* y = reinterpret_cast<Word*>(static_cast<T*>(a.y) + row * a.ldy);
    const RowStats s = row_stats<WIDEST>(a.D, a.eps, red, [&](auto f) {
#pragma unroll 4
        for (int64_t at = threadIdx.x; at < accesses; at += WIDEST) {
            float v[A::N];
            A::unpack(x[at], v);
#pragma unroll
            for (int j = 0; j < A::N; ++j) f(v[j]);
        }
    });
    for (int64_t at = threadIdx.x; at < accesses; at += WIDEST) {
        float v[A::N], w[A::N], b[A::N];
        A::unpack(x[at], v);
        if (a.w) load_params<W, A::N>(static_cast<const W*>(a.w) + at * A::N, w);
        if (a.b) load_params<W, A::N>(static_cast<const W*>(a.b) + at * A::N, b);
#pragma unroll
        for (int j = 0; j < A::N; ++j) v[j] = fmaf(s.normal(v[j]), a.w ? w[j] : 1.f, a.b ? b[j] : 0.f);
        y[at] = A::pack(v);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = (s.m + s.d) / s.scale;
        if (a.rstd) a.rstd[row] = s.r * s.scale;
    }
}

// ------------------------------------------------------------- backward --

struct NormGradArgs {
    int64_t N, D;
    const void* dy;
    int64_t lddy;
    const void* x;
    int64_t ldx;
    const void* w;          // NULL: ones
    const float* mean;
    const float* rstd;
    const void* dres;       // NULL: zeros
    int64_t lddres;
    void* dx;
    int64_t lddx;
    void* dw;               // NULL (both): not wanted
    void* db;
    float4* rows;           // [N]: sum u / D, sum u h / D, sum h / D (what the mean is off by)
    float* part;            // [S, 2, D]: a row chunk's sums of dy h and dy
    int S;
};

// Sums over a row, one CTA each.
template <typename T, typename W, int B>
__global__ void __launch_bounds__(256) norm_grad_rows_kernel(const NormGradArgs a) {
    using A = Access<T, B>;
    using Word = typename A::Word;
    __shared__ float2 red[32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const int64_t accesses = a.D / A::N;
    const Word* x = reinterpret_cast<const Word*>(static_cast<const T*>(a.x) + row * a.ldx);
    const Word* dy = reinterpret_cast<const Word*>(static_cast<const T*>(a.dy) + row * a.lddy);
    const float m = a.mean[row], r = a.rstd[row];
    float su = 0.f, suh = 0.f, sh = 0.f;
#pragma unroll 2
    for (int64_t at = threadIdx.x; at < accesses; at += 256) {
        float v[A::N], g[A::N], w[A::N];
        A::unpack(x[at], v);
        A::unpack(dy[at], g);
        if (a.w) load_params<W, A::N>(static_cast<const W*>(a.w) + at * A::N, w);
#pragma unroll
        for (int j = 0; j < A::N; ++j) {
            const float h = (v[j] - m) * r, u = a.w ? g[j] * w[j] : g[j];
            su += u;
            suh = fmaf(u, h, suh);
            sh += h;
        }
    }
    const float inv = 1.f / (float)a.D;
    const float2 p = row_sum2<256>(su, suh, red);
    const float off = row_sum2<256>(sh, 0.f, red).x * inv, d = fabsf(m * r) > 1.f ? off : 0.f;
    if (threadIdx.x == 0) a.rows[row] = make_float4(p.x * inv, fmaf(-d, p.x, p.y) * inv, d, 0.f);
}

// dx, and a row chunk's column sums: a thread has one access's columns.
template <typename T, typename W, int B>
__global__ void __launch_bounds__(128) norm_grad_apply_kernel(const NormGradArgs a) {
    using A = Access<T, B>;
    using Word = typename A::Word;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t at = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (at >= a.D / A::N) return;
    const int64_t lo = a.N * blockIdx.y / gridDim.y, hi = a.N * (blockIdx.y + 1) / gridDim.y;
    float w[A::N], sw[A::N], sb[A::N];
    if (a.w) load_params<W, A::N>(static_cast<const W*>(a.w) + at * A::N, w);
#pragma unroll
    for (int j = 0; j < A::N; ++j) {
        if (!a.w) w[j] = 1.f;
        sw[j] = sb[j] = 0.f;
    }
#pragma unroll 4
    for (int64_t row = lo; row < hi; ++row) {
        float v[A::N], g[A::N], e[A::N];
        A::unpack(reinterpret_cast<const Word*>(static_cast<const T*>(a.x) + row * a.ldx)[at], v);
        A::unpack(reinterpret_cast<const Word*>(static_cast<const T*>(a.dy) + row * a.lddy)[at], g);
        if (a.dres) A::unpack(reinterpret_cast<const Word*>(static_cast<const T*>(a.dres) + row * a.lddres)[at], e);
        const float m = a.mean[row], r = a.rstd[row];
        const float4 s = a.rows[row];
#pragma unroll
        for (int j = 0; j < A::N; ++j) {
            const float h = fmaf(v[j] - m, r, -s.z);
            sw[j] = fmaf(g[j], h, sw[j]);
            sb[j] += g[j];
            v[j] = r * fmaf(-h, s.y, fmaf(g[j], w[j], -s.x));
            if (a.dres) v[j] += e[j];
        }
        reinterpret_cast<Word*>(static_cast<T*>(a.dx) + row * a.lddx)[at] = A::pack(v);
    }
    if (a.part != nullptr) {
        float* p = a.part + (int64_t)blockIdx.y * 2 * a.D + at * A::N;
#pragma unroll
        for (int j = 0; j < A::N; ++j) {
            p[j] = sw[j];
            p[a.D + j] = sb[j];
        }
    }
}

// dw and db from the chunks' sums, in chunk order: 32 columns to a CTA, eight
// threads to a column.
template <typename W>
__global__ void __launch_bounds__(256) norm_grad_params_kernel(const NormGradArgs a) {
    __shared__ float red[8][33];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;   // of dw's columns, then db's
    const int lo = a.S * grp / 8, hi = a.S * (grp + 1) / 8;
    float s = 0.f;
    if (c < 2 * a.D) {
#pragma unroll 8
        for (int k = lo; k < hi; ++k) s += a.part[(int64_t)k * 2 * a.D + c];
    }
    red[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && c < 2 * a.D) {
        for (int k = 1; k < 8; ++k) s += red[k][lane];
        W* out = static_cast<W*>(c < a.D ? a.dw : a.db) + (c < a.D ? c : c - a.D);
        if constexpr (sizeof(W) == 4)
            *out = s;
        else
            *out = __float2bfloat16_rn(s);
    }
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

template <typename T, typename W, int B>
tpmlp_status forward(const NormArgs& a, cudaStream_t s) {
    constexpr int R = B >= 4 ? HELD_WORDS * 4 / B : HELD_WORDS;
    const int64_t accesses = a.D / (B / (int)sizeof(T));
    LaunchScope ls("layernorm", s);
    if (accesses <= 32 * R)
        return launch(layernorm_kernel<T, W, B, 32>, dim3((unsigned)((a.N + 3) / 4)), 128, s, a);
    if (accesses <= 128 * R) return launch(layernorm_kernel<T, W, B, 128>, dim3((unsigned)a.N), 128, s, a);
    if (accesses <= 512 * R) return launch(layernorm_kernel<T, W, B, 512>, dim3((unsigned)a.N), 512, s, a);
    return launch(layernorm_long_kernel<T, W, B>, dim3((unsigned)a.N), WIDEST, s, a);
}

template <typename T, typename W>
tpmlp_status forward_width(const NormArgs& a, cudaStream_t s) {
    auto fits = [&](int bytes) {
        const int n = bytes / (int)sizeof(T);
        const int params = n * (int)sizeof(W) < 16 ? n * (int)sizeof(W) : 16;
        return a.D % n == 0 && access_fits(a.x, a.ldx * sizeof(T), bytes) &&
               access_fits(a.y, a.ldy * sizeof(T), bytes) && access_fits(a.w, 0, params) &&
               access_fits(a.b, 0, params);
    };
    if (fits(16)) return forward<T, W, 16>(a, s);
    if constexpr (sizeof(T) == 4) return forward<T, W, 4>(a, s);
    else return fits(4) ? forward<T, W, 4>(a, s) : forward<T, W, 2>(a, s);
}

// Row chunks of the column sums: enough CTAs to occupy the SMs some eight
// times over, at least four rows each.
int64_t row_chunks(int64_t N, int64_t D) {
    const int64_t blocks = (D + 1023) / 1024;
    int64_t S = 8LL * 152 / blocks;
    if (S > (N + 3) / 4) S = (N + 3) / 4;
    return S < 1 ? 1 : S > 1024 ? 1024 : S;
}

template <typename T, typename W, int B>
tpmlp_status backward(const NormGradArgs& a, cudaStream_t s) {
    LaunchScope ls("layernorm_backward", s);
    const int64_t accesses = a.D / (B / (int)sizeof(T));
    tpmlp_status st = launch(norm_grad_rows_kernel<T, W, B>, dim3((unsigned)a.N), 256, s, a);
    if (st != TPMLP_OK) return st;
    st = launch(norm_grad_apply_kernel<T, W, B>, dim3((unsigned)((accesses + 127) / 128), (unsigned)a.S), 128, s, a);
    if (st != TPMLP_OK || a.part == nullptr) return st;
    return launch(norm_grad_params_kernel<W>, dim3((unsigned)((2 * a.D + 31) / 32)), 256, s, a);
}

template <typename T, typename W>
tpmlp_status backward_width(const NormGradArgs& a, cudaStream_t s) {
    auto fits = [&](int bytes) {
        const int n = bytes / (int)sizeof(T);
        const int params = n * (int)sizeof(W) < 16 ? n * (int)sizeof(W) : 16;
        return a.D % n == 0 && access_fits(a.x, a.ldx * sizeof(T), bytes) &&
               access_fits(a.dy, a.lddy * sizeof(T), bytes) && access_fits(a.dx, a.lddx * sizeof(T), bytes) &&
               (a.dres == nullptr || access_fits(a.dres, a.lddres * sizeof(T), bytes)) &&
               access_fits(a.w, 0, params);
    };
    if (fits(16)) return backward<T, W, 16>(a, s);
    if constexpr (sizeof(T) == 4) return backward<T, W, 4>(a, s);
    else return fits(4) ? backward<T, W, 4>(a, s) : backward<T, W, 2>(a, s);
}

size_t rows_bytes(int64_t N) { return ((size_t)N * sizeof(float4) + 255) & ~(size_t)255; }

}  // namespace

tpmlp_status run_layernorm(int f32, int params_f32, const LayernormArgs& g, cudaStream_t s) {
    if (g.N == 0) return TPMLP_OK;
    const NormArgs a{g.N, g.D, g.x, g.ldx, g.weight, g.bias, g.eps, g.y, g.ldy, g.mean, g.rstd};
    if (f32) return forward_width<float, float>(a, s);
    return params_f32 ? forward_width<__nv_bfloat16, float>(a, s) : forward_width<__nv_bfloat16, __nv_bfloat16>(a, s);
}

size_t layernorm_backward_bytes(int64_t N, int64_t D) {
    return N == 0 ? 0 : rows_bytes(N) + (size_t)row_chunks(N, D) * 2 * (size_t)D * sizeof(float);
}

tpmlp_status run_layernorm_backward(int f32, int params_f32, const LayernormGradArgs& g, void* workspace,
                                    cudaStream_t s) {
    const bool params = g.dweight != nullptr;
    if (g.N == 0) {   // sums over no rows
        const size_t bytes = (size_t)g.D * (params_f32 ? 4 : 2);
        if (params && (cudaMemsetAsync(g.dweight, 0, bytes, s) != cudaSuccess ||
                       cudaMemsetAsync(g.dbias, 0, bytes, s) != cudaSuccess))
            return TPMLP_ERR_CUDA;
        return TPMLP_OK;
    }
    NormGradArgs a{g.N, g.D, g.dy, g.lddy, g.x, g.ldx, g.weight, g.mean, g.rstd, g.dresidual, g.lddres,
                   g.dx, g.lddx, g.dweight, g.dbias, nullptr, nullptr, (int)row_chunks(g.N, g.D)};
    a.rows = static_cast<float4*>(workspace);
    if (params) a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + rows_bytes(g.N));
    if (f32) return backward_width<float, float>(a, s);
    return params_f32 ? backward_width<__nv_bfloat16, float>(a, s)
                      : backward_width<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace tpmlp
