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

#include <atomic>

#include "access.cuh"
#include "ptx.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int HELD_WORDS = 32;   // 32-bit registers of a row that a thread holds
constexpr int WIDEST = 1024;     // threads of the widest row

// Rows in turn: CTAs that stay, of as many groups of nt threads (32 to 512) as a
// row needs at ELEMS elements a thread. A thread keeps its columns' parameters
// in registers, and its elements of the next rows are on their way to places of
// its own in shared memory (no barrier between the copy and its use).
constexpr int STAY = 512;        // threads of such a CTA
constexpr int ELEMS = 16;

__host__ __device__ __forceinline__ int group_threads(int64_t D) {
    int nt = 32;
    while (nt * ELEMS < D) nt *= 2;
    return nt;
}

// Sums over a group of nt threads (whole warps, a power of two of them), in every
// thread of it. red: where the CTA's warps put theirs; not the place that the
// sum before used, so that one barrier is enough.
template <int V, typename Op>
__device__ __forceinline__ void group_reduce(float (&v)[V], int nt, int group, float (*red)[V], Op op) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = op(v[k], __shfl_xor_sync(0xffffffffu, v[k], off));
    if (nt > 32) {
        const int warps = nt / 32, lane = threadIdx.x & 31, warp = (threadIdx.x / 32) & (warps - 1);
        red += group * warps;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < V; ++k) red[warp][k] = v[k];
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(nt) : "memory");
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = red[lane & (warps - 1)][k];
        for (int off = warps / 2; off > 0; off >>= 1)
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

// A row's statistics: x scaled by `scale` (1 but for rows whose squares
// overflow) has mean m + d and reciprocal deviation r.
struct RowStats {
    float scale, m, d, r;
    __device__ __forceinline__ float normal(float x) const { return (x * scale - m - d) * r; }
};

using Red = float (*)[WIDEST / 32][2];   // three places for the warps' numbers

// inv = 1 / D; each(f) calls f for every element of the row that this thread looks after.
template <typename Each>
__device__ __forceinline__ RowStats row_stats(float inv, float eps, int nt, int group, Red red, Each each) {
    RowStats s{1.f, 0.f, 0.f, 0.f};
    float var = 0.f;
    auto take = [&]() {
        float a[2] = {0.f, 0.f};
        each([&](float x) { a[0] += x * s.scale; });
        group_reduce(a, nt, group, red[0], Add());
        s.m = a[0] * inv;
        float c[2] = {0.f, 0.f};
        each([&](float x) {
            const float t = x * s.scale - s.m;
            c[0] += t;
            c[1] = fmaf(t, t, c[1]);
        });
        group_reduce(c, nt, group, red[1], Add());
        var = c[1] * inv;
        s.d = s.m * s.m > var ? c[0] * inv : 0.f;
        var = max_nan(fmaf(-s.d, s.d, var), 0.f);
    };
    take();
    if (!(var < INFINITY)) {   // the same for every thread of the row
        float big[2] = {0.f, 0.f};
        each([&](float x) { big[0] = max_nan(big[0], fabsf(x)); });
        group_reduce(big, nt, group, red[2], Max());
        if (big[0] < INFINITY) {   // finite elements: their squares overflowed
            s.scale = 0x1p-100f;
            take();
        }
    }
    s.r = 1.f / sqrtf(fmaf(eps * s.scale, s.scale, var));
    return s;
}

__device__ __forceinline__ void copy_async(void* dst, const uint4* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async(void* dst, const uint32_t* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async(void* dst, const unsigned short* src) {   // there is none of 2 bytes
    *static_cast<unsigned short*>(dst) = *src;
}

// The rows ahead of a group, one matrix's or several's: access i of matrix q of a row
// in stage k is at word ((k Q + q) R + i) STAY + thread.
template <typename T, int B, int Q, int STAGES>
struct RowRing {
    using A = Access<T, B>;
    using Word = typename A::Word;
    static constexpr int R = ELEMS / A::N;
    static constexpr int BYTES = STAGES * Q * R * STAY * B;
    Word* place;
    int t, nt, accesses;
    __device__ __forceinline__ Word& at(int k, int q, int i) const { return place[((k * Q + q) * R + i) * STAY]; }
    __device__ __forceinline__ bool mine(int i) const { return t + i * nt < accesses; }
    __device__ __forceinline__ void fetch(int k, int q, const void* base, int64_t row, int64_t ld) const {
        const Word* src = reinterpret_cast<const Word*>(static_cast<const T*>(base) + row * ld) + t;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (mine(i)) copy_async(&at(k, q, i), src + i * nt);
    }
    __device__ __forceinline__ void get(int k, int q, int i, float (&v)[A::N]) const { A::unpack(at(k, q, i), v); }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // all but the last STAGES - 1 rows have arrived
    static __device__ __forceinline__ void wait() {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    }
};

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
    __shared__ float red[3][WIDEST / 32][2];
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
    const RowStats s = row_stats(1.f / (float)a.D, a.eps, NT, threadIdx.x / NT, red, [&](auto f) {
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

// Many rows of up to STAY * ELEMS elements.
constexpr int AHEAD = 3;   // stages of the forward's ring

template <typename T, typename W, int B>
__global__ void __launch_bounds__(STAY, 2) layernorm_stay_kernel(const NormArgs a, int nt) {
    using Ring = RowRing<T, B, 1, AHEAD>;
    using A = typename Ring::A;
    using Word = typename Ring::Word;
    constexpr int R = Ring::R;
    extern __shared__ uint4 ring_memory[];
    __shared__ float red[3][WIDEST / 32][2];
    const int groups = STAY / nt, group = threadIdx.x / nt, t = threadIdx.x & (nt - 1);
    const Ring ring{reinterpret_cast<Word*>(ring_memory) + threadIdx.x, t, nt, (int)(a.D / A::N)};
    const int64_t step = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups + group;
    pdl_wait();
    pdl_launch_dependents();
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
        if (first + k * step < a.N) ring.fetch(k, 0, a.x, first + k * step, a.ldx);
        ring.commit();
    }
    float w[R][A::N], b[R][A::N];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int j = 0; j < A::N; ++j) w[i][j] = 1.f, b[i][j] = 0.f;
        if (ring.mine(i)) {
            if (a.w) load_params<W, A::N>(static_cast<const W*>(a.w) + (t + i * nt) * A::N, w[i]);
            if (a.b) load_params<W, A::N>(static_cast<const W*>(a.b) + (t + i * nt) * A::N, b[i]);
        }
    }
    const float inv = 1.f / (float)a.D;
    int k = 0;
    for (int64_t row = first; row < a.N; row += step) {
        ring.wait();
        const RowStats s = row_stats(inv, a.eps, nt, group, red, [&](auto f) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (ring.mine(i)) {
                    float v[A::N];
                    ring.get(k, 0, i, v);
#pragma unroll
                    for (int j = 0; j < A::N; ++j) f(v[j]);
                }
        });
        Word* y = reinterpret_cast<Word*>(static_cast<T*>(a.y) + row * a.ldy) + t;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (ring.mine(i)) {
                float v[A::N];
                ring.get(k, 0, i, v);
#pragma unroll
                for (int j = 0; j < A::N; ++j) v[j] = fmaf(s.normal(v[j]), w[i][j], b[i][j]);
                y[i * nt] = A::pack(v);
            }
        if (t == 0) {
            if (a.mean) a.mean[row] = (s.m + s.d) / s.scale;
            if (a.rstd) a.rstd[row] = s.r * s.scale;
        }
        if (row + AHEAD * step < a.N) ring.fetch(k, 0, a.x, row + AHEAD * step, a.ldx);
        ring.commit();
        k = k == AHEAD - 1 ? 0 : k + 1;
    }
}

// A row of any length, read three times (from L2 but for the first).
template <typename T, typename W, int B>
__global__ void __launch_bounds__(WIDEST) layernorm_long_kernel(const NormArgs a) {
    using A = Access<T, B>;
    using Word = typename A::Word;
    __shared__ float red[3][WIDEST / 32][2];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const int64_t accesses = a.D / A::N;
    const Word* x = reinterpret_cast<const Word*>(static_cast<const T*>(a.x) + row * a.ldx);
    Word* y = reinterpret_cast<Word*>(static_cast<T*>(a.y) + row * a.ldy);
    const RowStats s = row_stats(1.f / (float)a.D, a.eps, WIDEST, 0, red, [&](auto f) {
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

template <typename T> constexpr int GRAD_AHEAD = sizeof(T) == 2 ? 4 : 2;   // stages: 192 KB

// All of it in one reading, for rows of up to STAY * ELEMS elements: a thread
// keeps its columns' sums of dy h and dy over the rows of its group; a CTA's
// sums go to part[blockIdx.x] (with one CTA to dw and db).
template <typename T, typename W, int B>
__global__ void __launch_bounds__(STAY, 1) norm_grad_kernel(const NormGradArgs a, int nt) {
    using Ring = RowRing<T, B, 3, GRAD_AHEAD<T>>;
    using A = typename Ring::A;
    using Word = typename Ring::Word;
    constexpr int R = Ring::R;
    extern __shared__ uint4 ring_memory[];
    __shared__ float red[2][STAY / 32][3];
    const int groups = STAY / nt, group = threadIdx.x / nt, t = threadIdx.x & (nt - 1);
    const Ring ring{reinterpret_cast<Word*>(ring_memory) + threadIdx.x, t, nt, (int)(a.D / A::N)};
    const int64_t step = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups + group;
    pdl_wait();
    pdl_launch_dependents();
    auto fetch = [&](int k, int64_t row) {
        if (row < a.N) {
            ring.fetch(k, 0, a.x, row, a.ldx);
            ring.fetch(k, 1, a.dy, row, a.lddy);
            if (a.dres) ring.fetch(k, 2, a.dres, row, a.lddres);
        }
        ring.commit();
    };
#pragma unroll
    for (int k = 0; k < GRAD_AHEAD<T>; ++k) fetch(k, first + k * step);
    float w[R][A::N], sw[R][A::N], sb[R][A::N];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int j = 0; j < A::N; ++j) w[i][j] = 1.f, sw[i][j] = sb[i][j] = 0.f;
        if (a.w && ring.mine(i)) load_params<W, A::N>(static_cast<const W*>(a.w) + (t + i * nt) * A::N, w[i]);
    }
    const float inv = 1.f / (float)a.D;
    float m = 0.f, r = 0.f;
    if (first < a.N) m = a.mean[first], r = a.rstd[first];
    int k = 0, turn = 0;
    for (int64_t row = first; row < a.N; row += step, turn ^= 1) {
        const float cm = m, cr = r;
        if (row + step < a.N) m = a.mean[row + step], r = a.rstd[row + step];
        ring.wait();
        float s[3] = {0.f, 0.f, 0.f};   // u, u h, h
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (ring.mine(i)) {
                float v[A::N], y[A::N];
                ring.get(k, 0, i, v);
                ring.get(k, 1, i, y);
#pragma unroll
                for (int j = 0; j < A::N; ++j) {
                    const float h = (v[j] - cm) * cr, u = y[j] * w[i][j];
                    s[0] += u;
                    s[1] = fmaf(u, h, s[1]);
                    s[2] += h;
                }
            }
        group_reduce(s, nt, group, red[turn], Add());
        const float d = fabsf(cm * cr) > 1.f ? s[2] * inv : 0.f;
        const float c1 = s[0] * inv, c2 = fmaf(-d, s[0], s[1]) * inv;
        Word* out = reinterpret_cast<Word*>(static_cast<T*>(a.dx) + row * a.lddx) + t;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (ring.mine(i)) {
                float v[A::N], y[A::N], z[A::N];
                ring.get(k, 0, i, v);
                ring.get(k, 1, i, y);
                if (a.dres) ring.get(k, 2, i, z);
#pragma unroll
                for (int j = 0; j < A::N; ++j) {
                    const float h = fmaf(v[j] - cm, cr, -d);
                    sw[i][j] = fmaf(y[j], h, sw[i][j]);
                    sb[i][j] += y[j];
                    v[j] = cr * fmaf(-h, c2, fmaf(y[j], w[i][j], -c1));
                    if (a.dres) v[j] += z[j];
                }
                out[i * nt] = A::pack(v);
            }
        fetch(k, row + GRAD_AHEAD<T> * step);
        k = k == GRAD_AHEAD<T> - 1 ? 0 : k + 1;
    }
    if (a.dw == nullptr) return;
    if (groups > 1) {   // the groups' sums in their order, through the ring's memory
        float* sums = reinterpret_cast<float*>(ring_memory);
        static_assert(2 * STAY / 2 * ELEMS * sizeof(float) <= Ring::BYTES, "room for two sums a column");
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (int q = 0; q < groups; ++q) {
            __syncthreads();
            if (group == q)
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (ring.mine(i))
#pragma unroll
                        for (int j = 0; j < A::N; ++j) {
                            float* at = sums + 2 * ((t + i * nt) * A::N + j);
                            if (q > 0) {
                                sw[i][j] += at[0];
                                sb[i][j] += at[1];
                            }
                            at[0] = sw[i][j];
                            at[1] = sb[i][j];
                        }
        }
        if (group != groups - 1) return;   // the last group has them all
    }
    float* p = a.part + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (ring.mine(i))
#pragma unroll
            for (int j = 0; j < A::N; ++j) {
                const int c = (t + i * nt) * A::N + j;
                if (gridDim.x > 1) {
                    p[c] = sw[i][j];
                    p[a.D + c] = sb[i][j];
                } else if constexpr (sizeof(W) == 4) {
                    static_cast<W*>(a.dw)[c] = sw[i][j];
                    static_cast<W*>(a.db)[c] = sb[i][j];
                } else {
                    static_cast<W*>(a.dw)[c] = __float2bfloat16_rn(sw[i][j]);
                    static_cast<W*>(a.db)[c] = __float2bfloat16_rn(sb[i][j]);
                }
            }
}

// Longer rows are read twice.
// Sums over a row, one CTA each.
template <typename T, typename W, int B>
__global__ void __launch_bounds__(256) norm_grad_rows_kernel(const NormGradArgs a) {
    using A = Access<T, B>;
    using Word = typename A::Word;
    __shared__ float red[256 / 32][3];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const int64_t accesses = a.D / A::N;
    const Word* x = reinterpret_cast<const Word*>(static_cast<const T*>(a.x) + row * a.ldx);
    const Word* dy = reinterpret_cast<const Word*>(static_cast<const T*>(a.dy) + row * a.lddy);
    const float m = a.mean[row], r = a.rstd[row];
    float s[3] = {0.f, 0.f, 0.f};   // u, u h, h
#pragma unroll 2
    for (int64_t at = threadIdx.x; at < accesses; at += 256) {
        float v[A::N], g[A::N], w[A::N];
        A::unpack(x[at], v);
        A::unpack(dy[at], g);
        if (a.w) load_params<W, A::N>(static_cast<const W*>(a.w) + at * A::N, w);
#pragma unroll
        for (int j = 0; j < A::N; ++j) {
            const float h = (v[j] - m) * r, u = a.w ? g[j] * w[j] : g[j];
            s[0] += u;
            s[1] = fmaf(u, h, s[1]);
            s[2] += h;
        }
    }
    const float inv = 1.f / (float)a.D;
    group_reduce(s, 256, 0, red, Add());
    const float d = fabsf(m * r) > 1.f ? s[2] * inv : 0.f;
    if (threadIdx.x == 0) a.rows[row] = make_float4(s[0] * inv, fmaf(-d, s[0], s[1]) * inv, d, 0.f);
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
tpmlp_status launch_smem(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return TPMLP_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

template <typename... P, typename... A>
tpmlp_status launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
    return launch_smem(kernel, grid, threads, 0, s, args...);
}

// The kernel may use `bytes` of dynamic shared memory: asked for once a device
// (`asked`: one bit each; devices beyond ask every time).
template <typename K>
bool allow_smem(K kernel, int bytes, std::atomic<uint64_t>& asked) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (asked.load() & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    asked.fetch_or(bit);
    return true;
}

template <typename T, typename W, int B>
tpmlp_status forward(const NormArgs& a, cudaStream_t s) {
    constexpr int R = B >= 4 ? HELD_WORDS * 4 / B : HELD_WORDS;
    const int64_t accesses = a.D / (B / (int)sizeof(T));
    LaunchScope ls("layernorm", s);
    if (a.D <= STAY * ELEMS) {
        const int nt = group_threads(a.D);
        const int64_t turns = (a.N + STAY / nt - 1) / (STAY / nt), most = 2LL * device_sm_count();
        if (turns > most) {
            constexpr int BYTES = RowRing<T, B, 1, AHEAD>::BYTES;
            static std::atomic<uint64_t> asked{0};
            if (!allow_smem(layernorm_stay_kernel<T, W, B>, BYTES, asked)) return TPMLP_ERR_CUDA;
            return launch_smem(layernorm_stay_kernel<T, W, B>, dim3((unsigned)most), STAY, BYTES, s, a, nt);
        }
    }
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

constexpr int MOST_CTAS = 152;   // that stay, of the backward: one an SM

template <typename T, typename W, int B>
tpmlp_status backward(NormGradArgs a, cudaStream_t s) {
    LaunchScope ls("layernorm_backward", s);
    if (a.D <= STAY * ELEMS) {
        const int nt = group_threads(a.D);
        const int64_t turns = (a.N + STAY / nt - 1) / (STAY / nt);
        a.S = (int)(turns < MOST_CTAS ? turns : MOST_CTAS);
        constexpr int BYTES = RowRing<T, B, 3, GRAD_AHEAD<T>>::BYTES;
        static std::atomic<uint64_t> asked{0};
        if (!allow_smem(norm_grad_kernel<T, W, B>, BYTES, asked)) return TPMLP_ERR_CUDA;
        const tpmlp_status st =
            launch_smem(norm_grad_kernel<T, W, B>, dim3((unsigned)a.S), STAY, BYTES, s, a, nt);
        if (st != TPMLP_OK || a.part == nullptr || a.S == 1) return st;
        return launch(norm_grad_params_kernel<W>, dim3((unsigned)((2 * a.D + 31) / 32)), 256, s, a);
    }
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
    if (N == 0) return 0;
    const int64_t S = D <= STAY * ELEMS ? MOST_CTAS : row_chunks(N, D);
    return rows_bytes(N) + (size_t)S * 2 * (size_t)D * sizeof(float);
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
