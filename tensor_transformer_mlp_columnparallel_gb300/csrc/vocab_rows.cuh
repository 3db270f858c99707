// Rows over a vocabulary: how a row is split over a cluster's CTAs and threads,
// its 16-byte vectors, the running maximum and sum of its softmax.
#pragma once
#include <cuda_bf16.h>

#include <cmath>

#include "act.cuh"
#include "f32x2.cuh"
#include "ptx.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int ROW_THREADS = 256;
constexpr int VPT = 8;                        // 16-byte vectors a thread holds
constexpr int MAX_SPLIT = 8;                  // CTAs of a row (the portable cluster size)
constexpr float kLowest = -3.402823466e38f;   // FLT_MAX's negative
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return bf2f(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A 16-byte vector of logits: its pairs as fp32, its largest element, how many
// elements beat a given one.
template <typename T> struct Vec;

template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8, PAIRS = 4;
    static constexpr uint32_t MASKED = 0xff80ff80u;   // a pair of -inf
    static __device__ __forceinline__ float lowest() { return __uint_as_float(0xff7f0000u); }
    using Wide = __nv_bfloat162;                       // packed running maximum or count
    static __device__ __forceinline__ uint32_t word(const uint4& x, int k) {
        return k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w;
    }
    static __device__ __forceinline__ Wide as2(uint32_t w) { return *reinterpret_cast<Wide*>(&w); }
    static __device__ __forceinline__ F2 pair(const uint4& x, int k) {
        const uint32_t w = word(x, k);
        return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    // pairs no lower than the lowest finite value, so that e (z - m) is 0 for masked tokens
    static __device__ __forceinline__ F2 pair_floor(const uint4& x, int k) {
        const Wide m = __hmax2_nan(as2(word(x, k)), as2(0xff7fff7fu));
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
        return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ float elem(const uint4& x, int j) {
        const uint32_t w = word(x, j >> 1);
        return __uint_as_float((j & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    template <int R> static __device__ __forceinline__ float largest(const uint4 (&x)[R]) {
        Wide m = __hmax2_nan(__hmax2_nan(as2(x[0].x), as2(x[0].y)), __hmax2_nan(as2(x[0].z), as2(x[0].w)));
#pragma unroll
        for (int r = 1; r < R; ++r)
            m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(as2(x[r].x), as2(x[r].y)),
                                           __hmax2_nan(as2(x[r].z), as2(x[r].w))));
        return max_nan(__low2float(m), __high2float(m));
    }
    // packed counts: whole numbers up to 256 are exact in bf16
    struct Count {
        Wide c;
        __device__ __forceinline__ Count() : c(__float2bfloat162_rn(0.f)) {}
        __device__ __forceinline__ void gt(const uint4& x, Wide t) {
#pragma unroll
            for (int k = 0; k < 4; ++k) c = __hadd2(c, __hgt2(as2(word(x, k)), t));
        }
        __device__ __forceinline__ void ge(const uint4& x, Wide t) {
#pragma unroll
            for (int k = 0; k < 4; ++k) c = __hadd2(c, __hge2(as2(word(x, k)), t));
        }
        __device__ __forceinline__ int total() const { return (int)(__low2float(c) + __high2float(c)); }
    };
    static __device__ __forceinline__ Wide wide(float z) { return __float2bfloat162_rn(z); }
    static __device__ __forceinline__ float narrow(Wide w) { return __low2float(w); }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
        return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                          pack_bf16x2(v[6], v[7]));
    }
    static __device__ __forceinline__ void set(uint4& x, int j, __nv_bfloat16 v) {
        reinterpret_cast<__nv_bfloat16*>(&x)[j] = v;
    }
};

template <> struct Vec<float> {
    static constexpr int N = 4, PAIRS = 2;
    static constexpr uint32_t MASKED = 0xff800000u;
    static __device__ __forceinline__ float lowest() { return kLowest; }
    using Wide = float;
    static __device__ __forceinline__ F2 pair(const uint4& x, int k) {
        return k == 0 ? f2(__uint_as_float(x.x), __uint_as_float(x.y))
                      : f2(__uint_as_float(x.z), __uint_as_float(x.w));
    }
    static __device__ __forceinline__ F2 pair_floor(const uint4& x, int k) {
        return k == 0 ? f2(max_nan(__uint_as_float(x.x), kLowest), max_nan(__uint_as_float(x.y), kLowest))
                      : f2(max_nan(__uint_as_float(x.z), kLowest), max_nan(__uint_as_float(x.w), kLowest));
    }
    static __device__ __forceinline__ float elem(const uint4& x, int j) {
        return __uint_as_float(j == 0 ? x.x : j == 1 ? x.y : j == 2 ? x.z : x.w);
    }
    template <int R> static __device__ __forceinline__ float largest(const uint4 (&x)[R]) {
        float m = -INFINITY;
#pragma unroll
        for (int r = 0; r < R; ++r)
            m = max_nan(m, max_nan(max_nan(elem(x[r], 0), elem(x[r], 1)), max_nan(elem(x[r], 2), elem(x[r], 3))));
        return m;
    }
    struct Count {   // counts of one chunk as fp32 pairs
        F2 c;
        __device__ __forceinline__ Count() : c(f2(0.f, 0.f)) {}
        __device__ __forceinline__ void gt(const uint4& x, float t) {
#pragma unroll
            for (int j = 0; j < 4; j += 2)
                c = add2(c, f2(elem(x, j) > t ? 1.f : 0.f, elem(x, j + 1) > t ? 1.f : 0.f));
        }
        __device__ __forceinline__ void ge(const uint4& x, float t) {
#pragma unroll
            for (int j = 0; j < 4; j += 2)
                c = add2(c, f2(elem(x, j) >= t ? 1.f : 0.f, elem(x, j + 1) >= t ? 1.f : 0.f));
        }
        __device__ __forceinline__ int total() const {
            float a, b;
            split2(c, a, b);
            return (int)(a + b);
        }
    };
    static __device__ __forceinline__ Wide wide(float z) { return z; }
    static __device__ __forceinline__ float narrow(Wide w) { return w; }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
    static __device__ __forceinline__ void set(uint4& x, int j, float v) {
        reinterpret_cast<float*>(&x)[j] = v;
    }
};

// A row in 16-byte vectors. Vector i holds elements head + i N ... + N - 1, for
// 0 <= i < full; the elements before the first 16-byte boundary are vector -1,
// those after the last whole vector are vector `full` (the row's edges), with
// -inf for what lies outside the row. The row's CTA `rank` owns the whole
// vectors [lo, hi), elements [e_lo, e_hi): the first CTA with the front
// edge, the last with the back edge.
template <typename T, int NT>
struct Row {
    using V4 = Vec<T>;
    static constexpr int CHUNK = NT * VPT;   // vectors the CTA's registers hold
    const T* z;
    int head, full, len;
    int lo, hi;
    int e_lo, e_hi;
    __device__ __forceinline__ Row(const void* base, int64_t row, int64_t ld, int64_t V, int rank, int log_split) {
        z = static_cast<const T*>(base) + row * ld;
        len = (int)V;
        const int off = (int)((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / (int)sizeof(T);
        head = off < len ? off : len;
        full = (len - head) / V4::N;
        lo = (int)(((int64_t)full * rank) >> log_split);
        hi = (int)(((int64_t)full * (rank + 1)) >> log_split);
        e_lo = rank == 0 ? 0 : start(lo);
        e_hi = rank == (1 << log_split) - 1 ? len : start(hi);
    }
    __device__ __forceinline__ int start(int i) const { return head + i * V4::N; }
    __device__ __forceinline__ int vector_of(int e) const { return (e - head + V4::N) / V4::N - 1; }
    __device__ __forceinline__ bool mine(int e) const { return e >= e_lo && e < e_hi; }
    __device__ __forceinline__ bool edges() const { return e_lo < start(lo) || e_hi > start(hi); }
    // the edge that this thread looks after (full + 1: none)
    __device__ __forceinline__ int edge() const {
        if (threadIdx.x == 0 && e_lo < start(lo)) return -1;
        if (threadIdx.x == 1 && e_hi > start(hi)) return full;
        return full + 1;
    }
    __device__ __forceinline__ uint4 load_edge(int i) const {
        uint4 x = make_uint4(V4::MASKED, V4::MASKED, V4::MASKED, V4::MASKED);
        if (i > full) return x;
        const int e0 = start(i);
#pragma unroll
        for (int j = 0; j < V4::N; ++j)
            if (e0 + j >= 0 && e0 + j < len) V4::set(x, j, z[e0 + j]);
        return x;
    }
    __device__ __forceinline__ const uint4* vectors() const { return reinterpret_cast<const uint4*>(z + head); }
    __device__ __forceinline__ uint4 load(int i) const { return __ldcs(vectors() + i); }
    // this thread's vectors of the chunk at `base`: base + r NT + thread
    __device__ __forceinline__ void load_chunk(int base, uint4 (&x)[VPT]) const {
        const uint4* p = vectors() + base + threadIdx.x;
#pragma unroll
        for (int r = 0; r < VPT; ++r) x[r] = __ldcs(p + r * NT);
    }
    // the same for the slice's last chunk, -inf beyond it
    __device__ __forceinline__ void load_rest(int base, uint4 (&x)[VPT]) const {
        const uint4* p = vectors() + base + threadIdx.x;
        const int left = hi - base - (int)threadIdx.x;
#pragma unroll
        for (int r = 0; r < VPT; ++r) {
            x[r] = make_uint4(V4::MASKED, V4::MASKED, V4::MASKED, V4::MASKED);
            if (r * NT < left) x[r] = __ldcs(p + r * NT);
        }
    }
    // where the last chunk starts: it has 1 to CHUNK vectors (none in an empty slice)
    __device__ __forceinline__ int rest() const {
        const int n = hi - lo;
        return n > 0 ? lo + (n - 1) / CHUNK * CHUNK : lo;
    }
};

// sum of e = 2^((z - ref) c) and sum of e (z - ref)
struct Soft {
    float ref, s, e;
};

// The state relative to another reference, not below its own.
__device__ __forceinline__ void rebase(Soft& a, float ref, float c) {
    const float d = a.ref - ref;
    const float f = ex2(d * c);   // NaN with ref
    a.e = f == 0.f ? 0.f : f * fmaf(a.s, d, a.e);   // d may be -inf with f = 0
    a.s *= f;
    a.ref = ref;
}

// One chunk in registers added to a thread's state; ENT: with the entropy's sum.
template <typename T, bool ENT, int R>
__device__ __forceinline__ void soft_chunk(Soft& st, const uint4 (&x)[R], float largest, float c) {
    const float ref = max_nan(st.ref, largest);
    rebase(st, ref, c);
    const F2 c2 = f2(c, c), r2 = f2(-ref, -ref);
    F2 s0 = f2(0.f, 0.f), s1 = s0, e0 = s0, e1 = s0;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < Vec<T>::PAIRS; ++k) {
            const F2 z = ENT ? Vec<T>::pair_floor(x[r], k) : Vec<T>::pair(x[r], k);
            const F2 t = add2(z, r2);
            float a, b;
            split2(mul2(t, c2), a, b);
            const F2 p = f2(ex2(a), ex2(b));
            if (k & 1) {
                s1 = add2(s1, p);
                if (ENT) e1 = fma2(p, t, e1);
            } else {
                s0 = add2(s0, p);
                if (ENT) e0 = fma2(p, t, e0);
            }
        }
    float a, b;
    split2(add2(s0, s1), a, b);
    st.s += a + b;
    if (ENT) {
        split2(add2(e0, e1), a, b);
        st.e += a + b;
    }
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// (reference, sum) of every warp of the row's CTAs, in one place of each CTA
struct __align__(8) WarpSoft {
    float ref, s;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// CTAs per row, as a power of two. Few rows: enough CTAs to occupy the SMs
// four times over, while a slice still has a vector for every thread. A
// slice should also be no longer than `hold` vectors (0: any length).
inline int row_split(int64_t N, int64_t row_bytes, int threads, int64_t hold) {
    const int64_t want = 4LL * device_sm_count();
    if (N * MAX_SPLIT > 0x7fffffffLL) return 0;
    int l = 0;
    while ((1 << l) < MAX_SPLIT && (N << l) < want && (row_bytes >> (l + 1)) >= threads * 16) ++l;
    while ((1 << l) < MAX_SPLIT && hold > 0 && (row_bytes >> l) > hold * 16) ++l;
    return l;
}

template <typename... P, typename... A>
tpmlp_status launch_rows(void (*kernel)(P...), int threads, size_t smem, int64_t N, int log_split,
                         cudaStream_t s, A... args) {
    const int split = 1 << log_split;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)(N * split));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    // the kernel waits for what runs before it, and lets what runs after it
    // be launched while its last rows are on their way
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (split > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)split;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return TPMLP_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

}  // namespace
}  // namespace tpmlp
