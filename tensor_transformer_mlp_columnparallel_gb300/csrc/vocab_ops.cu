// Token log probabilities and distillation over vocabulary rows.
//
// vocab_logprobs: per row m = max z, S = sum exp(z - m), lse = m + ln S, the
//   given token's z_t - lse and rank, the entropy ln S - (sum e (z - m)) / S
//   with e = exp(z - m), and the K largest logits.
// vocab_distill: q = softmax of the teacher's slots over tau, p = softmax(z / tau),
//   loss = tau^2 sum q (ln q - ln p), dz = w (p - q) with w = g tau.
//
// Both read a row once. A row belongs to a cluster of 1, 2, 4 or 8 CTAs, each
// taking a contiguous slice in 16-byte vectors; a thread keeps VPT vectors in
// registers at a time (128 KB an SM in flight), so the maximum of what it
// holds is known before the first exponential. Exponentials are 2^((z - m) c)
// with c = log2(e) / tau and m the running maximum, so the largest token's is
// exactly 1 and a certain token's log probability exactly 0. m starts at the
// lowest finite number: no finite logit is below it, and a thread that has
// seen only masked tokens (-inf) meets no inf - inf.
//
// HBM bounds both on many rows (what they read and write, over the time, on
// GB300, where a copy runs at 6.8 TB/s):
//   log probabilities, 8192 x 128000 bf16: 295 us without a top list (7.1
//   TB/s), 315 with 5 tokens, 359 with 20 (5.8 TB/s: the list's own work);
//   2048 rows with 5: 96 us (5.5 TB/s: a start and a tail);
//   distillation with its gradient, 4096 x 128000 bf16: 350 us (6.0 TB/s).
// Few rows are a launch and a cluster's two exchanges: 5 us for one of 32000 fp32
// logits, 13 for 48 of 128000 bf16 with 20 tokens (from a captured graph).
#include <cuda_bf16.h>

#include <cmath>

#include "act.cuh"
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

// Two fp32 values in a 64-bit register pair: one issue slot for two results.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split2(F2 x, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
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

// What the CTAs of a row tell one another.
struct __align__(16) Part {
    Soft soft;
    int before;   // entries in front of the target
};

__device__ __forceinline__ Part combine(const Part* parts, int n, float c) {
    float m = parts[0].soft.ref;
    for (int i = 1; i < n; ++i) m = max_nan(m, parts[i].soft.ref);
    Part r{Soft{m, 0.f, 0.f}, 0};
    for (int i = 0; i < n; ++i) {
        Soft o = parts[i].soft;
        rebase(o, m, c);
        r.soft.s += o.s;
        r.soft.e += o.e;
        r.before += parts[i].before;
    }
    return r;
}

// The block's state from its threads' (fixed order), in every thread.
template <int WARPS>
__device__ __forceinline__ Part block_part(Soft st, int before, Part* red, float c) {
    float m = st.ref;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    rebase(st, m, c);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        st.s += __shfl_xor_sync(0xffffffffu, st.s, off);
        st.e += __shfl_xor_sync(0xffffffffu, st.e, off);
        before += __shfl_xor_sync(0xffffffffu, before, off);
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = Part{st, before};
    __syncthreads();
    return combine(red, WARPS, c);
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// `part` into slot `slot` of the array at `dst` in CTA `to` of the cluster
__device__ __forceinline__ void send_part(Part* dst, int slot, uint32_t to, const Part& part) {
    const uint32_t a = mapa_shared(smem_u32(dst + slot), to);
    st_cluster_v4(a, part.soft.ref, part.soft.s, part.soft.e, __int_as_float(part.before));
}

// Whole-block reduction in a fixed order; every thread gets the result.
template <typename T, typename Op>
__device__ T block_reduce(T v, Op op, T* red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, off));
    __syncthreads();   // red may hold an earlier reduction's values
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    T r = red[0];
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) r = op(r, red[w]);
    __syncthreads();
    return r;
}

struct Sum {
    template <typename T> __device__ T operator()(T a, T b) const { return a + b; }
};
struct MaxU64 {
    __device__ unsigned long long operator()(unsigned long long a, unsigned long long b) const {
        return a > b ? a : b;
    }
};

// A row's distribution: ln p = (z - ref) / tau - ln s; nothing: no finite logit,
// every ln p = -inf.
struct Dist {
    float ref, s, ln_s, c, inv_tau;
    bool nothing;
    __device__ __forceinline__ float exponent(float z) const { return (z - ref) * c; }
    __device__ __forceinline__ float ln_p(float z) const {
        return nothing ? -INFINITY : fmaf(z - ref, inv_tau, -ln_s);
    }
    __device__ __forceinline__ float lse() const {   // of z / tau
        return nothing ? -INFINITY : fmaf(ref, inv_tau, ln_s);
    }
};

__device__ __forceinline__ Dist distribution(const Soft& t, float c, float inv_tau) {
    Dist d;
    d.ref = t.ref;
    d.s = t.s;
    d.ln_s = logf(t.s);
    d.c = c;
    d.inv_tau = inv_tau;
    d.nothing = t.s == 0.f;
    return d;
}

// Entries with a probability in a row whose maximum is the lowest finite value
// or -inf: they all hold that value.
template <typename T, int NT>
__device__ __noinline__ float count_finite(const T* z, int64_t V, float* red) {
    float n = 0.f;
    for (int64_t i = threadIdx.x; i < V; i += NT) n += to_f32(z[i]) != -INFINITY ? 1.f : 0.f;
    return block_reduce(n, Sum(), red);
}

// sum e (z - ref) over a whole row a plain element at a time, for a row whose
// (z - ref) overflows at a masked token (a maximum near the type's largest value)
template <typename T, int NT>
__device__ __noinline__ float slow_esum(const T* z, int64_t V, const Dist& d, float* red) {
    float es = 0.f;
    for (int64_t i = threadIdx.x; i < V; i += NT) {
        const float x = to_f32(z[i]), p = ex2(d.exponent(x));
        es += p == 0.f ? 0.f : p * (x - d.ref);
    }
    return block_reduce(es, Sum(), red);
}

// ------------------------------------------------------- top tokens ------

// An order of all floats (NaN with its sign bit clear on top); -0 = +0.
__device__ __forceinline__ uint32_t order32(float z) {
    const uint32_t b = __float_as_uint(z + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
// One number per entry that falls with the logit, then rises with the index:
// the list's order.
__device__ __forceinline__ unsigned long long order_key(uint32_t o, uint32_t v) {
    return ((unsigned long long)o << 32) | (0xffffffffu - v);
}

template <int NT>
struct TopShared {
    static constexpr int MAX_CAND = 4 * NT;
    // lists of several CTAs: rows that are split have CTAs of ROW_THREADS
    static constexpr int ALL = NT == ROW_THREADS ? MAX_SPLIT * TPMLP_MAX_TOP : 1;
    unsigned long long cand[MAX_CAND];
    unsigned long long list[TPMLP_MAX_TOP];                  // this CTA's first K, in order
    unsigned long long all[ALL];       // the leader's copy of every CTA's list
    unsigned long long red[NT / 32];
    uint32_t thr[NT / 32];
    uint32_t max_of[NT];    // maxima that reach the first bound
    int chunk_of[NT];       // (chunk, thread) whose vectors are looked at
    int whole_of[NT];       // threads all of whose vectors are
    uint32_t bound;
    int n_max, n_chunk, n_whole, n_cand;
};

// The elements of vector i that are in the row and at least `thr` (strictly
// above with `above`) join the candidates; beyond MAX_CAND they are only counted.
template <typename T, int NT>
__device__ __forceinline__ void offer(const Row<T, NT>& row, int i, const uint4& x, uint32_t thr, bool above,
                                      TopShared<NT>& sh) {
    const int e0 = row.start(i);
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) {
        const uint32_t o = order32(Vec<T>::elem(x, j));
        if ((above ? o > thr : o >= thr) && e0 + j >= 0 && e0 + j < row.len) {
            const int at = atomicAdd(&sh.n_cand, 1);
            if (at < TopShared<NT>::MAX_CAND) sh.cand[at] = order_key(o, (uint32_t)(e0 + j));
        }
    }
}

// The slice's first K entries into sh.list (0: fewer than K entries).
//
// What a thread remembers of its part of the slice.
struct Peaks {
    float best;     // the largest in one of its chunks, the one at `base`
    float other;    // the largest of all else, the row's edges among it; NaN where a NaN was seen
    int base;
};

// The K-th largest of the threads' NT (at least K) maxima is reached by K
// different entries, so only entries at or above it can be in the list, and
// they sit with the threads whose maximum reaches it: K of NT unless maxima
// are equal. Of their vectors those of the chunk with the maximum are read
// again, from L2 as a rule and spread over all threads, and a thread's others
// (K / NT of the slice in all, from DRAM as a rule) only if one of them reaches
// the bound too: at 8192 x 128000 bf16 logits and K = 20 the list is 18% of the
// kernel. The K-th largest maximum comes in two steps: with g = ceil(K /
// warps), the least of the warps' g-th largest maxima leaves a few dozen, and
// those are ranked by counting.
// Where more than MAX_CAND entries reach the bound (a mask that leaves fewer
// than K tokens, rows of equal values), the entries above it are taken alone
// and equal ones follow by index; where even those are too many, K rounds
// over the slice.
template <typename T, int NT>
__device__ void slice_top(const Row<T, NT>& row, int K, const Peaks& peaks, TopShared<NT>& sh) {
    constexpr int MAX_CAND = TopShared<NT>::MAX_CAND;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t mine = order32(max_nan(peaks.best, peaks.other));
    uint32_t left = mine, g_th = 0;
    for (int g = 0; g < (K + NT / 32 - 1) / (NT / 32); ++g) {
        g_th = __reduce_max_sync(0xffffffffu, left);
        const uint32_t who = __ballot_sync(0xffffffffu, left == g_th);
        if (lane == __ffs(who) - 1) left = 0u;
    }
    if (lane == 0) sh.thr[warp] = g_th;
    if (threadIdx.x == 0) sh.n_max = sh.n_chunk = sh.n_whole = sh.n_cand = 0;
    for (int k = threadIdx.x; k < K; k += NT) sh.list[k] = 0ull;
    __syncthreads();
    uint32_t thr = sh.thr[0];
    for (int w = 1; w < NT / 32; ++w) thr = min(thr, sh.thr[w]);
    if (mine >= thr) {
        const int at = atomicAdd(&sh.n_max, 1);
        sh.max_of[at] = mine;
    }
    __syncthreads();
    if ((int)threadIdx.x < sh.n_max) {
        const uint32_t me = sh.max_of[threadIdx.x];
        int above = 0, reach = 0;
        for (int j = 0; j < sh.n_max; ++j) {
            above += sh.max_of[j] > me;
            reach += sh.max_of[j] >= me;
        }
        if (above < K && reach >= K) sh.bound = me;   // the K-th largest: one value
    }
    __syncthreads();
    thr = sh.bound;
    const int n = row.hi - row.lo;
    const int per = (n + NT - 1) / NT;   // vectors of a thread
    if (mine >= thr && row.edge() <= row.full) offer(row, row.edge(), row.load_edge(row.edge()), thr, false, sh);
    if (mine >= thr) {
        if (order32(peaks.other) >= thr)
            sh.whole_of[atomicAdd(&sh.n_whole, 1)] = (int)threadIdx.x;
        else if (order32(peaks.best) >= thr)
            sh.chunk_of[atomicAdd(&sh.n_chunk, 1)] = peaks.base + (int)threadIdx.x;
    }
    __syncthreads();
    for (int a = threadIdx.x; a < sh.n_chunk * VPT; a += NT) {
        const int i = sh.chunk_of[a / VPT] + (a % VPT) * NT;
        if (i < row.hi) offer(row, i, row.load(i), thr, false, sh);
    }
    for (int a = threadIdx.x; a < sh.n_whole * per; a += NT) {
        const int i = row.lo + (a % per) * NT + sh.whole_of[a / per];
        if (i < row.hi) offer(row, i, row.load(i), thr, false, sh);
    }
    __syncthreads();
    int count = sh.n_cand;
    if (count > MAX_CAND) {
        __syncthreads();
        if (threadIdx.x == 0) sh.n_cand = 0;
        __syncthreads();
        if (row.edge() <= row.full) offer(row, row.edge(), row.load_edge(row.edge()), thr, true, sh);
        for (int i = row.lo + (int)threadIdx.x; i < row.hi; i += NT)
            offer(row, i, row.load(i), thr, true, sh);
        __syncthreads();
        count = sh.n_cand;
        if (count <= MAX_CAND - K) {
            // entries equal to the bound, in index order, until there are K
            for (int e = row.e_lo; e < row.e_hi && count < K; e += NT) {
                const int at = e + (int)threadIdx.x;
                const bool hit = at < row.e_hi && order32(to_f32(row.z[at])) == thr;
                const uint32_t b = __ballot_sync(0xffffffffu, hit);
                if (lane == 0) sh.thr[warp] = __popc(b);
                __syncthreads();
                int pos = count + __popc(b & ((1u << lane) - 1u));
                for (int w = 0; w < warp; ++w) pos += (int)sh.thr[w];
                for (int w = 0; w < NT / 32; ++w) count += (int)sh.thr[w];
                if (hit && pos < MAX_CAND) sh.cand[pos] = order_key(thr, (uint32_t)at);
                __syncthreads();
            }
            count = min(count, MAX_CAND);
        } else {
            unsigned long long last = ~0ull;
            for (int k = 0; k < K; ++k) {
                unsigned long long best = 0ull;
                for (int e = row.e_lo + (int)threadIdx.x; e < row.e_hi; e += NT) {
                    const unsigned long long key = order_key(order32(to_f32(row.z[e])), (uint32_t)e);
                    if (key < last && key > best) best = key;
                }
                last = block_reduce(best, MaxU64(), sh.red);
                if (threadIdx.x == 0) sh.list[k] = last;
                if (last == 0ull) break;
            }
            __syncthreads();
            return;
        }
    }
    for (int a = threadIdx.x; a < count; a += NT) {
        const unsigned long long key = sh.cand[a];
        int place = 0;
        for (int b = 0; b < count; ++b) place += sh.cand[b] > key;
        if (place < K) sh.list[place] = key;
    }
    __syncthreads();
}

// ---------------------------------------------------- log probabilities --

template <typename T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) logprobs_kernel(const LogprobArgs a, int log_split, int* err) {
    __shared__ Part red[NT / 32];
    __shared__ Part parts[MAX_SPLIT];
    __shared__ float redf[NT / 32];
    __shared__ TopShared<NT> sh;
    const int split = 1 << log_split;
    const int64_t row_i = blockIdx.x >> log_split;
    const int rank = (int)(blockIdx.x & (unsigned)(split - 1));
    if (split > 1) cluster_arrive();   // this CTA runs: its shared memory may be written
    pdl_wait();
    pdl_launch_dependents();
    constexpr int CHUNK = Row<T, NT>::CHUNK;
    uint4 x[VPT];
    Soft st{Vec<T>::lowest(), 0.f, 0.f};
    int before = 0;
    Peaks peaks{-INFINITY, -INFINITY, 0};
    int t = -1;                                      // the target; -1: none, or out of range
    auto zw = Vec<T>::wide(INFINITY);                // its logit; +inf: not counted in the loop
    {
        const Row<T, NT> row(a.logits, row_i, a.ld, a.V, rank, log_split);
        // the row's loads go out before anything waits for the target's
        const int rest = row.rest();
        if (row.lo < rest)
            row.load_chunk(row.lo, x);
        else
            row.load_rest(rest, x);
        const int64_t given = a.targets ? a.targets[row_i] : -1;
        if (given >= 0 && given < a.V) {
            t = (int)given;
            const float z = to_f32(row.z[t]);
            if (z > -INFINITY) zw = Vec<T>::wide(z);
        }
        // entries in front of the target: above it anywhere, equal to it before it.
        // Vectors before the target's count equals; inside its own vector they
        // are added below. A masked target is counted apart.
        const int tvec = row.vector_of(t);
        auto chunk = [&](int base) {
            const float largest = Vec<T>::largest(x);
            const bool better = largest > peaks.best;
            peaks.other = max_nan(peaks.other, better ? peaks.best : largest);
            peaks.best = better ? largest : peaks.best;
            peaks.base = better ? base : peaks.base;
            soft_chunk<T, true>(st, x, largest, kLog2e);
            typename Vec<T>::Count cnt;
            if (base + CHUNK <= tvec) {
#pragma unroll
                for (int r = 0; r < VPT; ++r) cnt.ge(x[r], zw);
            } else if (base >= tvec) {
#pragma unroll
                for (int r = 0; r < VPT; ++r) cnt.gt(x[r], zw);
            } else {
#pragma unroll
                for (int r = 0; r < VPT; ++r) {
                    if (base + r * NT + (int)threadIdx.x < tvec)
                        cnt.ge(x[r], zw);
                    else
                        cnt.gt(x[r], zw);
                }
            }
            before += cnt.total();
        };
        if (row.edges()) {
            const uint4 e[1] = {row.load_edge(row.edge())};
            peaks.other = Vec<T>::largest(e);
            soft_chunk<T, true>(st, e, peaks.other, kLog2e);
            typename Vec<T>::Count cnt;
            if (row.edge() < tvec)
                cnt.ge(e[0], zw);
            else
                cnt.gt(e[0], zw);
            before += cnt.total();
        }
        for (int base = row.lo; base < rest; base += CHUNK) {
            chunk(base);
            if (base + CHUNK < rest)
                row.load_chunk(base + CHUNK, x);
            else
                row.load_rest(rest, x);
        }
        if (rest < row.hi) chunk(rest);
    }
    // Once more, from an index the compiler takes for new: kept over the loop,
    // the row's sizes would not fit the registers.
    int64_t row_j = row_i;
    asm volatile("" : "+l"(row_j));
    const Row<T, NT> row(a.logits, row_j, a.ld, a.V, rank, log_split);
    const bool good = t >= 0, counted = good && Vec<T>::narrow(zw) < INFINITY;
    const float zt = counted ? Vec<T>::narrow(zw) : -INFINITY;
    if (counted && threadIdx.x == 0 && row.mine(t))
        for (int e = max(row.start(row.vector_of(t)), 0); e < t; ++e) before += to_f32(row.z[e]) == zt;
    if (good && !counted) {   // a masked target (or a NaN): every entry is compared
        before = 0;
        const float z = to_f32(row.z[t]);
        for (int e = row.e_lo + (int)threadIdx.x; e < row.e_hi; e += NT) {
            const float v = to_f32(row.z[e]);
            before += v > z || (v == z && e < t);
        }
    }
    Part part = block_part<NT / 32>(st, before, red, kLog2e);
    if (a.K > 0) slice_top(row, a.K, peaks, sh);
    if (split > 1) {
        cluster_wait();
        if (threadIdx.x == 0) send_part(parts, rank, 0u, part);
        for (int k = threadIdx.x; k < a.K; k += NT)
            st_cluster_u64(mapa_shared(smem_u32(&sh.all[rank * a.K + k]), 0u), sh.list[k]);
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
        part = combine(parts, split, kLog2e);
    }
    // masked tokens were summed as the lowest finite value, which tells
    // nothing only where the row has no larger one
    if (part.soft.ref == Vec<T>::lowest()) {
        part.soft.s = count_finite<T, NT>(row.z, a.V, redf);
        part.soft.e = 0.f;
    }
    const Dist d = distribution(part.soft, kLog2e, 1.f);
    float esum = part.soft.e;
    if (isnan(esum) && !isnan(d.s)) esum = slow_esum<T, NT>(row.z, a.V, d, redf);
    if (threadIdx.x == 0) {
        if (a.targets && !good) atomicCAS(err, 0, (int)TPMLP_ERR_ARG);
        if (a.lse) a.lse[row_j] = d.lse();
        if (a.entropy) a.entropy[row_j] = d.nothing ? 0.f : d.ln_s - esum / d.s;
        if (a.logprob) a.logprob[row_j] = good ? d.ln_p(zt) : NAN;
        if (a.rank) a.rank[row_j] = good ? part.before + 1 : 0;
    }
    const unsigned long long* all = split > 1 ? sh.all : sh.list;
    const int m = split * a.K;
    for (int i = threadIdx.x; i < m; i += NT) {
        const unsigned long long key = all[i];
        int place = i;
        if (split > 1) {
            place = 0;
            for (int j = 0; j < m; ++j) place += all[j] > key;
        }
        if (key != 0ull && place < a.K) {
            a.top_ids[row_j * a.K + place] = (int32_t)(0xffffffffu - (uint32_t)key);
            a.top_logprobs[row_j * a.K + place] = d.ln_p(order_value((uint32_t)(key >> 32)));
        }
    }
}

// --------------------------------------------------------- distillation --

// The teacher's slots of one row that are this CTA's, and its distribution:
// slot k has q_k = 2^((t_k - max t) c) / sum. The loss is
//   tau^2 (sum q ln q - sum q ln p),  ln p_v = (z_v - m) / tau - ln S,
// and needs no more of the slots than sum q ln q, their largest logit zmax and
// sum q (z - zmax), all known before the row's m and S.
struct TeacherShared {
    float sum;                      // of e over all slots
    float q_ln_q, zmax, q_z;
    int some, bad, n;               // n: slots of this CTA
};
// one of them, in dynamic shared memory ([K])
struct TeacherSlot {
    int id;
    float e;                        // q times the sum over all slots
    float z;                        // the student's logit at id, as it is before an in-place sweep
};

// A lane's first slots (k = lane + 32 u), loaded at once: all of them for K <=
// 32 SLOTS. What lies beyond is read again where it is needed.
constexpr int SLOTS = 4;
struct LaneSlots {
    int id[SLOTS];       // -1: empty, or no such slot
    float t[SLOTS];
};
__device__ __forceinline__ LaneSlots load_slots(const int32_t* ids, const float* tl, int K) {
    const int lane = threadIdx.x & 31;
    LaneSlots r;
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) {
        const int k = lane + 32 * u;
        r.id[u] = k < K ? ids[k] : -1;
        r.t[u] = k < K ? tl[k] : -INFINITY;
    }
    return r;
}

// Warp 0: statistics over the K slots (for the loss with LOSS), then the slots
// whose id is in the CTA's slice, in slot order. The student's logits they
// need are loaded first, as they are before an in-place sweep.
template <typename T, int NT>
__device__ __forceinline__ void teacher_row(const DistillArgs& a, const int32_t* ids, const float* tl,
                                            const LaneSlots& slots, const Row<T, NT>& row, bool loss, bool lists,
                                            TeacherShared& sh, TeacherSlot* list) {
    const int lane = threadIdx.x;
    const float ct = kLog2e / a.tau;
    auto logit = [&](int id) {
        return id >= 0 && id < a.V && (loss || row.mine(id)) ? to_f32(row.z[id]) : -INFINITY;
    };
    float z[SLOTS];
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) z[u] = logit(slots.id[u]);
    float mx = -INFINITY;
    int bad = 0;
    auto look = [&](int id, float t) {
        if (id != -1) mx = max_nan(mx, t);
        bad |= id < -1 || id >= a.V;
    };
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) look(slots.id[u], slots.t[u]);
    for (int k = lane + 32 * SLOTS; k < a.K; k += 32) look(ids[k], tl[k]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    bad = __any_sync(0xffffffffu, bad);
    const bool some = mx != -INFINITY;
    float s = 0.f;
    auto weight = [&](int id, float t) { return some && id != -1 ? ex2((t - mx) * ct) : 0.f; };
    float e[SLOTS];
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) {
        e[u] = weight(slots.id[u], slots.t[u]);
        s += e[u];
    }
    for (int k = lane + 32 * SLOTS; k < a.K; k += 32) s += weight(ids[k], tl[k]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float inv = 1.f / s;
    float q_ln_q = 0.f, zmax = -INFINITY, q_z = 0.f;
    if (loss && some && !bad) {
        const float log2_sum = log2f(s);
        auto entropy = [&](float ek, float t) {
            if (ek != 0.f) q_ln_q = fmaf(ek * inv, kLn2 * ((t - mx) * ct - log2_sum), q_ln_q);
        };
        auto cross = [&](float ek, float zk) {
            if (ek != 0.f) q_z = fmaf(ek * inv, zk - zmax, q_z);
        };
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            zmax = max_nan(zmax, z[u]);
            entropy(e[u], slots.t[u]);
        }
        for (int k = lane + 32 * SLOTS; k < a.K; k += 32) {
            zmax = max_nan(zmax, logit(ids[k]));
            entropy(weight(ids[k], tl[k]), tl[k]);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) zmax = max_nan(zmax, __shfl_xor_sync(0xffffffffu, zmax, off));
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) cross(e[u], z[u]);
        for (int k = lane + 32 * SLOTS; k < a.K; k += 32) cross(weight(ids[k], tl[k]), logit(ids[k]));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            q_ln_q += __shfl_xor_sync(0xffffffffu, q_ln_q, off);
            q_z += __shfl_xor_sync(0xffffffffu, q_z, off);
        }
    }
    int n = 0;
    if (lists && some && !bad) {
        auto keep = [&](bool hit, int id, float ek, float zk) {
            const uint32_t b = __ballot_sync(0xffffffffu, hit);
            if (hit) {
                const int at = n + __popc(b & ((1u << lane) - 1u));
                list[at] = TeacherSlot{id, ek, zk};
            }
            n += __popc(b);
        };
#pragma unroll
        for (int u = 0; u < SLOTS; ++u)
            keep(slots.id[u] != -1 && row.mine(slots.id[u]), slots.id[u], e[u], z[u]);
        for (int k0 = 32 * SLOTS; k0 < a.K; k0 += 32) {
            const int id = k0 + lane < a.K ? ids[k0 + lane] : -1;
            const bool hit = id != -1 && row.mine(id);
            keep(hit, id, hit ? weight(id, tl[k0 + lane]) : 0.f, hit ? to_f32(row.z[id]) : 0.f);
        }
    }
    if (lane == 0) {
        sh.sum = s;
        sh.q_ln_q = q_ln_q;
        sh.zmax = zmax;
        sh.q_z = q_z;
        sh.some = some;
        sh.bad = bad;
        sh.n = n;
    }
}

// (reference, sum) of every warp of the row's CTAs, in one place of each CTA
struct __align__(8) WarpSoft {
    float ref, s;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Up to which |lse| the gradient takes p from lse. It is one fp32 number, and
// next to a maximum of some size it holds ln S to half an ulp of itself:
// 2^-24 |lse| of every p, at most 2^-19 here for an fp32 gradient and 2^-15 for
// a bf16 one, whose own rounding is 2^-8. (Of a row whose tokens all hold a
// huge value nothing is left of ln S.)
template <typename T> constexpr float kFarLse = sizeof(T) == 2 ? 512.f : 32.f;

// The gradient of a row beyond, its statistics taken again by a reading of its
// own. Not inlined, and called where lse is needed first: the other rows are
// not to pay for it. (bf16 on GB300, all rows near / all beyond: 4096 x 128000
// 332 / 464 us, 16384 x 32000 327 / 457; fp32, 1003 x 50001: 71 / 96. Always
// taking them again in one reading, as the fused form does, costs 369, 348
// and 93. lse read at the kernel's start: 333 near for 16384 x 32000.)
template <typename T, int NT> __device__ __noinline__ void far_row(const DistillArgs& a, int log_split, int* err);

// One row, of this CTA's cluster. LOSS: loss and lse; GRAD: the gradient, with
// SUMS (LOSS has them) from this reading's statistics, else from the given lse.
//
// With both, the row is read once and stays on the chip: the slice's last
// chunk in registers, the one before it in shared memory (a thread's own
// vectors, so no barrier), 64 KB a CTA and 256 KB an SM: 4096 rows of 128000
// bf16 logits take 350 us on GB300, and DRAM moves what the algorithm has to.
// A cluster holds 131072 fp32 or 262144 bf16 logits of a row that way; a longer
// slice reads its other chunks again, last one first (fp32 rows of 131072: 5.4
// TB/s read and written, of 132500: 4.2, of 151936: 4.4).
template <typename T, int NT, bool LOSS, bool SUMS, bool GRAD>
__device__ __forceinline__ void distill_row(const DistillArgs& a, int log_split, int* err) {
    constexpr bool STAGE = LOSS && GRAD;
    constexpr int WARPS = NT / 32, CHUNK = Row<T, NT>::CHUNK;
    extern __shared__ uint4 stage[];   // STAGE: one chunk; GRAD: then the teacher's slots
    TeacherSlot* list = reinterpret_cast<TeacherSlot*>(stage + (STAGE ? CHUNK : 0));
    __shared__ WarpSoft parts[MAX_SPLIT * WARPS];
    __shared__ TeacherShared te;
    const int split = 1 << log_split;
    const int64_t row_i = blockIdx.x >> log_split;
    const int rank = (int)(blockIdx.x & (unsigned)(split - 1));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (SUMS && split > 1) cluster_arrive();   // this CTA runs: its shared memory may be written
    if (LOSS || !SUMS) {   // (a far row's kernel has done both)
        pdl_wait();
        pdl_launch_dependents();
    }
    const Row<T, NT> row(a.logits, row_i, a.ld, a.V, rank, log_split);
    T* d = GRAD ? static_cast<T*>(a.dlogits) + row_i * a.ldd : nullptr;
    const int32_t* ids = a.ids + row_i * a.K;
    const float* tl = a.teacher + row_i * a.K;
    const float c = kLog2e / a.tau;
    const int rest = row.rest();

    // A row without a live slot is not read. Every warp looks for one by
    // itself (among the first slots, as a rule), so that its loads of the row
    // are on their way before warp 0 takes the teacher's statistics.
    const LaneSlots slots = load_slots(ids, tl, a.K);
    bool live = false;
    auto counts = [&](int id, float t) { return id != -1 && (t != -INFINITY || id < -1 || id >= a.V); };
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) live = live || counts(slots.id[u], slots.t[u]);
    live = __any_sync(0xffffffffu, live);
    for (int k = 32 * SLOTS; !live && k < a.K; k += 32)
        live = __any_sync(0xffffffffu, k + lane < a.K && counts(ids[k + lane], tl[k + lane]));
    uint4 x[VPT];
    const int staged = STAGE && rest > row.lo ? rest - CHUNK : rest;   // where the chunk in shared memory starts
    const bool early = staged == row.lo;   // nothing is read through the registers before the last chunk
    if (live) {
        if (staged < rest) {
            const uint4* p = row.vectors() + staged + threadIdx.x;
#pragma unroll
            for (int r = 0; r < VPT; ++r) cp_async16(smem_u32(stage + r * NT + threadIdx.x), p + r * NT);
        }
        if (early) row.load_rest(rest, x);
    }
    if (warp == 0) teacher_row(a, ids, tl, slots, row, LOSS && rank == 0, GRAD, te, list);

    Dist dist{};
    if constexpr (SUMS) {
        Soft st{kLowest, 0.f, 0.f};
        if (live) {
            if (row.edges()) {
                const uint4 e[1] = {row.load_edge(row.edge())};
                soft_chunk<T, false>(st, e, Vec<T>::largest(e), c);
            }
            for (int base = row.lo; base < staged; base += CHUNK) {
                row.load_chunk(base, x);
                soft_chunk<T, false>(st, x, Vec<T>::largest(x), c);
            }
            if (!early) row.load_rest(rest, x);
            soft_chunk<T, false>(st, x, Vec<T>::largest(x), c);
            if (staged < rest) {
                cp_async_wait();
#pragma unroll 1
                for (int r = 0; r < VPT; r += 2) {
                    const uint4 y[2] = {stage[r * NT + threadIdx.x], stage[(r + 1) * NT + threadIdx.x]};
                    soft_chunk<T, false>(st, y, Vec<T>::largest(y), c);
                }
            }
        }
        // every warp's sums to every CTA of the row; all of them add the same
        // numbers in the same order
        float m = st.ref;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        rebase(st, m, c);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) st.s += __shfl_xor_sync(0xffffffffu, st.s, off);
        if (split > 1) {
            cluster_wait();
            if (lane < split) {
                const uint32_t at = mapa_shared(smem_u32(&parts[rank * WARPS + warp]), (uint32_t)lane);
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(m), "f"(st.s) : "memory");
            }
            cluster_arrive();
            cluster_wait();
        } else {
            if (lane == 0) parts[warp] = WarpSoft{m, st.s};
            __syncthreads();
        }
        constexpr int PPL = (MAX_SPLIT * WARPS + 31) / 32;   // parts a lane takes
        const int total = split * WARPS;
        WarpSoft part[PPL];
        m = kLowest;
#pragma unroll
        for (int u = 0; u < PPL; ++u) {
            part[u] = lane + 32 * u < total ? parts[lane + 32 * u] : WarpSoft{kLowest, 0.f};
            m = max_nan(m, part[u].ref);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        Soft s0{m, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < PPL; ++u) s0.s = fmaf(part[u].s, ex2((part[u].ref - m) * c), s0.s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s0.s += __shfl_xor_sync(0xffffffffu, s0.s, off);
        dist.ref = s0.ref;
        dist.s = s0.s;
        dist.c = c;
        dist.nothing = s0.s == 0.f;
        if (LOSS && rank == 0 && threadIdx.x == 0) {
            const float inv_tau = 1.f / a.tau, ln_s = logf(dist.s);
            // a masked token that the teacher wants: ln p = -inf
            const float cross = te.zmax == -INFINITY ? INFINITY : ln_s - (te.q_z + (te.zmax - dist.ref)) * inv_tau;
            a.loss[row_i] = te.bad ? NAN : te.some ? a.tau * a.tau * (te.q_ln_q + cross) : 0.f;
            if (a.lse) {
                // ref / tau + ln S: what the quotient's rounding left over joins ln S
                const float quot = dist.ref * inv_tau, over = fmaf(-quot, a.tau, dist.ref) * inv_tau;
                a.lse[row_i] = te.bad ? NAN : !te.some ? 0.f : dist.nothing ? -INFINITY
                               : isinf(quot) ? quot : quot + (over + ln_s);
            }
        }
    } else {
        __syncthreads();   // the teacher's statistics
        // p = 2^((z - lse tau) c); what the product's rounding left over is in s
        dist.c = c;
        dist.nothing = false;
        const float lse = a.lse_in[row_i];
        if (!(fabsf(lse) <= kFarLse<T>)) {
            far_row<T, NT>(a, log_split, err);
            return;
        }
        dist.ref = lse * a.tau;
        dist.s = ex2(fmaf(lse, a.tau, -dist.ref) * c);
    }
    if (GRAD) {
        const float w = a.grad_scale * (a.grad_tokens ? a.grad_tokens[row_i] : 1.f) * a.tau;
        const float ws = w / dist.s;   // times 2^exponent: w p
        // rows without probabilities hold `fill` and, where the teacher has some, its part
        const bool flat = te.bad || !te.some || dist.nothing;
        const float fill = te.bad ? NAN : 0.f;
        const bool same = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(row.z)) & 15) == 0;
        const F2 c2 = f2(c, c), r2 = f2(-dist.ref, -dist.ref), w2 = f2(ws, ws);
        auto store = [&](int i, const float (&v)[Vec<T>::N]) {
            T* at = d + row.start(i);
            if (same) {
                __stcs(reinterpret_cast<uint4*>(at), Vec<T>::pack(v));
            } else {
#pragma unroll
                for (int j = 0; j < Vec<T>::N; ++j) at[j] = from_f32<T>(v[j]);
            }
        };
        auto gradient = [&](const uint4& z, float (&v)[Vec<T>::N]) {
#pragma unroll
            for (int k = 0; k < Vec<T>::PAIRS; ++k) {
                float e0, e1;
                split2(mul2(add2(Vec<T>::pair(z, k), r2), c2), e0, e1);
                split2(mul2(f2(ex2(e0), ex2(e1)), w2), v[2 * k], v[2 * k + 1]);
            }
        };
        if (row.edge() <= row.full) {
            const int i = row.edge(), e0 = row.start(i);
            float v[Vec<T>::N];
            if (!flat) gradient(row.load_edge(i), v);
#pragma unroll
            for (int j = 0; j < Vec<T>::N; ++j)
                if (e0 + j >= 0 && e0 + j < row.len) d[e0 + j] = from_f32<T>(flat ? fill : v[j]);
        }
        if (flat) {
            float v[Vec<T>::N];
#pragma unroll
            for (int j = 0; j < Vec<T>::N; ++j) v[j] = fill;
            for (int i = row.lo + (int)threadIdx.x; i < row.hi; i += NT) store(i, v);
        } else {
            // Back to front: the last chunk is still in registers, what was read
            // last is the likeliest to be in L2.
            if (!SUMS && !early) row.load_rest(rest, x);
#pragma unroll
            for (int r = 0; r < VPT; ++r) {
                const int i = rest + r * NT + (int)threadIdx.x;
                if (i < row.hi) {
                    float v[Vec<T>::N];
                    gradient(x[r], v);
                    store(i, v);
                }
            }
            if (staged < rest) {
#pragma unroll
                for (int r = 0; r < VPT; ++r) {
                    float v[Vec<T>::N];
                    gradient(stage[r * NT + threadIdx.x], v);
                    store(staged + r * NT + (int)threadIdx.x, v);
                }
            }
            for (int base = staged - CHUNK; base >= row.lo; base -= CHUNK) {
                row.load_chunk(base, x);
#pragma unroll
                for (int r = 0; r < VPT; ++r) {
                    float v[Vec<T>::N];
                    gradient(x[r], v);
                    store(base + r * NT + (int)threadIdx.x, v);
                }
            }
        }
        // the teacher's tokens over the sweep; slots of one id all write the
        // row's full value
        if (te.n > 0) {
            __syncthreads();
            for (int k = threadIdx.x; k < te.n; k += NT) {
                const int id = list[k].id;
                float e = 0.f;
                for (int j = 0; j < te.n; ++j)
                    if (list[j].id == id) e += list[j].e;
                // divided, not times 1 / sum: 1 exactly where the sum is this token's alone
                d[id] = from_f32<T>(fmaf(-w, e / te.sum, flat ? fill : ws * ex2(dist.exponent(list[k].z))));
            }
        }
    }
    if (rank == 0 && threadIdx.x == 0 && te.bad) atomicCAS(err, 0, (int)TPMLP_ERR_ARG);
}

template <typename T, int NT>
__device__ __noinline__ void far_row(const DistillArgs& a, int log_split, int* err) {
    distill_row<T, NT, false, true, true>(a, log_split, err);
}

template <typename T, int NT, bool GRAD>
__global__ void __launch_bounds__(NT, 1024 / NT) distill_loss_kernel(const DistillArgs a, int log_split, int* err) {
    distill_row<T, NT, true, true, GRAD>(a, log_split, err);
}

// __grid_constant__: the far rows' call takes the arguments by address.
template <typename T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT)
    distill_grad_kernel(const __grid_constant__ DistillArgs a, int log_split, int* err) {
    distill_row<T, NT, false, false, true>(a, log_split, err);
}

// ---------------------------------------------------------------- launch --

// CTAs per row, as a power of two. Few rows: enough CTAs to occupy the SMs
// four times over, while a slice still has a vector for every thread. A
// slice should also be no longer than `hold` vectors (0: any length).
int row_split(int64_t N, int64_t row_bytes, int threads, int64_t hold) {
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

template <typename T, int NT>
tpmlp_status distill_rows(const DistillArgs& a, cudaStream_t s, int* err) {
    const int64_t bytes = a.V * (int64_t)sizeof(T);
    const size_t list = a.K * sizeof(TeacherSlot);
    if (a.dlogits == nullptr) {
        const int split = row_split(a.N, bytes, NT, 0);
        LaunchScope ls("vocab_distill", s);
        return launch_rows(distill_loss_kernel<T, NT, false>, NT, 0, a.N, split, s, a, split, err);
    }
    if (a.loss == nullptr) {
        const int split = row_split(a.N, bytes, NT, 0);
        LaunchScope ls("vocab_distill_backward", s);
        return launch_rows(distill_grad_kernel<T, NT>, NT, list, a.N, split, s, a, split, err);
    }
    constexpr int CHUNK = Row<T, NT>::CHUNK;
    // what a launch has without asking for more
    static_assert(CHUNK * sizeof(uint4) + TPMLP_MAX_TEACHER * sizeof(TeacherSlot) +
                          MAX_SPLIT * (NT / 32) * sizeof(WarpSoft) + sizeof(TeacherShared) <= 48 * 1024,
                  "shared memory");
    const int split = row_split(a.N, bytes, NT, 2 * CHUNK);
    LaunchScope ls("vocab_distill_with_grad", s);
    return launch_rows(distill_loss_kernel<T, NT, true>, NT, CHUNK * sizeof(uint4) + list, a.N, split, s, a,
                       split, err);
}

// Many short rows: the fewest threads whose two chunks hold the row, for more
// rows an SM; a row of a few KB is latency for 256 threads. (4000 bf16 rows on
// GB300, loss and gradient, 64 / 128 / 256 threads: 8 KB 25 / 29 / 45 us, 16 KB
// 35 / 37 / 49, 32 KB 71 / 55 / 60, 64 KB 129 / 97 / 91; loss alone, 8 KB 16 /
// 21 / 31.) Few rows are split over more CTAs instead.
template <typename T>
tpmlp_status distill_launch(const DistillArgs& a, cudaStream_t s, int* err) {
    const int64_t vectors = a.V * (int64_t)sizeof(T) / 16;
    if (a.N >= 4LL * device_sm_count()) {
        if (vectors <= 2 * Row<T, 64>::CHUNK) return distill_rows<T, 64>(a, s, err);
        if (vectors <= 2 * Row<T, 128>::CHUNK) return distill_rows<T, 128>(a, s, err);
    }
    return distill_rows<T, ROW_THREADS>(a, s, err);
}

// Many rows take smaller CTAs, for more rows an SM: 64 threads where their two
// chunks hold the row, else 128. The list's bound is the K-th largest of the
// threads' maxima, so fewer threads leave more candidates, in the end more than
// there is room for: at most one token of the list for two threads, in rows of
// more chunks one for six. (bf16 on GB300, 64 / 128 / 256 threads: 4000 rows of
// 8 KB, K = 0 16 / 22 / 37 us, K = 20 29 / 36 / 56; of 32 KB, K = 20 51 / 53 / 61;
// 8192 rows of 256 KB, K = 0 335 / 321 / 326, K = 20 503 / 386 / 376; K = 64 - /
// 654 / 467.)
template <typename T>
tpmlp_status logprobs_launch(const LogprobArgs& a, int log_split, cudaStream_t s, int* err) {
    const int64_t vectors = a.V * (int64_t)sizeof(T) / 16;
    if (a.N >= 4LL * device_sm_count()) {   // not split
        if (vectors <= 2 * Row<T, 64>::CHUNK && a.K * 2 <= 64)
            return launch_rows(logprobs_kernel<T, 64>, 64, 0, a.N, log_split, s, a, log_split, err);
        if (a.K * (vectors <= 2 * Row<T, 128>::CHUNK ? 2 : 6) <= 128)
            return launch_rows(logprobs_kernel<T, 128>, 128, 0, a.N, log_split, s, a, log_split, err);
    }
    return launch_rows(logprobs_kernel<T, ROW_THREADS>, ROW_THREADS, 0, a.N, log_split, s, a, log_split, err);
}

}  // namespace

tpmlp_status run_vocab_logprobs(int f32, const LogprobArgs& a, cudaStream_t s) {
    if (a.N == 0) return TPMLP_OK;
    int* err = device_error_word();
    if (err == nullptr) return TPMLP_ERR_CUDA;
    const int split = row_split(a.N, a.V * (f32 ? 4 : 2), ROW_THREADS, 0);
    LaunchScope ls("vocab_logprobs", s);
    return f32 ? logprobs_launch<float>(a, split, s, err) : logprobs_launch<__nv_bfloat16>(a, split, s, err);
}

tpmlp_status run_vocab_distill(int f32, const DistillArgs& a, cudaStream_t s) {
    if (a.N == 0) return TPMLP_OK;
    int* err = device_error_word();
    if (err == nullptr) return TPMLP_ERR_CUDA;
    return f32 ? distill_launch<float>(a, s, err) : distill_launch<__nv_bfloat16>(a, s, err);
}

}  // namespace tpmlp
