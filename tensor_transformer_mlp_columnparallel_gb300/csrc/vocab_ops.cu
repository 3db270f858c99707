// Token log probabilities and distillation over vocabulary rows.
//
// vocab_logprobs: per row m = max z, S = sum exp(z - m), lse = m + ln S, the
//   given token's z_t - lse and rank, the entropy ln S - (sum e (z - m)) / S
//   with e = exp(z - m), and the K largest logits.
// vocab_distill: q = softmax of the teacher's slots over tau, p = softmax(z / tau),
//   loss = tau^2 sum q (ln q - ln p), dz = w (p - q) with w = g tau.
#include <cuda_bf16.h>

#include <cmath>

#include "act.cuh"
#include "ptx.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int ROW_THREADS = 256;

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return bf2f(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Whole-block reduction in a fixed order; every thread gets the result.
template <typename T, typename Op>
__device__ __forceinline__ T block_reduce(T v, Op op, T* red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, off));
    __syncthreads();   // red may hold an earlier reduction's values
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    T r = red[0];
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) r = op(r, red[w]);
    return r;
}

struct Sum {
    template <typename T> __device__ T operator()(T a, T b) const { return a + b; }
};
struct MaxNan {
    __device__ float operator()(float a, float b) const { return max_nan(a, b); }
};
struct MaxU64 {
    __device__ unsigned long long operator()(unsigned long long a, unsigned long long b) const {
        return a > b ? a : b;
    }
};

// One number per entry that falls with the logit, then rises with the index:
// the list's order. (z + 0 turns -0 into +0.)
__device__ __forceinline__ unsigned long long order_key(float z, uint32_t v) {
    const uint32_t b = __float_as_uint(z + 0.f);
    const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return ((unsigned long long)o << 32) | (0xffffffffu - v);
}

// z - lse where lse = -inf (no finite logit) leaves nothing but -inf
__device__ __forceinline__ float log_prob(float z, float m, float ln_s, float lse) {
    return lse == -INFINITY ? -INFINITY : (z - m) - ln_s;
}

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) logprobs_kernel(const LogprobArgs a, int* err) {
    __shared__ float red[ROW_THREADS / 32];
    __shared__ int redi[ROW_THREADS / 32];
    __shared__ unsigned long long redk[ROW_THREADS / 32];
    const int64_t row = blockIdx.x;
    const T* z = static_cast<const T*>(a.logits) + row * a.ld;
    float m = -INFINITY;
    for (int64_t i = threadIdx.x; i < a.V; i += ROW_THREADS) m = max_nan(m, to_f32(z[i]));
    m = block_reduce(m, MaxNan(), red);
    const float ms = m == -INFINITY ? 0.f : m;
    const int64_t t = a.targets ? a.targets[row] : 0;
    const bool good = t >= 0 && t < a.V;
    const float zt = good ? to_f32(z[t]) : 0.f;
    float s = 0.f, es = 0.f;
    int before = 0;
    for (int64_t i = threadIdx.x; i < a.V; i += ROW_THREADS) {
        const float x = to_f32(z[i]);
        const float d = x - ms, e = expf(d);
        s += e;
        es += e == 0.f ? 0.f : e * d;
        before += x > zt || (x == zt && i < t);
    }
    s = block_reduce(s, Sum(), red);
    es = block_reduce(es, Sum(), red);
    before = block_reduce(before, Sum(), redi);
    const float ln_s = logf(s), lse = ms + ln_s;
    if (threadIdx.x == 0) {
        if (a.targets && !good) atomicCAS(err, 0, (int)TPMLP_ERR_ARG);
        if (a.lse) a.lse[row] = lse;
        if (a.entropy) a.entropy[row] = s == 0.f ? 0.f : ln_s - es / s;
        if (a.logprob) a.logprob[row] = good ? log_prob(zt, ms, ln_s, lse) : NAN;
        if (a.rank) a.rank[row] = good ? before + 1 : 0;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < a.K; ++k) {
        unsigned long long best = 0;
        for (int64_t i = threadIdx.x; i < a.V; i += ROW_THREADS) {
            const unsigned long long key = order_key(to_f32(z[i]), (uint32_t)i);
            if (key < last && key > best) best = key;
        }
        last = block_reduce(best, MaxU64(), redk);
        if (threadIdx.x == 0) {
            const uint32_t v = 0xffffffffu - (uint32_t)last;
            a.top_ids[row * a.K + k] = (int32_t)v;
            a.top_logprobs[row * a.K + k] = log_prob(to_f32(z[v]), ms, ln_s, lse);
        }
    }
}

// The teacher's distribution of one row: slot k has q_k = exp(t_k / tau - tm) / sum.
struct Teacher {
    float tm, sum;
    bool some;   // a slot with a probability
    bool bad;    // an id outside [-1, V)
};

__device__ __forceinline__ Teacher teacher_stats(const DistillArgs& a, int64_t row, float* red) {
    const int32_t* ids = a.ids + row * a.K;
    const float* tl = a.teacher + row * a.K;
    float mx = -INFINITY, bad = 0.f;
    for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
        const int id = ids[k];
        if (id != -1) mx = max_nan(mx, tl[k] / a.tau);
        if (id < -1 || id >= a.V) bad = 1.f;
    }
    Teacher r;
    r.tm = block_reduce(mx, MaxNan(), red);
    r.bad = block_reduce(bad, MaxNan(), red) != 0.f;
    r.some = r.tm != -INFINITY;
    float s = 0.f;
    if (r.some)
        for (int k = threadIdx.x; k < a.K; k += blockDim.x)
            if (ids[k] != -1) s += expf(tl[k] / a.tau - r.tm);
    r.sum = block_reduce(s, Sum(), red);
    return r;
}

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) distill_kernel(const DistillArgs a, int* err) {
    __shared__ float red[ROW_THREADS / 32];
    __shared__ float fix[TPMLP_MAX_TEACHER];
    const int64_t row = blockIdx.x;
    const T* z = static_cast<const T*>(a.logits) + row * a.ld;
    T* d = a.dlogits ? static_cast<T*>(a.dlogits) + row * a.ldd : nullptr;
    const int32_t* ids = a.ids + row * a.K;
    const float* tl = a.teacher + row * a.K;
    const Teacher te = teacher_stats(a, row, red);
    if (te.bad || !te.some) {
        const float fill = te.bad ? NAN : 0.f;
        if (threadIdx.x == 0) {
            if (te.bad) atomicCAS(err, 0, (int)TPMLP_ERR_ARG);
            if (a.loss) a.loss[row] = fill;
            if (a.lse) a.lse[row] = fill;
        }
        if (d)
            for (int64_t i = threadIdx.x; i < a.V; i += ROW_THREADS) d[i] = from_f32<T>(fill);
        return;
    }
    float lse;
    if (a.loss) {
        float m = -INFINITY;
        for (int64_t i = threadIdx.x; i < a.V; i += ROW_THREADS) m = max_nan(m, to_f32(z[i]));
        m = block_reduce(m, MaxNan(), red);
        const float ms = m == -INFINITY ? 0.f : m / a.tau;
        float s = 0.f;
        for (int64_t i = threadIdx.x; i < a.V; i += ROW_THREADS) s += expf(to_f32(z[i]) / a.tau - ms);
        s = block_reduce(s, Sum(), red);
        lse = ms + logf(s);
        float loss = 0.f;
        for (int k = threadIdx.x; k < a.K; k += ROW_THREADS) {
            if (ids[k] == -1) continue;
            const float lq = tl[k] / a.tau - te.tm - logf(te.sum);
            const float q = expf(lq);
            if (q == 0.f) continue;
            loss += q * (lq - log_prob(to_f32(z[ids[k]]) / a.tau, ms, logf(s), lse));
        }
        loss = block_reduce(loss, Sum(), red);
        if (threadIdx.x == 0) {
            a.loss[row] = a.tau * a.tau * loss;
            if (a.lse) a.lse[row] = lse;
        }
    } else {
        lse = a.lse_in[row];
    }
    if (!d) return;
    const float w = a.grad_scale * (a.grad_tokens ? a.grad_tokens[row] : 1.f) * a.tau;
    auto prob = [&](float x) { return lse == -INFINITY ? 0.f : expf(x / a.tau - lse); };
    // the teacher's tokens, from the logits as they are before an in-place sweep
    for (int k = threadIdx.x; k < a.K; k += ROW_THREADS) {
        const int id = ids[k];
        float q = 0.f;
        if (id != -1)
            for (int j = 0; j < a.K; ++j)
                if (ids[j] == id) q += expf(tl[j] / a.tau - te.tm) / te.sum;
        fix[k] = id != -1 ? w * (prob(to_f32(z[id])) - q) : 0.f;
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < a.V; i += ROW_THREADS) d[i] = from_f32<T>(w * prob(to_f32(z[i])));
    __syncthreads();
    for (int k = threadIdx.x; k < a.K; k += ROW_THREADS)
        if (ids[k] != -1) d[ids[k]] = from_f32<T>(fix[k]);   // slots of one id hold one value
}

}  // namespace

tpmlp_status run_vocab_logprobs(int f32, const LogprobArgs& a, cudaStream_t s) {
    if (a.N == 0) return TPMLP_OK;
    int* err = device_error_word();
    if (err == nullptr) return TPMLP_ERR_CUDA;
    {
        LaunchScope ls("vocab_logprobs", s);
        if (f32)
            logprobs_kernel<float><<<(unsigned)a.N, ROW_THREADS, 0, s>>>(a, err);
        else
            logprobs_kernel<__nv_bfloat16><<<(unsigned)a.N, ROW_THREADS, 0, s>>>(a, err);
    }
    return cudaGetLastError() == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

tpmlp_status run_vocab_distill(int f32, const DistillArgs& a, cudaStream_t s) {
    if (a.N == 0) return TPMLP_OK;
    int* err = device_error_word();
    if (err == nullptr) return TPMLP_ERR_CUDA;
    {
        LaunchScope ls(a.dlogits == nullptr ? "vocab_distill" : a.loss ? "vocab_distill_with_grad"
                                                                       : "vocab_distill_backward", s);
        if (f32)
            distill_kernel<float><<<(unsigned)a.N, ROW_THREADS, 0, s>>>(a, err);
        else
            distill_kernel<__nv_bfloat16><<<(unsigned)a.N, ROW_THREADS, 0, s>>>(a, err);
    }
    return cudaGetLastError() == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

}  // namespace tpmlp
