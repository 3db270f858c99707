// Clipped policy loss of given tokens over vocabulary rows, and its gradient.
//
//   ln p = log softmax(z / tau),  l = ln p_t,  rho = exp(l - old)
//   loss = -min(rho A, clip(rho, 1 - low, 1 + high) A) + beta k,
//   k = e^r - r - 1 with r = ref - l
//   s = d loss / d l = -A rho [rho inside its border on A's side] + beta (1 - e^r)
//   dz_v = w ([v = t] - p_v),  w = g s / tau
//
// As for the distillation, a row belongs to a cluster of 1 to 8 CTAs, which
// read it once: loss and gradient together keep the slice on the chip (last
// chunk in registers, the one before in shared memory). The maximum and the
// sum are taken without the given token, R = sum_{v != t}, and the token's own
// term is added at the end, so that 1 - p_t = R / (R + e_t) and, for p_t > 1/2,
// l = -log1p(R / e_t) keep all their digits for tokens the policy is sure of.
//
// HBM bounds it: 4096 rows of 128000 bf16 logits, loss and gradient at once, take
// 300 us on GB300, 6.1 TB/s (a quarter of the rows is without a token and only
// written); the loss alone of 1003 x 50001 fp32 40 us, the gradient 50.
#include "vocab_rows.cuh"

namespace tpmlp {
namespace {

// A number as the sum of two fp32 ones.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {   // Knuth: a + b exactly
    const float s = a + b, t = s - a;
    return Two{s, (a - (s - t)) + (b - t)};
}

// (z - ref) / tau - ln S to more digits than one fp32 number holds (l enters the
// ratio and the KL term as a difference of near numbers): ln S as k ln 2 + ln f
// with S = 2^k f, 1/sqrt(2) <= f < sqrt(2), ln 2 in two parts of which the first
// times k is exact (Cody and Waite's reduction, used backwards).
__device__ __forceinline__ Two log_prob(float z, float ref, float tau, float S) {
    const float inv_tau = 1.f / tau;
    const Two d = two_sum(z, -ref);
    const float q = d.hi * inv_tau;
    if (isinf(q)) return Two{q, 0.f};
    const float q_lo = (fmaf(-q, tau, d.hi) + d.lo) * inv_tau;
    int k;
    float f = frexpf(S, &k);
    if (f < 0.70710678f) {
        f *= 2.f;
        --k;
    }
    constexpr float kLn2Hi = 355.f / 512.f;   // 9 bits, Cody and Waite's own split
    constexpr float kLn2Lo = (float)(0.69314718055994530942 - 355. / 512.);
    const Two h = two_sum(q, -(float)k * kLn2Hi);
    const float lo = h.lo + (q_lo - fmaf((float)k, kLn2Lo, logf(f)));
    Two r;
    r.hi = h.hi + lo;
    r.lo = isinf(r.hi) ? 0.f : lo - (r.hi - h.hi);
    return r;
}

// e^x - x - 1: by its series where the difference would cancel (Taylor; the
// next term is below 2^-26 of the sum for |x| < 1/2).
__device__ __forceinline__ float kl_term(float x) {
    if (fabsf(x) < 0.5f) {
        float s = 1.f / 362880.f;
        s = fmaf(s, x, 1.f / 40320.f);
        s = fmaf(s, x, 1.f / 5040.f);
        s = fmaf(s, x, 1.f / 720.f);
        s = fmaf(s, x, 1.f / 120.f);
        s = fmaf(s, x, 1.f / 24.f);
        s = fmaf(s, x, 1.f / 6.f);
        s = fmaf(s, x, 0.5f);
        return s * x * x;
    }
    return x == INFINITY ? x : expm1f(x) - x;
}

struct Terms {
    float loss, kl, slope;
};

__device__ __forceinline__ Terms policy_terms(const PolicyArgs& a, int64_t row, Two l) {
    Terms t{0.f, 0.f, 0.f};
    const float adv = a.advantages[row];
    if (adv != 0.f) {   // nothing to gain: no matter what the ratio is
        const float rho = expf((l.hi - a.old_logprobs[row]) + l.lo);
        const float border = adv > 0.f ? 1.f + a.high : 1.f - a.low;
        const bool held = adv > 0.f ? rho > border : rho < border;   // a NaN is not held
        t.loss = -adv * (held ? border : rho);
        t.slope = held ? 0.f : -adv * rho;
    }
    if (a.ref_logprobs != nullptr) {
        const float r = (a.ref_logprobs[row] - l.hi) - l.lo;
        t.kl = kl_term(r);
        if (a.kl_coef != 0.f) {
            t.loss = fmaf(a.kl_coef, t.kl, t.loss);
            t.slope = fmaf(-a.kl_coef, expm1f(r), t.slope);
        }
    }
    return t;
}

// x without element e of vector i, in a chunk whose thread holds vectors first,
// first + NT, ...
template <typename T, int NT, int R>
__device__ __forceinline__ void drop_element(uint4 (&x)[R], int first, int i, int e) {
    const int o = i - first;
    if (o < 0 || o >= R * NT || o % NT != 0) return;   // one thread of the row has it
    constexpr int WORD = 4 / (int)sizeof(T);           // elements of a 32-bit word
    const uint32_t keep = sizeof(T) == 4 ? 0u : e % WORD == 0 ? 0xffff0000u : 0x0000ffffu;
    const int word = e / WORD;
    auto drop = [&](uint32_t w) { return (w & keep) | (Vec<T>::MASKED & ~keep); };
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (o == r * NT) {
            if (word == 0) x[r].x = drop(x[r].x);
            if (word == 1) x[r].y = drop(x[r].y);
            if (word == 2) x[r].z = drop(x[r].z);
            if (word == 3) x[r].w = drop(x[r].w);
        }
}

// Up to which |l| the gradient of a later call takes p from l, one fp32 number: its
// rounding, 2^-24 of |l| at most, and those of z - z_t, log2e / tau and l log2e, as
// much again each, come to less than 2^-17 of p for fp32 logits (2^-20 in the mean
// square), 2^-14 (2^-16) for bf16 ones, whose gradient is rounded to 2^-9. A row
// beyond is read twice.
template <typename T> constexpr float kFarLogprob = sizeof(T) == 2 ? 512.f : 32.f;

template <typename T, int NT> __device__ __noinline__ void far_policy_row(const PolicyArgs& a, int log_split, int* err);

// One row, of this CTA's cluster. LOSS: loss, logprob, kl; GRAD: the gradient,
// with SUMS (LOSS has them) from this reading's statistics, else from the given l.
template <typename T, int NT, bool LOSS, bool SUMS, bool GRAD>
__device__ __forceinline__ void policy_row(const PolicyArgs& a, int log_split, int* err) {
    constexpr bool STAGE = LOSS && GRAD;
    constexpr int WARPS = NT / 32, CHUNK = Row<T, NT>::CHUNK;
    extern __shared__ uint4 stage[];   // STAGE: one chunk
    __shared__ WarpSoft parts[MAX_SPLIT * WARPS];
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
    const int64_t target = a.targets[row_i];
    const bool live = target >= 0 && target < a.V, bad = target >= a.V;
    const int t = live ? (int)target : 0;
    const bool owner = live && row.mine(t);
    const int tv = owner ? row.vector_of(t) : -2, te = owner ? t - row.start(tv) : 0;
    const float c = kLog2e / a.tau;
    const int rest = row.rest();
    float zt = -INFINITY;
    if (live) zt = to_f32(row.z[t]);   // as it is before an in-place sweep
    const float g = GRAD ? a.grad_scale * (a.grad_tokens ? a.grad_tokens[row_i] : 1.f) : 0.f;

    uint4 x[VPT];
    const int staged = STAGE && rest > row.lo ? rest - CHUNK : rest;   // where the chunk in shared memory starts
    const bool early = staged == row.lo;   // nothing is read through the registers before the last chunk

    // p_v = 2^((z_v - ref) c + shift) / s
    float ref = 0.f, s = 1.f, shift = 0.f, others = 0.f, w = 0.f;
    bool flat = !live;   // rows without a gradient hold one value, fill
    float fill = bad ? NAN : 0.f;
    if constexpr (SUMS) {
        Soft st{kLowest, 0.f, 0.f};
        if (live) {
            if (staged < rest) {
                const uint4* p = row.vectors() + staged + threadIdx.x;
#pragma unroll
                for (int r = 0; r < VPT; ++r) cp_async16(smem_u32(stage + r * NT + threadIdx.x), p + r * NT);
            }
            if (early) row.load_rest(rest, x);
            if (row.edges()) {
                uint4 e[1] = {row.load_edge(row.edge())};
                drop_element<T, NT>(e, row.edge(), tv, te);
                soft_chunk<T, false>(st, e, Vec<T>::largest(e), c);
            }
            for (int base = row.lo; base < staged; base += CHUNK) {
                row.load_chunk(base, x);
                drop_element<T, NT>(x, base + (int)threadIdx.x, tv, te);
                soft_chunk<T, false>(st, x, Vec<T>::largest(x), c);
            }
            if (!early) row.load_rest(rest, x);
            drop_element<T, NT>(x, rest + (int)threadIdx.x, tv, te);
            soft_chunk<T, false>(st, x, Vec<T>::largest(x), c);
            if (staged < rest) {
                cp_async_wait();
#pragma unroll 1
                for (int r = 0; r < VPT; r += 2) {
                    uint4 y[2] = {stage[r * NT + threadIdx.x], stage[(r + 1) * NT + threadIdx.x]};
                    drop_element<T, NT>(y, staged + r * NT + (int)threadIdx.x, tv, te);
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
        m = max_nan(zt, kLowest);
#pragma unroll
        for (int u = 0; u < PPL; ++u) {
            part[u] = lane + 32 * u < total ? parts[lane + 32 * u] : WarpSoft{kLowest, 0.f};
            m = max_nan(m, part[u].ref);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        float R = 0.f;
#pragma unroll
        for (int u = 0; u < PPL; ++u) R = fmaf(part[u].s, ex2((part[u].ref - m) * c), R);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) R += __shfl_xor_sync(0xffffffffu, R, off);
        const float own = ex2((zt - m) * c);   // 0 for a masked token
        ref = m;
        s = R + own;
        others = s == 0.f ? 1.f : R / s;
        Two l{-INFINITY, 0.f};
        if (s != s)
            l.hi = NAN;
        else if (own > R)
            l.hi = -log1pf(R / own);
        else if (s != 0.f && zt > -INFINITY)   // (where its term underflowed, its logarithm need not)
            l = log_prob(zt, ref, a.tau, s);
        if (live) {
            const Terms y = policy_terms(a, row_i, l);
            w = g * y.slope / a.tau;
            flat = s == 0.f || w == 0.f;
            if (s == 0.f && w != 0.f) fill = NAN;   // all masked, the loss infinite: p is 0 / 0
            if (LOSS && rank == 0 && threadIdx.x == 0) {
                a.loss[row_i] = y.loss;
                if (a.logprob) a.logprob[row_i] = l.hi;
                if (a.kl) a.kl[row_i] = y.kl;
            }
        } else if (LOSS && rank == 0 && threadIdx.x == 0) {
            const float v = bad ? NAN : 0.f;
            a.loss[row_i] = v;
            if (a.logprob) a.logprob[row_i] = v;
            if (a.kl) a.kl[row_i] = v;
        }
    } else {
        const float l = a.logprob_in[row_i];
        if (live) {
            w = g * policy_terms(a, row_i, Two{l, 0.f}).slope / a.tau;
            flat = w == 0.f;   // and the row is not read
            if (!flat && !(fabsf(l) <= kFarLogprob<T>)) {
                far_policy_row<T, NT>(a, log_split, err);
                return;
            }
        }
        ref = zt;
        shift = l * kLog2e;
        others = -expm1f(l);
        if (split > 1) {   // every CTA has its zt before one of them writes there
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
    }
    if (GRAD) {
        const float ws = -w / s;
        const bool same = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(row.z)) & 15) == 0;
        const F2 c2 = f2(c, c), r2 = f2(-ref, -ref), w2 = f2(ws, ws), h2 = f2(shift, shift);
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
                const F2 from = add2(Vec<T>::pair(z, k), r2);
                split2(SUMS ? mul2(from, c2) : fma2(from, c2, h2), e0, e1);
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
            if (!SUMS) row.load_rest(rest, x);
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
            // the token itself, over the sweep
            __syncthreads();
            if (owner && threadIdx.x == 0) d[t] = from_f32<T>(w * others);
        }
    }
    if (rank == 0 && threadIdx.x == 0 && bad) atomicCAS(err, 0, (int)TPMLP_ERR_ARG);
}

template <typename T, int NT>
__device__ __noinline__ void far_policy_row(const PolicyArgs& a, int log_split, int* err) {
    policy_row<T, NT, false, true, true>(a, log_split, err);
}

template <typename T, int NT, bool GRAD>
__global__ void __launch_bounds__(NT, 1024 / NT) policy_loss_kernel(const PolicyArgs a, int log_split, int* err) {
    policy_row<T, NT, true, true, GRAD>(a, log_split, err);
}

// __grid_constant__: the far rows' call takes the arguments by address.
template <typename T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT)
    policy_grad_kernel(const __grid_constant__ PolicyArgs a, int log_split, int* err) {
    policy_row<T, NT, false, false, true>(a, log_split, err);
}

template <typename T, int NT>
tpmlp_status policy_rows(const PolicyArgs& a, cudaStream_t s, int* err) {
    const int64_t bytes = a.V * (int64_t)sizeof(T);
    if (a.dlogits == nullptr) {
        const int split = row_split(a.N, bytes, NT, 0);
        LaunchScope ls("vocab_policy", s);
        return launch_rows(policy_loss_kernel<T, NT, false>, NT, 0, a.N, split, s, a, split, err);
    }
    if (a.loss == nullptr) {
        const int split = row_split(a.N, bytes, NT, 0);
        LaunchScope ls("vocab_policy_backward", s);
        return launch_rows(policy_grad_kernel<T, NT>, NT, 0, a.N, split, s, a, split, err);
    }
    constexpr int CHUNK = Row<T, NT>::CHUNK;
    static_assert(CHUNK * sizeof(uint4) + MAX_SPLIT * (NT / 32) * sizeof(WarpSoft) <= 48 * 1024, "shared memory");
    const int split = row_split(a.N, bytes, NT, 2 * CHUNK);
    LaunchScope ls("vocab_policy_with_grad", s);
    return launch_rows(policy_loss_kernel<T, NT, true>, NT, CHUNK * sizeof(uint4), a.N, split, s, a, split, err);
}

// Many short rows take smaller CTAs, for more rows an SM, as the distillation's do.
template <typename T>
tpmlp_status policy_launch(const PolicyArgs& a, cudaStream_t s, int* err) {
    const int64_t vectors = a.V * (int64_t)sizeof(T) / 16;
    if (a.N >= 4LL * device_sm_count()) {
        if (vectors <= 2 * Row<T, 64>::CHUNK) return policy_rows<T, 64>(a, s, err);
        if (vectors <= 2 * Row<T, 128>::CHUNK) return policy_rows<T, 128>(a, s, err);
    }
    return policy_rows<T, ROW_THREADS>(a, s, err);
}

}  // namespace

tpmlp_status run_vocab_policy(int f32, const PolicyArgs& a, cudaStream_t s) {
    if (a.N == 0) return TPMLP_OK;
    int* err = device_error_word();
    if (err == nullptr) return TPMLP_ERR_CUDA;
    return f32 ? policy_launch<float>(a, s, err) : policy_launch<__nv_bfloat16>(a, s, err);
}

}  // namespace tpmlp
