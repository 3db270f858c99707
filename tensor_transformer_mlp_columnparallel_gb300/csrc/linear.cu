// What the split linear layers' backward does besides its products:
//   dZ = dY act'(Z),  db = sum_n dZ
// in one pass over dY and Z, which memory bounds: a thread has a few columns of
// many rows, writes dZ and keeps the columns' sums (of dZ before it is rounded) in
// fp32; a second launch adds the CTAs' sums in order.
#include <cuda_bf16.h>

#include "row_ring.cuh"

namespace tpmlp {
namespace {

constexpr int COLS = 128;   // threads (accesses) of a CTA

struct DactParams {
    DactArgs a;
    int S;
    int stall;   // failure-detection self test
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

// The same with rows in turn: a CTA has one panel of F columns (an even share of
// at most LONGEST) and its groups every so many rows of it, which come to shared
// memory by bulk copies of up to 16 KB (fp32: 32 KB). (4096 x 16384 bf16, gelu, with
// the bias gradient on GB300: 75 us, 5.4 TB/s read and written; between the products of
// a whole call 86, by columns 99 there. Four issue slots of five are the derivative's.)
// The ring has 96 KB for bf16 and 192 KB for fp32, so two CTAs an SM or one.
constexpr int TURN_THREADS = 512, TURN_STAGES = 3;
constexpr int TURN_SMS = 152;
constexpr int turn_ctas(int elem_size) { return elem_size == 2 ? 2 : 1; }   // an SM

template <typename T, int NT, bool FULL>
__global__ void __launch_bounds__(TURN_THREADS, turn_ctas(sizeof(T))) dact_turns_kernel(const DactParams p, int act, int panels, int width,
                                                                     int* err, uint64_t timeout_ns) {
    using Ring = RowRing<T, 16, 2, TURN_STAGES, TURN_THREADS, NT, FULL>;
    using A = typename Ring::A;
    using Word = typename Ring::Word;
    constexpr int R = Ring::R;
    extern __shared__ __align__(16) uint4 ring_memory[];
    __shared__ uint64_t bars[Ring::GROUPS * TURN_STAGES];
    __shared__ uint64_t spare[Ring::GROUPS];
    __shared__ int late[2][Ring::GROUPS];
    const DactArgs& a = p.a;
    const int panel = blockIdx.x % panels, chunk = blockIdx.x / panels;
    const int64_t c0 = (int64_t)panel * width;
    const int cols = (int)(a.F - c0 < width ? a.F - c0 : width);   // of this panel
    if (threadIdx.x < 2 * Ring::GROUPS) (&late[0][0])[threadIdx.x] = 0;
    __syncthreads();
    Ring ring(ring_memory, bars, cols);
    const uint32_t N = (uint32_t)a.N, step = (uint32_t)p.S * Ring::GROUPS, first = (uint32_t)chunk * Ring::GROUPS + ring.group;
    pdl_wait();
    pdl_launch_dependents();
    auto ask = [&](int s, uint32_t row) {
        ring.ask(s, row < N, [&](int to) {
            ring.fetch(to, 0, static_cast<const T*>(a.dY) + c0, row, a.lddy);
            ring.fetch(to, 1, static_cast<const T*>(a.Z) + c0, row, a.ldz);
        });
    };
#pragma unroll
    for (int s = 0; s < TURN_STAGES; ++s) ask(s, first + s * step);
    float sum[R][A::N];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < A::N; ++j) sum[i][j] = 0.f;
    int turn = 0;
    uint32_t row = first;
    const bool go = !p.stall || ring.stall(&spare[ring.group], &late[0][ring.group], err, timeout_ns);
    for (; go && row < N; row += step, turn ^= 1, ring.next()) {
        volatile int* flag = &late[turn][ring.group];
        const bool ok = ring.wait(flag, err, timeout_ns);
        Word g[R], z[R];
#pragma unroll
        for (int i = 0; i < R; ++i) g[i] = ring.at(0, i), z[i] = ring.at(1, i);
        group_sync<NT>(ring.group);
        if (!ok || (NT > 32 && *flag)) break;   // the whole group
        ask(ring.k, row + TURN_STAGES * step);
        Word* out = reinterpret_cast<Word*>(static_cast<T*>(a.dZ) + (int64_t)row * a.F + c0) + ring.t;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (!ring.mine(i)) continue;
            float v[A::N], s[A::N];
            A::unpack(g[i], v);
            A::unpack(z[i], s);
            auto apply = [&](auto fixed) {
#pragma unroll
                for (int j = 0; j < A::N; ++j) v[j] *= slope<T>(decltype(fixed)::value, s[j]);
            };
            switch (act) {
                case TPMLP_ACT_RELU: apply(std::integral_constant<int, TPMLP_ACT_RELU>()); break;
                case TPMLP_ACT_GELU_ERF: apply(std::integral_constant<int, TPMLP_ACT_GELU_ERF>()); break;
                case TPMLP_ACT_GELU_SIGMOID: apply(std::integral_constant<int, TPMLP_ACT_GELU_SIGMOID>()); break;
                default: apply(std::integral_constant<int, TPMLP_ACT_GELU_TANH>()); break;
            }
#pragma unroll
            for (int j = 0; j < A::N; ++j) sum[i][j] += v[j];
            out[i * NT] = A::pack(v);
        }
    }
    if (row < N) ring.drain((N - row + step - 1) / step, &late[turn][ring.group], err, timeout_ns);
    if (a.db[0] == nullptr) return;
    // the groups' sums in their order, through the ring's memory
    float* sums = reinterpret_cast<float*>(ring_memory);
    static_assert(NT * R * A::N * sizeof(float) <= Ring::MOST, "room for a sum a column");
    for (int q = 0; q < Ring::GROUPS; ++q) {
        __syncthreads();
        if (ring.group == q)
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (ring.mine(i))
#pragma unroll
                    for (int j = 0; j < A::N; ++j) {
                        float* at = sums + (ring.t + i * NT) * A::N + j;
                        *at = q > 0 ? *at + sum[i][j] : sum[i][j];
                    }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += TURN_THREADS) a.part[(int64_t)chunk * a.F + c0 + c] = sums[c];
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

// row chunks of the form without turns
int64_t chunks(int64_t N, int64_t F) {
    const int64_t blocks = (F + 1023) / 1024;
    int64_t S = 16LL * 152 / blocks;
    if (S > (N + 7) / 8) S = (N + 7) / 8;
    return S < 1 ? 1 : S > 1024 ? 1024 : S;
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

// Panels of 16-byte accesses, the CTAs of each.
struct Turns {
    int panels, width, chunks;
};
Turns turns_of(int64_t F, int elem_size) {
    Turns t;
    const int elems = 16 / elem_size, ctas = turn_ctas(elem_size) * TURN_SMS;
    t.panels = (int)((F + LONGEST - 1) / LONGEST);
    t.width = (int)((F / elems + t.panels - 1) / t.panels) * elems;
    t.panels = (int)((F + t.width - 1) / t.width);
    t.chunks = ctas / t.panels > 0 ? ctas / t.panels : 1;
    return t;
}

template <typename T>
tpmlp_status dact_turns(int act, DactParams p, cudaStream_t s) {
    int* err = device_error_word();
    if (err == nullptr) return TPMLP_ERR_CUDA;
    LaunchScope ls("linear_dact", s);
    const Turns t = turns_of(p.a.F, (int)sizeof(T));
    p.S = t.chunks;
    const tpmlp_status st = with_group<TURN_THREADS, 64>(t.width, [&](auto nt, auto full) {
        constexpr int NT = decltype(nt)::value;
        // (a last panel may be narrower)
        auto go = [&](auto whole) {
            constexpr bool FULL = decltype(whole)::value;
            using Ring = RowRing<T, 16, 2, TURN_STAGES, TURN_THREADS, NT, FULL>;
            static std::atomic<uint64_t> asked{0};
            if (!allow_smem(dact_turns_kernel<T, NT, FULL>, Ring::MOST, asked)) return TPMLP_ERR_CUDA;
            return launch_smem(dact_turns_kernel<T, NT, FULL>, dim3((unsigned)(t.panels * t.chunks)), TURN_THREADS,
                               Ring::MOST, s, p, act, t.panels, t.width, err, wait_timeout_ns());
        };
        return decltype(full)::value && p.a.F == (int64_t)t.panels * t.width ? go(std::true_type()) : go(std::false_type());
    });
    if (st != TPMLP_OK || p.a.db[0] == nullptr) return st;
    return launch(dact_sums_kernel<T>, dim3((unsigned)((p.a.F + 31) / 32)), 256, s, p);
}

}  // namespace

size_t dact_part_bytes(int64_t N, int64_t F) {
    int64_t S = chunks(N, F);
    for (int elem_size = 2; elem_size <= 4; elem_size += 2) {
        const int64_t t = turns_of(F, elem_size).chunks;
        if (t > S) S = t;
    }
    return ((size_t)S * (size_t)F * sizeof(float) + 255) & ~(size_t)255;
}

tpmlp_status run_dact(int f32, int act, const DactArgs& a, cudaStream_t s) {
    const DactParams p{a, (int)chunks(a.N, a.F), row_stall()};
    const int elems = f32 ? 4 : 8, size = f32 ? 4 : 2;
    const bool wide = a.F % elems == 0 && access_fits(a.dY, a.lddy * size, 16) && access_fits(a.Z, a.ldz * size, 16) &&
                      access_fits(a.dZ, a.F * size, 16);   // on the bf16 path always
    // Rows in turn from ten million elements on, four rows a group of bf16 (with the
    // launch of the sums; bf16 of F = 16384: 305 rows 14.6 us against 15.1 by columns, 610
    // 19.4 against 20.1, 1220 29.2 against 32.7, 2441 48.3 against 58.0; the worst, F =
    // 8192, 1220 rows 20.8 against 18.7. fp32 of F = 8192: 610 rows 18.5 against 17.0,
    // 1220 26.7 against 30.0, 2441 46.7 against 52.8, 8178 144 against 145).
    if (wide && !a.rest && a.N * a.F >= 8LL * TURN_SMS * LONGEST)
        return f32 ? dact_turns<float>(act, p, s) : dact_turns<__nv_bfloat16>(act, p, s);
    if (!f32) return dact<__nv_bfloat16, 16>(act, p, s);
    return wide ? dact<float, 16>(act, p, s) : dact<float, 4>(act, p, s);
}

}  // namespace tpmlp
