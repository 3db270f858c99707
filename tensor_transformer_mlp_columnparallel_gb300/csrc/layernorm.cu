// Layer norm over rows.
//
//   mean = sum x / D,  var = sum (x - mean)^2 / D,  rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd w + b
//
// Memory bounds it: a row's elements are read once and written once. The
// variance is taken around the row's own mean (a second pass over the elements
// a thread holds), never as a difference of squares. The fp32 mean m of a row
// far from zero is off by its sum's rounding, which is not small next to the
// row's spread; what it is off by, d = sum (x - m) / D, is known to many digits
// (x - m is exact where x and m are near), so such a row takes (x - m) - d. A row
// whose mean is within its spread takes d = 0: its m is better than such a d,
// which would hold m's own digits cut to those of x (bf16 rows around zero, the
// mean's relative error 2e-6 instead of 4e-8).
#include <cuda_bf16.h>

#include "row_sums.cuh"

namespace tpmlp {
namespace {

constexpr int HELD_WORDS = 32;   // 32-bit registers of a row that a thread of layernorm_kernel holds
constexpr int WIDEST = 1024;     // threads of the widest row

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
    int* err;
    uint64_t timeout_ns;
    int stall;       // failure-detection self test
};

// 16-byte aligned, whole 16-byte words
__device__ __forceinline__ void bulk_prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// A row's statistics: the row, times scale (1 but for rows whose squares
// overflow, which the caller's rescale has multiplied by 2^-100), has mean m + d,
// variance var around m and reciprocal deviation r; rstd is the row's own.
struct RowStats {
    float scale, m, d, r, rstd, var;
    // from the variance around m + d
    __device__ __forceinline__ void deviation(float left, float eps) {
        r = 1.f / sqrtf(fmaf(eps * scale, scale, left));
        rstd = r * scale;
        if (scale != 1.f && left == 0.f) {   // equal elements, and eps has underflowed beside them
            rstd = 1.f / sqrtf(eps);
            r = eps > 0.f ? 0.f : rstd;      // their distances from the mean are 0
        }
    }
    __device__ __forceinline__ void write(const NormArgs& a, int64_t row) const {
        if (a.mean) a.mean[row] = (m + d) / scale;
        if (a.rstd) a.rstd[row] = rstd;
    }
};

// Where the warps put their parts of the sums.
struct Red {
    float sum[WIDEST / 32][1], spread[WIDEST / 32][2], most[WIDEST / 32][1];
};

// sum(): over the elements that this thread looks after; spread(m, v): of their
// distances from m (v[0]) and those squared (v[1]). Returns false, the same for every
// thread of the row, for a row that takes another look: its squares overflow (or a NaN
// or an infinity is in it), or its spread is no larger than what m is off by, so that
// var - d d cancels (equal elements, or all but equal, far from zero: any row whose
// eps and spread are together below a third of d d).
template <int NT, typename Sum, typename Spread>
__device__ __forceinline__ bool row_stats(RowStats& s, int64_t D, float eps, int group, Red& red, Sum sum, Spread spread) {
    const float inv = 1.f / (float)D;
    float c[1] = {sum()}, v[2] = {0.f, 0.f};
    group_reduce<NT>(c, group, red.sum, Add());
    s.m = c[0] * inv;
    spread(s.m, v);
    group_reduce<NT>(v, group, red.spread, Add());
    s.var = v[1] * inv;
    s.d = s.m * s.m > s.var ? v[0] * inv : 0.f;
    const float left = max_nan(fmaf(-s.d, s.d, s.var), 0.f);
    s.deviation(left, eps);
    return s.var < INFINITY && !(fmaf(eps * s.scale, s.scale, left) < 0.75f * s.var);
}

// A row of any length, read three times (from L2 but for the first) by NT threads,
// one access of B bytes at a time. Finite elements whose squares overflow are
// taken times 2^-100; where m's rounding hides the spread, d is taken again from the
// distances to m + d, each time to another 2^-20 or so of itself, so that equal
// elements end with a spread of exactly 0 (x - m is exact near m).
template <typename T, typename W, int B, int NT, int UNROLL>
__device__ __forceinline__ void long_row(const NormArgs& a, int64_t row, int t, int group, Red& red) {
    using A = Access<T, B>;
    using Word = typename A::Word;
    const int64_t accesses = a.D / A::N;
    const Word* x = reinterpret_cast<const Word*>(static_cast<const T*>(a.x) + row * a.ldx);
    Word* y = reinterpret_cast<Word*>(static_cast<T*>(a.y) + row * a.ldy);
    RowStats s{1.f};
    auto each = [&](auto f) {
#pragma unroll UNROLL
        for (int64_t at = t; at < accesses; at += NT) {
            float v[A::N];
            A::unpack(x[at], v);
#pragma unroll
            for (int j = 0; j < A::N; ++j) f(v[j] * s.scale);
        }
    };
    auto take = [&] {
        return row_stats<NT>(
            s, a.D, a.eps, group, red,
            [&] {
                float c = 0.f;
                each([&](float v) { c += v; });
                return c;
            },
            [&](float m, float (&v)[2]) {
                each([&](float e) {
                    v[0] += e - m;
                    v[1] = fmaf(e - m, e - m, v[1]);
                });
            });
    };
    bool fine = take();
    if (!(s.var < INFINITY)) {
        float big[1] = {0.f};
        each([&](float v) { big[0] = max_nan(big[0], fabsf(v)); });
        group_reduce<NT>(big, group, red.most, Max());
        fine = !(big[0] < INFINITY);   // not finite: nothing to look at
        if (!fine) {
            s.scale = 0x1p-100f;
            fine = take();
        }
    }
    const float inv = 1.f / (float)a.D;
    for (int looks = 0; !fine && looks < 4; ++looks) {
        float v[2] = {0.f, 0.f};
        each([&](float e) {
            const float u = (e - s.m) - s.d;
            v[0] += u;
            v[1] = fmaf(u, u, v[1]);
        });
        group_sync<NT>(group);   // red.spread is read
        group_reduce<NT>(v, group, red.spread, Add());
        const float c = v[0] * inv, var = v[1] * inv;
        s.d += c;
        s.deviation(max_nan(fmaf(-c, c, var), 0.f), a.eps);
        fine = c * c <= 0.25f * var;   // what d was off by is within the spread
    }
#pragma unroll 1
    for (int64_t at = t; at < accesses; at += NT) {
        float v[A::N], w[A::N], b[A::N];
        A::unpack(x[at], v);
        if (a.w) load_params<W, A::N>(static_cast<const W*>(a.w) + at * A::N, w);
        if (a.b) load_params<W, A::N>(static_cast<const W*>(a.b) + at * A::N, b);
#pragma unroll
        for (int j = 0; j < A::N; ++j)
            v[j] = fmaf(((v[j] * s.scale - s.m) - s.d) * s.r, a.w ? w[j] : 1.f, a.b ? b[j] : 0.f);
        y[at] = A::pack(v);
    }
    if (t == 0) s.write(a, row);
    group_sync<NT>(group);   // red is read
}

// The same for a row among others that takes another look: not inlined there, one
// access of 4 bytes at a time (its registers are the other rows' too: 4096 x 16384
// bf16 48.6 us with 16-byte accesses, 43.8), and the arguments by value (by address,
// they are read again after every barrier: 58 us against 44 for 8192 rows of 8192 bf16).
template <typename T, typename W, int B, int NT>
__device__ __noinline__ void huge_row(const NormArgs a, int64_t row, int t, int group, Red* red) {
    long_row<T, W, B < 4 ? B : 4, NT, 1>(a, row, t, group, *red);
}

template <typename T, typename W, int B>
__global__ void __launch_bounds__(WIDEST) layernorm_long_kernel(const NormArgs a) {
    __shared__ Red red;
    pdl_wait();
    pdl_launch_dependents();
    long_row<T, W, B, WIDEST, 4>(a, blockIdx.x, threadIdx.x, 0, red);
}

// The row in the registers of NT threads, R accesses of B bytes each (groups of up
// to a warp: 128 threads to a CTA; a larger group is a CTA, whose one barrier the
// compiler knows: two groups of 64 in a CTA took 53 us where one takes 42). What
// hides one row's two reductions is the other rows of the SM. 8192 x 8192 bf16 with
// bf16 parameters on GB300: 42.4 us, 6.3 TB/s read and written, 0.93 of a copy's
// rate; fp32 rows of 1024 to 8192 elements 6.4 to 6.6.
// EARLY: the parameters too, from the start, for few rows, whose time is one row's
// latency. Else they are read when the row's statistics are known, from L1 or L2;
// where a step has driven them out, all of the first rows would wait for memory
// there: the first CTA has them brought to L2 ahead of its own row (8192 x 8192
// bf16, 43.2 us against 44.8; with fp32 parameters 48.7 against 51.5).
template <typename T, typename W, int B, int NT, int R, bool EARLY>
__global__ void __launch_bounds__(NT > 32 ? NT : 128) layernorm_kernel(const NormArgs a) {
    using A = Access<T, B>;
    using Word = typename A::Word;
    using Pair = typename A::Pair;
    constexpr int P = A::PAIRS;
    constexpr int GROUPS = NT > 32 ? 1 : 128 / NT;
    __shared__ Red red;
    if (!EARLY && B >= 8 && blockIdx.x == 0 && threadIdx.x == 0) {
        const uint32_t bytes = (uint32_t)(a.D * sizeof(W));   // of whole 16-byte words
        if (a.w) bulk_prefetch_l2(a.w, bytes);
        if (a.b) bulk_prefetch_l2(a.b, bytes);
    }
    pdl_wait();
    pdl_launch_dependents();
    const int group = GROUPS > 1 ? threadIdx.x / NT : 0, t = threadIdx.x % NT;
    const int64_t row = (int64_t)blockIdx.x * GROUPS + group;
    if (row >= a.N) return;   // a whole group
    const int accesses = (int)(a.D / A::N);
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (t + i * NT < accesses) f(i);
    };
    const Word* x = reinterpret_cast<const Word*>(static_cast<const T*>(a.x) + row * a.ldx) + t;
    const W* pw = static_cast<const W*>(a.w) + t * A::N;
    const W* pb = static_cast<const W*>(a.b) + t * A::N;
    auto params = [&](int i, Pair (&u)[P], Pair (&v)[P]) {
#pragma unroll
        for (int j = 0; j < P; ++j) u[j] = A::both(1.f), v[j] = A::both(0.f);
        if (a.w) load_params<W, A::N>(pw + i * NT * A::N, u);
        if (a.b) load_params<W, A::N>(pb + i * NT * A::N, v);
    };
    Word held[R];
    Pair w[EARLY ? R : 1][P], b[EARLY ? R : 1][P];
    each([&](int i) { held[i] = x[i * NT]; });
    if constexpr (EARLY) each([&](int i) { params(i, w[i], b[i]); });
    RowStats s{1.f};
    const bool fine = row_stats<NT>(
        s, a.D, a.eps, group, red,
        [&] {
            Pair c = A::both(0.f);
            each([&](int i) {
                Pair v[P];
                A::unpack(held[i], v);
#pragma unroll
                for (int j = 0; j < P; ++j) c = add2(c, v[j]);
            });
            return A::total(c);
        },
        [&](float m, float (&sums)[2]) {
            Pair c = A::both(0.f), q = c;
            each([&](int i) {
                Pair v[P];
                A::unpack(held[i], v);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const Pair u = add2(v[j], A::both(-m));
                    c = add2(c, u);
                    q = fma2(u, u, q);
                }
            });
            sums[0] = A::total(c), sums[1] = A::total(q);
        });
    if (!fine) {   // the same for every thread of the row
        group_sync<NT>(group);
        huge_row<T, W, B, NT>(a, row, t, group, &red);
        return;
    }
    Word* y = reinterpret_cast<Word*>(static_cast<T*>(a.y) + row * a.ldy) + t;
    const Pair m = A::both(-s.m), r = A::both(s.r), dr = A::both(-s.d * s.r);
    each([&](int i) {
        const int k = EARLY ? i : 0;
        if constexpr (!EARLY) params(i, w[0], b[0]);
        Pair v[P];
        A::unpack(held[i], v);
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = fma2(fma2(add2(v[j], m), r, dr), w[k][j], b[k][j]);
        y[i * NT] = A::pack(v);
    });
    if (t == 0) s.write(a, row);
}

// --------------------------------------------------------- rows in turn --

constexpr int NORM_THREADS = 256, NORM_STAGES = 6;   // 96 KB of bf16 rows a CTA, two CTAs an SM

// Rows of 16-byte accesses, a CTA to a row, its columns' parameters in registers,
// for bf16 rows with fp32 parameters, whose 64 bytes of parameters to 16 of x the
// form above reads again for every row. 8192 x 8192 on GB300: 43.8 us, 6.1 TB/s.
template <typename T, typename W, bool FULL>
__global__ void __launch_bounds__(NORM_THREADS, 2) layernorm_turns_kernel(const NormArgs a) {
    constexpr int NT = NORM_THREADS, STAGES = NORM_STAGES;
    using Ring = RowRing<T, 16, 1, STAGES, NT, NT, FULL>;
    using A = typename Ring::A;
    using Word = typename Ring::Word;
    using Pair = typename A::Pair;
    constexpr int R = Ring::R, P = A::PAIRS;
    extern __shared__ __align__(16) uint4 ring_memory[];
    __shared__ uint64_t bars[STAGES], spare;
    __shared__ Red red;
    __shared__ int late[2];   // a wait of this turn ran out
    if (threadIdx.x < 2) late[threadIdx.x] = 0;
    __syncthreads();
    Ring ring(ring_memory, bars, a.D);
    const uint32_t N = (uint32_t)a.N, step = gridDim.x, first = blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    auto ask = [&](int s, uint32_t row) {
        ring.ask(s, row < N, [&](int to) { ring.fetch(to, 0, a.x, row, a.ldx); });
    };
#pragma unroll
    for (int s = 0; s < STAGES; ++s) ask(s, first + s * step);
    Pair w[R][P], b[R][P];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int j = 0; j < P; ++j) w[i][j] = A::both(1.f), b[i][j] = A::both(0.f);
        if (a.w && ring.mine(i)) load_params<W, A::N>(static_cast<const W*>(a.w) + (ring.t + i * NT) * A::N, w[i]);
        if (a.b && ring.mine(i)) load_params<W, A::N>(static_cast<const W*>(a.b) + (ring.t + i * NT) * A::N, b[i]);
    }
    int turn = 0;
    uint32_t row = first;
    const bool go = !a.stall || ring.stall(&spare, &late[0], a.err, a.timeout_ns);
    for (; go && row < N; row += step, turn ^= 1, ring.next()) {
        volatile int* flag = &late[turn];
        const bool ok = ring.wait(flag, a.err, a.timeout_ns);
        Word held[R];
#pragma unroll
        for (int i = 0; i < R; ++i) held[i] = ring.at(0, i);
        RowStats s{1.f};
        const bool fine = row_stats<NT>(
            s, a.D, a.eps, 0, red,
            [&] {
                Pair c = A::both(0.f);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    Pair v[P];
                    A::unpack(held[i], v);
#pragma unroll
                    for (int j = 0; j < P; ++j) c = add2(c, v[j]);
                }
                return A::total(c);
            },
            [&](float m, float (&sums)[2]) {
                Pair c = A::both(0.f), q = c;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    Pair v[P];
                    A::unpack(held[i], v);
                    const Pair less = A::both(ring.mine(i) ? -m : 0.f);
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const Pair u = add2(v[j], less);
                        c = add2(c, u);
                        q = fma2(u, u, q);
                    }
                }
                sums[0] = A::total(c), sums[1] = A::total(q);
            });
        if (!ok || *flag) break;   // the whole group
        ask(ring.k, row + STAGES * step);   // every thread holds its elements
        if (!fine) {
            group_sync<NT>(0);   // red is read
            huge_row<T, W, 16, NT>(a, row, ring.t, 0, &red);
            continue;
        }
        Word* y = reinterpret_cast<Word*>(static_cast<T*>(a.y) + (int64_t)row * a.ldy) + ring.t;
        const Pair m = A::both(-s.m), r = A::both(s.r), dr = A::both(-s.d * s.r);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            Pair v[P];
            A::unpack(held[i], v);
#pragma unroll
            for (int j = 0; j < P; ++j) v[j] = fma2(fma2(add2(v[j], m), r, dr), w[i][j], b[i][j]);
            const Word out = A::pack(v);
            if (ring.mine(i)) y[i * NT] = out;
        }
        if (ring.t == 0) s.write(a, row);
    }
    if (row < N) ring.drain((N - row + step - 1) / step, &late[turn], a.err, a.timeout_ns);
}

template <int N> using Int = std::integral_constant<int, N>;

template <typename T, typename W, int B>
tpmlp_status forward(const NormArgs& a, bool turns, cudaStream_t s) {
    constexpr int R = B >= 4 ? HELD_WORDS * 4 / B : HELD_WORDS;
    const int64_t accesses = a.D / (B / (int)sizeof(T));
    LaunchScope ls("layernorm", s);
    tpmlp_status st = TPMLP_OK;
    // NT threads to a row, `eighths` of R accesses to each, if that is enough. Most
    // rows want as much of a row a thread as its registers hold (16384 x 4096 bf16:
    // eight accesses 42 us, four 52), and no idle ones (13107 x 5120: six 44 us, eight
    // 47; 524288 x 128: two 49, eight 71).
    auto held = [&](auto nt, auto eighths, auto early) {
        constexpr int NT = decltype(nt)::value, MOST = R * decltype(eighths)::value / 8;
        constexpr int GROUPS = NT > 32 ? 1 : 128 / NT;
        if (accesses > NT * MOST) return false;
        st = launch(layernorm_kernel<T, W, B, NT, MOST, decltype(early)::value>,
                    dim3((unsigned)((a.N + GROUPS - 1) / GROUPS)), NT * GROUPS, s, a);
        return true;
    };
    const std::false_type late;
    if constexpr (sizeof(W) > sizeof(T) && B >= 8)
        if (turns) {
            auto go = [&](auto full) {
                constexpr bool FULL = decltype(full)::value;
                using Ring = RowRing<T, 16, 1, NORM_STAGES, NORM_THREADS, NORM_THREADS, FULL>;
                static std::atomic<uint64_t> asked{0};
                if (!allow_smem(layernorm_turns_kernel<T, W, FULL>, Ring::MOST, asked)) return TPMLP_ERR_CUDA;
                return launch_smem(layernorm_turns_kernel<T, W, FULL>, dim3((unsigned)(2 * device_sm_count())),
                                   NORM_THREADS, Ring::MOST, s, a);
            };
            return a.D == LONGEST ? go(std::true_type()) : go(std::false_type());
        }
    if constexpr (B >= 8) {
        // Few rows: more threads, less each, up to 1024 threads an SM in all (bf16, as
        // above: 304 x 4096 2.7 us against 4.2, 1216 x 1024 2.7 against 4.0; but 1216 x
        // 4096 8.7 against 6.6, 4864 x 1024 7.8 against 6.1).
        auto few = [&](auto nt) {
            return a.N * decltype(nt)::value <= 1024LL * device_sm_count() && held(nt, Int<2>(), std::true_type());
        };
        if (few(Int<32>()) || few(Int<128>()) || few(Int<512>()) || few(Int<1024>())) return st;
        auto threads = [&](auto nt) { return held(nt, Int<6>(), late) || held(nt, Int<8>(), late); };
        if (held(Int<8>(), Int<2>(), late) || held(Int<8>(), Int<4>(), late) || threads(Int<8>()) ||
            threads(Int<16>()) || threads(Int<32>()) || threads(Int<64>()) || threads(Int<128>()) ||
            threads(Int<256>()) || threads(Int<512>()))
            return st;
    } else if (held(Int<32>(), Int<8>(), late) || held(Int<128>(), Int<8>(), late) || held(Int<512>(), Int<8>(), late)) {
        return st;
    }
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
    // bf16 rows with fp32 parameters by 8 bytes, so that a warp's reads of the
    // parameters are whole lines (8192 x 8192: 46 us; by 16 bytes 51)
    constexpr int WIDE = sizeof(W) > sizeof(T) ? 8 : 16;
    // (fp32 parameters only) rows that fill the turns' ring: 9362 x 7168 48.7 us
    // against 50.2 held, 8192 x 8192 43.8 against 48.7, but 10922 x 6144 54.6 against
    // 48.3 (the ring keeps its room, and the threads their work, for 8192 elements); and
    // eight rows a CTA, for the ring's start (2432 x 8192 14.9 us either way).
    const bool turns = a.D <= LONGEST && a.D >= LONGEST / 8 * 7 && a.N >= 16LL * device_sm_count() && fits(16);
    if (fits(WIDE)) return forward<T, W, WIDE>(a, turns, s);
    if constexpr (sizeof(T) == 4) return forward<T, W, 4>(a, false, s);
    else return fits(4) ? forward<T, W, 4>(a, false, s) : forward<T, W, 2>(a, false, s);
}

}  // namespace

tpmlp_status run_layernorm(int f32, int params_f32, const LayernormArgs& g, cudaStream_t s) {
    if (g.N == 0) return TPMLP_OK;
    const NormArgs a{g.N, g.D, g.x, g.ldx, g.weight, g.bias, g.eps, g.y, g.ldy, g.mean, g.rstd,
                     device_error_word(), wait_timeout_ns(), row_stall()};
    if (a.err == nullptr) return TPMLP_ERR_CUDA;
    if (f32) return forward_width<float, float>(a, s);
    return params_f32 ? forward_width<__nv_bfloat16, float>(a, s) : forward_width<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace tpmlp
