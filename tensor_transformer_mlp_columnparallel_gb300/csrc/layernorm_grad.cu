// Gradients of the layer norm over rows.
//
//   h = (x - mean) rstd,  u = dy w
//   dx = rstd (u - sum u / D - h (sum u h) / D) + dresidual
//   dw = sum_n dy h,  db = sum_n dy
//
// Memory bounds it: dy, x and dresidual are read once, dx is written once.
#include <cuda_bf16.h>

#include "row_sums.cuh"

namespace tpmlp {
namespace {

constexpr int GRAD_THREADS = 512;   // of a CTA that takes rows in turn
constexpr int MOST_CTAS = 152;      // of those: one an SM
template <typename T> constexpr int GRAD_STAGES = sizeof(T) == 2 ? 4 : 2;   // 192 KB

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
    float4* rows;           // [N]: sum u / D, sum u h / D, d rstd (long rows)
    float* part;            // [S, 2, D]: a CTA's (long rows: a row chunk's) sums of dy h and dy
    int S;
    int panels, width;      // of a long row's columns
    int* err;
    uint64_t timeout_ns;
    int stall;
};

// Up to this many deviations a row's fp32 mean is near enough for h (it is off by
// 2^-24 of itself at most, 4.8e-7 of a deviation); beyond, d is taken.
constexpr float FAR_MEAN = 8.f;

__device__ __forceinline__ void write_param(float* at, float v) { *at = v; }
__device__ __forceinline__ void write_param(__nv_bfloat16* at, float v) { *at = __float2bfloat16_rn(v); }

// All of it in one reading, for rows of up to LONGEST elements (PANEL: the second
// reading of longer ones, a CTA having an even share of the columns): a thread
// keeps its columns' sums of dy h and dy over the rows of its group; a CTA's
// sums go to part[blockIdx.x] (with one CTA to dw and db). (8192 x 8192 bf16 with dresidual on
// GB300: 87 us with the launch that adds the CTAs' sums, 6.2 TB/s read and written;
// without its reductions or its column sums the same: HBM. Without dresidual 75 us,
// 5.4 TB/s; rows that leave threads idle wait for one row's reductions, with one group
// an SM from 4097 elements on: 13107 x 5120 96 us, 4.2 TB/s; 112 if the idle accesses
// pass through the arithmetic as zeros.)
template <typename T, typename W, int B, int NT, bool FULL, bool RES, bool PANEL>
__global__ void __launch_bounds__(GRAD_THREADS, 1) norm_grad_kernel(const NormGradArgs a) {
    constexpr int Q = RES ? 3 : 2, STAGES = GRAD_STAGES<T>;
    using Ring = RowRing<T, B, Q, STAGES, GRAD_THREADS, NT, FULL>;
    using A = typename Ring::A;
    using Word = typename Ring::Word;
    using Pair = typename A::Pair;
    constexpr int R = Ring::R, P = A::PAIRS;
    extern __shared__ __align__(16) uint4 ring_memory[];
    __shared__ uint64_t bars[Ring::GROUPS * STAGES];
    __shared__ float red[2][GRAD_THREADS / 32][3];
    __shared__ uint64_t spare[Ring::GROUPS];
    __shared__ int late[2][Ring::GROUPS];
    const int64_t c0 = PANEL ? (int64_t)(blockIdx.x % a.panels) * a.width : 0;
    const int chunk = PANEL ? blockIdx.x / a.panels : blockIdx.x;
    const int cols = (int)(PANEL && a.D - c0 > a.width ? a.width : a.D - c0);
    if (threadIdx.x < 2 * Ring::GROUPS) (&late[0][0])[threadIdx.x] = 0;
    __syncthreads();
    Ring ring(ring_memory, bars, cols);
    constexpr int groups = Ring::GROUPS;
    const int group = ring.group, t = ring.t;
    const uint32_t N = (uint32_t)a.N, step = a.S * groups, first = chunk * groups + group;
    pdl_wait();
    pdl_launch_dependents();
    auto ask = [&](int s, uint32_t row) {
        ring.ask(s, row < N, [&](int to) {
            ring.fetch(to, 0, static_cast<const T*>(a.x) + c0, row, a.ldx);
            ring.fetch(to, 1, static_cast<const T*>(a.dy) + c0, row, a.lddy);
            if (RES) ring.fetch(to, Q - 1, static_cast<const T*>(a.dres) + c0, row, a.lddres);
        });
    };
#pragma unroll
    for (int s = 0; s < STAGES; ++s) ask(s, first + s * step);
    Pair w[R][P], sw[R][P], sb[R][P];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int j = 0; j < P; ++j) w[i][j] = A::both(1.f), sw[i][j] = sb[i][j] = A::both(0.f);
        if (a.w && ring.mine(i)) load_params<W, A::N>(static_cast<const W*>(a.w) + c0 + (t + i * NT) * A::N, w[i]);
    }
    const float inv = 1.f / (float)a.D;
    float m_next = 0.f, r_next = 0.f;
    float4 s_next = make_float4(0.f, 0.f, 0.f, 0.f);
    if (first < N) {
        m_next = a.mean[first], r_next = a.rstd[first];
        if (PANEL) s_next = a.rows[first];
    }
    int turn = 0;
    uint32_t row = first;
    const bool go = !a.stall || ring.stall(&spare[ring.group], &late[0][ring.group], a.err, a.timeout_ns);
    for (; go && row < N; row += step, turn ^= 1, ring.next()) {
        const float m1 = m_next, r1 = r_next;
        const float4 s1 = s_next;
        if (row + step < N) {
            m_next = a.mean[row + step], r_next = a.rstd[row + step];
            if (PANEL) s_next = a.rows[row + step];
        }
        volatile int* flag = &late[turn][group];
        const bool ok = ring.wait(flag, a.err, a.timeout_ns);
        const Pair m = A::both(-m1), r = A::both(r1);
        Word x[R], g[R];
        Pair su = A::both(0.f), suh = su, sh = su;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (!ring.mine(i)) continue;
            x[i] = ring.at(0, i);
            g[i] = ring.at(1, i);
            if (PANEL) continue;
            Pair v[P], y[P];
            A::unpack(x[i], v);
            A::unpack(g[i], y);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const Pair h = mul2(add2(v[j], m), r), u = mul2(y[j], w[i][j]);
                su = add2(su, u);
                suh = fma2(u, h, suh);
                sh = add2(sh, h);
            }
        }
        float s[3] = {A::total(su), A::total(suh), A::total(sh)};
        if constexpr (PANEL) group_sync<NT>(group);
        else group_reduce<NT>(s, group, red[turn], Add());
        if (!ok || (NT > 32 && *flag)) break;   // the whole group
        if (!RES) ask(ring.k, row + STAGES * step);   // every thread holds its elements
        const float d = PANEL ? s1.z : fabsf(m1 * r1) > FAR_MEAN ? s[2] * inv : 0.f;
        // dx = r u - r mean(u) - r mean(u h) h
        const Pair d1 = A::both(-d), c1 = A::both(-r1 * (PANEL ? s1.x : s[0] * inv));
        const Pair c2 = A::both(-r1 * (PANEL ? s1.y : fmaf(-d, s[0], s[1]) * inv));
        Word* out = reinterpret_cast<Word*>(static_cast<T*>(a.dx) + (int64_t)row * a.lddx + c0) + t;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (!ring.mine(i)) continue;
            Pair v[P], y[P], z[P > 1 ? P : 2];
            A::unpack(x[i], v);
            A::unpack(g[i], y);
            if (RES) A::unpack(ring.at(Q - 1, i), *reinterpret_cast<Pair(*)[P]>(&z));
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const Pair h = fma2(add2(v[j], m), r, d1);
                sw[i][j] = fma2(y[j], h, sw[i][j]);
                sb[i][j] = add2(sb[i][j], y[j]);
                v[j] = fma2(mul2(y[j], w[i][j]), r, fma2(h, c2, RES ? add2(z[j], c1) : c1));
            }
            out[i * NT] = A::pack(v);
        }
        if (RES) {
            if (Ring::BULK) group_sync<NT>(group);
            ask(ring.k, row + STAGES * step);
        }
    }
    if (row < N) ring.drain((N - row + step - 1) / step, &late[turn][group], a.err, a.timeout_ns);
    if (a.dw == nullptr) return;
    // the groups' sums in their order, through the ring's memory
    float* sums = reinterpret_cast<float*>(ring_memory);
    static_assert(2 * NT * R * A::N * sizeof(float) <= Ring::MOST, "room for two sums a column");
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (int q = 0; q < groups; ++q) {
        __syncthreads();
        if (group == q)
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (ring.mine(i))
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        Pair* gw = reinterpret_cast<Pair*>(sums + (t + i * NT) * A::N) + j;
                        Pair* gb = reinterpret_cast<Pair*>(sums + NT * R * A::N + (t + i * NT) * A::N) + j;
                        *gw = q > 0 ? add2(*gw, sw[i][j]) : sw[i][j];
                        *gb = q > 0 ? add2(*gb, sb[i][j]) : sb[i][j];
                    }
    }
    __syncthreads();
    float* part = a.part + (int64_t)chunk * 2 * a.D + c0;
    for (int c = threadIdx.x; c < cols; c += GRAD_THREADS) {
        const float gw = sums[c], gb = sums[NT * R * A::N + c];
        if (PANEL || a.S > 1) {
            part[c] = gw;
            part[a.D + c] = gb;
        } else {
            write_param(static_cast<W*>(a.dw) + c, gw);
            write_param(static_cast<W*>(a.db) + c, gb);
        }
    }
}

// Rows longer than LONGEST are read twice: their columns' sums do not fit the
// registers of a CTA. (5461 x 12288 bf16: 132 us, 3.0 TB/s of one reading; 256 threads
// by two accesses at once, 512 threads 140 to 150, more accesses 137. Shorter rows
// read twice: 8192 x 8192 152 us against 75, 1 x 512 4.8 us against 3.9.) Sums over a
// row, one CTA each:
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
    group_reduce<256>(s, 0, red, Add());
    const float d = fabsf(m * r) > FAR_MEAN ? s[2] * inv : 0.f;
    if (threadIdx.x == 0) a.rows[row] = make_float4(s[0] * inv, fmaf(-d, s[0], s[1]) * inv, d, 0.f);
}

// dx, and a row chunk's column sums: a thread has one access's columns. For fewer
// rows than norm_grad_kernel's rings are worth, and for rows of 4- and 2-byte accesses.
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
        write_param(static_cast<W*>(c < a.D ? a.dw : a.db) + (c < a.D ? c : c - a.D), s);
    }
}

// Row chunks of the column sums: enough CTAs to occupy the SMs some eight
// times over, at least four rows each.
int64_t row_chunks(int64_t N, int64_t D) {
    const int64_t blocks = (D + 1023) / 1024;
    int64_t S = 8LL * 152 / blocks;
    if (S > (N + 3) / 4) S = (N + 3) / 4;
    return S < 1 ? 1 : S > 1024 ? 1024 : S;
}

template <typename T, typename W, int B, int NT, bool FULL, bool RES, bool PANEL>
tpmlp_status backward_turns(NormGradArgs& a, cudaStream_t s) {
    using Ring = RowRing<T, B, RES ? 3 : 2, GRAD_STAGES<T>, GRAD_THREADS, NT, FULL>;
    static std::atomic<uint64_t> asked{0};
    if (!allow_smem(norm_grad_kernel<T, W, B, NT, FULL, RES, PANEL>, Ring::MOST, asked)) return TPMLP_ERR_CUDA;
    const int64_t turns = (a.N + Ring::GROUPS - 1) / Ring::GROUPS;
    const int panels = PANEL ? a.panels : 1, most = MOST_CTAS / panels > 0 ? MOST_CTAS / panels : 1;
    a.S = (int)(turns < most ? turns : most);
    return launch_smem(norm_grad_kernel<T, W, B, NT, FULL, RES, PANEL>, dim3((unsigned)(a.S * panels)), GRAD_THREADS,
                       Ring::MOST, s, a);
}

template <typename T, typename W, int B>
tpmlp_status backward(NormGradArgs a, cudaStream_t s) {
    LaunchScope ls("layernorm_backward", s);
    const int64_t accesses = a.D / (B / (int)sizeof(T));
    if (a.D <= LONGEST) {
        const tpmlp_status st = with_group<GRAD_THREADS, 32>(a.D, [&](auto nt, auto full) {
            constexpr int NT = decltype(nt)::value;
            constexpr bool FULL = decltype(full)::value && B == 16;
            return a.dres != nullptr ? backward_turns<T, W, B, NT, FULL, true, false>(a, s)
                                     : backward_turns<T, W, B, NT, FULL, false, false>(a, s);
        });
        if (st != TPMLP_OK || a.part == nullptr || a.S == 1) return st;
        return launch(norm_grad_params_kernel<W>, dim3((unsigned)((2 * a.D + 31) / 32)), 256, s, a);
    }
    tpmlp_status st = launch(norm_grad_rows_kernel<T, W, B>, dim3((unsigned)a.N), 256, s, a);
    if (st != TPMLP_OK) return st;
    // the second reading by panels in turn, from eight rows of a panel a CTA on (900 x
    // 12288 bf16 26 us in all against 34, 5461 x 12288 132 against 151)
    if constexpr (B == 16)
        if (a.N * a.D >= 8LL * MOST_CTAS * LONGEST) {
            constexpr int N = 16 / (int)sizeof(T);
            a.panels = (int)((a.D + LONGEST - 1) / LONGEST);   // of more than LONGEST / 2 columns
            a.width = (int)((a.D / N + a.panels - 1) / a.panels) * N;
            a.panels = (int)((a.D + a.width - 1) / a.width);
            const bool full = a.D == (int64_t)a.panels * LONGEST, res = a.dres != nullptr;
            st = full ? res ? backward_turns<T, W, B, GRAD_THREADS, true, true, true>(a, s)
                            : backward_turns<T, W, B, GRAD_THREADS, true, false, true>(a, s)
                      : res ? backward_turns<T, W, B, GRAD_THREADS, false, true, true>(a, s)
                            : backward_turns<T, W, B, GRAD_THREADS, false, false, true>(a, s);
            if (st != TPMLP_OK || a.part == nullptr) return st;
            return launch(norm_grad_params_kernel<W>, dim3((unsigned)((2 * a.D + 31) / 32)), 256, s, a);
        }
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

size_t layernorm_backward_bytes(int64_t N, int64_t D) {
    if (N == 0) return 0;
    const int64_t chunks = row_chunks(N, D), S = chunks > MOST_CTAS ? chunks : MOST_CTAS;
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
                   g.dx, g.lddx, g.dweight, g.dbias, nullptr, nullptr, (int)row_chunks(g.N, g.D), 1, 0,
                   device_error_word(), wait_timeout_ns(), row_stall()};
    if (a.err == nullptr) return TPMLP_ERR_CUDA;
    a.rows = static_cast<float4*>(workspace);
    if (params) a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + rows_bytes(g.N));
    if (f32) return backward_width<float, float>(a, s);
    return params_f32 ? backward_width<__nv_bfloat16, float>(a, s)
                      : backward_width<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace tpmlp
