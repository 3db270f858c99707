// Embedding lookup times a factor, and the table's gradient by sorted tokens.
//
// Lookup: out[n] = c E[id_n]; a warp per token, one read and one write of the row.
// Gradient: dE[v] = c sum_{n: id_n = v} dout[n]. The tokens are sorted by id
//   (stable, least significant digit first, RADIX_BITS a pass), which gives
//   every table row a contiguous segment of tokens in rising order; each
//   table row is then written once from its segment's fp32 sum. No
//   floating-point atomics, so the bits are the same on every run.
#include <cuda_bf16.h>

#include "act.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return bf2f(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------- lookup --

struct LookupArgs {
    const int64_t* ids;
    const void* table[kMaxG];
    void* out;
    int64_t N, V, Vs, H;
    float scale;
    int* err;
};

template <typename T>
__global__ void __launch_bounds__(256) embedding_scaled_kernel(const LookupArgs p) {
    const int64_t n = blockIdx.x;
    const int64_t id = p.ids[n];
    const bool good = id >= 0 && id < p.V;
    if (!good && threadIdx.x == 0) atomicCAS(p.err, 0, (int)TPMLP_ERR_ARG);
    const int64_t k = good ? id / p.Vs : 0;
    const T* src = good ? static_cast<const T*>(p.table[k]) + (id - k * p.Vs) * p.H : nullptr;
    T* dst = static_cast<T*>(p.out) + n * p.H;
    for (int64_t c = threadIdx.x; c < p.H; c += 256)
        dst[c] = from_f32<T>(good ? p.scale * to_f32(src[c]) : 0.f);
}

// ------------------------------------------------------------------ sort --

constexpr int RADIX_BITS = 9;
constexpr int BINS = 1 << RADIX_BITS;
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ROUNDS = 8;                               // tokens per lane
constexpr int SORT_TILE = SORT_THREADS * SORT_ROUNDS;        // tokens per CTA
static_assert(SORT_THREADS == BINS, "one thread per digit");

struct SortArgs {
    const int64_t* ids;     // first pass: the keys (in token order)
    const uint2* in;        // later passes: (key, token)
    uint2* out;
    int* hist;              // [CTAs][BINS]
    int64_t N, V;
    int shift;
    int* err;
};

// Pair of sorted position i before this pass. An id outside [0, V) gets key V
// and lands behind every row's segment.
__device__ __forceinline__ uint2 sort_item(const SortArgs& p, int64_t i) {
    if (p.ids == nullptr) return p.in[i];
    const int64_t id = p.ids[i];
    return make_uint2(id >= 0 && id < p.V ? (uint32_t)id : (uint32_t)p.V, (uint32_t)i);
}

__global__ void __launch_bounds__(SORT_THREADS) sort_hist_kernel(const SortArgs p) {
    __shared__ int cnt[BINS];
    cnt[threadIdx.x] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * SORT_TILE;
    for (int r = 0; r < SORT_ROUNDS; ++r) {
        const int64_t i = base + r * SORT_THREADS + threadIdx.x;
        if (i >= p.N) break;
        const uint32_t key = sort_item(p, i).x;
        if (p.ids != nullptr && key == (uint32_t)p.V) atomicCAS(p.err, 0, (int)TPMLP_ERR_ARG);
        atomicAdd(&cnt[(key >> p.shift) & (BINS - 1)], 1);
    }
    __syncthreads();
    p.hist[(int64_t)blockIdx.x * BINS + threadIdx.x] = cnt[threadIdx.x];
}

// Stable: a warp takes 32 x SORT_ROUNDS consecutive tokens, 32 at a time; lanes
// with one digit rank themselves by lane (match), behind the warp's count of
// earlier rounds; then warps, CTAs and digits follow in order.
__global__ void __launch_bounds__(SORT_THREADS) sort_scatter_kernel(const SortArgs p) {
    __shared__ int cnt[SORT_WARPS][BINS];
    __shared__ int scan[SORT_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int w = 0; w < SORT_WARPS; ++w) cnt[w][threadIdx.x] = 0;
    // digit threadIdx.x: all its tokens, and those in CTAs before this one
    int total = 0, before = 0;
    for (int b = 0; b < (int)gridDim.x; ++b) {
        const int h = p.hist[(int64_t)b * BINS + threadIdx.x];
        total += h;
        if (b < (int)blockIdx.x) before += h;
    }
    int inc = total;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += x;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int start = inc - total + before;
    for (int w = 0; w < warp; ++w) start += scan[w];

    const int64_t base = (int64_t)blockIdx.x * SORT_TILE + warp * (32 * SORT_ROUNDS);
    uint2 item[SORT_ROUNDS];
    int rank[SORT_ROUNDS];
#pragma unroll
    for (int r = 0; r < SORT_ROUNDS; ++r) {
        const int64_t i = base + r * 32 + lane;
        const bool in = i < p.N;
        item[r] = in ? sort_item(p, i) : make_uint2(0u, 0u);
        const uint32_t digit = in ? (item[r].x >> p.shift) & (BINS - 1) : (uint32_t)BINS;
        const uint32_t peers = __match_any_sync(0xffffffffu, digit);
        const int mine = __popc(peers & ((1u << lane) - 1u));
        const int seen = in ? cnt[warp][digit] : 0;
        rank[r] = seen + mine;
        __syncwarp();
        if (in && mine == 0) cnt[warp][digit] = seen + __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    for (int w = 0; w < SORT_WARPS; ++w) {   // digit threadIdx.x: each warp's first place
        const int c = cnt[w][threadIdx.x];
        cnt[w][threadIdx.x] = start;
        start += c;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < SORT_ROUNDS; ++r) {
        const int64_t i = base + r * 32 + lane;
        if (i < p.N) p.out[cnt[warp][(item[r].x >> p.shift) & (BINS - 1)] + rank[r]] = item[r];
    }
}

// seg[v] = [first, last + 1) of row v's tokens in sorted order ({0, 0}: none)
__global__ void __launch_bounds__(256) segment_kernel(const uint2* sorted, int64_t N, int64_t V, int2* seg) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= N) return;
    const uint32_t key = sorted[i].x;
    if (key >= (uint32_t)V) return;
    if (i == 0 || sorted[i - 1].x != key) seg[key].x = (int)i;
    if (i == N - 1 || sorted[i + 1].x != key) seg[key].y = (int)i + 1;
}

// -------------------------------------------------------------- gradient --

struct GradArgs {
    const uint2* sorted;
    const int2* seg;
    const void* dout;
    void* dtable[kMaxG];
    int64_t V, Vs, H;
    float scale;
    int accumulate;
};

template <typename T, typename GT>
__global__ void __launch_bounds__(256) embedding_grad_kernel(const GradArgs p) {
    const int64_t v = blockIdx.x;
    const int2 sg = p.seg[v];
    if (p.accumulate && sg.y == sg.x) return;
    const int64_t k = v / p.Vs;
    GT* dst = static_cast<GT*>(p.dtable[k]) + (v - k * p.Vs) * p.H;
    for (int64_t c = threadIdx.x; c < p.H; c += 256) {
        float acc = 0.f;
        for (int i = sg.x; i < sg.y; ++i)
            acc += to_f32(static_cast<const T*>(p.dout)[(int64_t)p.sorted[i].y * p.H + c]);
        acc *= p.scale;
        if (p.accumulate) acc += to_f32(dst[c]);
        dst[c] = from_f32<GT>(acc);
    }
}

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline int64_t sort_ctas(int64_t N) { return (N + SORT_TILE - 1) / SORT_TILE; }

// Workspace: two arrays of (key, token) pairs, the digit counts, the segments.
struct GradLayout {
    size_t pairs[2], hist, seg, total;
};
GradLayout grad_layout(int64_t N, int64_t V) {
    GradLayout l;
    size_t o = 0;
    l.pairs[0] = o;
    o += round256((size_t)N * sizeof(uint2));
    l.pairs[1] = o;
    o += round256((size_t)N * sizeof(uint2));
    l.hist = o;
    o += round256((size_t)sort_ctas(N) * BINS * sizeof(int));
    l.seg = o;
    o += round256((size_t)V * sizeof(int2));
    l.total = o;
    return l;
}

}  // namespace

tpmlp_status run_vocab_embedding_scaled(int f32, int64_t N, int64_t V, int64_t H, int T,
                                        const int64_t* ids, const void* const* table, float scale,
                                        void* out, cudaStream_t s) {
    if (N == 0) return TPMLP_OK;
    if (N > 0x7fffffffLL) return TPMLP_ERR_SHAPE;
    LookupArgs p{};
    p.ids = ids;
    for (int k = 0; k < T; ++k) p.table[k] = table[k];
    p.out = out;
    p.N = N;
    p.V = V;
    p.Vs = V / T;
    p.H = H;
    p.scale = scale;
    p.err = device_error_word();
    if (p.err == nullptr) return TPMLP_ERR_CUDA;
    {
        LaunchScope ls("vocab_embedding_scaled", s);
        if (f32)
            embedding_scaled_kernel<float><<<(unsigned)N, 256, 0, s>>>(p);
        else
            embedding_scaled_kernel<__nv_bfloat16><<<(unsigned)N, 256, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

size_t embedding_grad_bytes(int64_t N, int64_t V, int64_t H) {
    (void)H;
    return grad_layout(N, V).total;
}

tpmlp_status run_vocab_embedding_backward(int f32, int grad_f32, int64_t N, int64_t V, int64_t H,
                                          int T, const int64_t* ids, const void* dout, float scale,
                                          int accumulate, void* const* dtable, void* workspace,
                                          cudaStream_t s) {
    const GradLayout l = grad_layout(N, V);
    char* ws = static_cast<char*>(workspace);
    int2* seg = reinterpret_cast<int2*>(ws + l.seg);
    int* err = device_error_word();
    if (err == nullptr) return TPMLP_ERR_CUDA;
    if (N == 0 && accumulate) return TPMLP_OK;
    {
        LaunchScope ls("embedding_grad_sort", s);
        if (cudaMemsetAsync(seg, 0, (size_t)V * sizeof(int2), s) != cudaSuccess) return TPMLP_ERR_CUDA;
    }
    const uint2* sorted = nullptr;
    if (N > 0) {
        int bits = 1;
        while ((V >> bits) != 0) ++bits;   // keys 0..V
        SortArgs p{};
        p.ids = ids;
        p.hist = reinterpret_cast<int*>(ws + l.hist);
        p.N = N;
        p.V = V;
        p.err = err;
        int which = 0;
        for (p.shift = 0; p.shift < bits; p.shift += RADIX_BITS) {
            p.out = reinterpret_cast<uint2*>(ws + l.pairs[which]);
            const unsigned g = (unsigned)sort_ctas(N);
            {
                LaunchScope ls("embedding_grad_sort", s);
                sort_hist_kernel<<<g, SORT_THREADS, 0, s>>>(p);
            }
            {
                LaunchScope ls("embedding_grad_sort", s);
                sort_scatter_kernel<<<g, SORT_THREADS, 0, s>>>(p);
            }
            sorted = p.out;
            p.ids = nullptr;
            p.in = p.out;
            which ^= 1;
        }
        LaunchScope ls("embedding_grad_sort", s);
        segment_kernel<<<(unsigned)((N + 255) / 256), 256, 0, s>>>(sorted, N, V, seg);
    }
    GradArgs g{};
    g.sorted = sorted;
    g.seg = seg;
    g.dout = dout;
    for (int k = 0; k < T; ++k) g.dtable[k] = dtable[k];
    g.V = V;
    g.Vs = V / T;
    g.H = H;
    g.scale = scale;
    g.accumulate = accumulate;
    {
        LaunchScope ls("embedding_grad", s);
        const unsigned grid = (unsigned)V;
        if (f32 && grad_f32)
            embedding_grad_kernel<float, float><<<grid, 256, 0, s>>>(g);
        else if (f32)
            embedding_grad_kernel<float, __nv_bfloat16><<<grid, 256, 0, s>>>(g);
        else if (grad_f32)
            embedding_grad_kernel<__nv_bfloat16, float><<<grid, 256, 0, s>>>(g);
        else
            embedding_grad_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, 256, 0, s>>>(g);
    }
    return cudaGetLastError() == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

}  // namespace tpmlp
