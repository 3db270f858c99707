// Embedding lookup times a factor, and the table's gradient by sorted tokens.
//
// Lookup: out[n] = c E[id_n], one read and one write of the row.
// Gradient: dE[v] = c sum_{n: id_n = v} dout[n]. The tokens are sorted by id
//   (stable, least significant digit first, RADIX_BITS a pass), so every table
//   row has a contiguous segment of sorted positions, in token order. The
//   positions are cut into blocks of SPAN. A segment inside one block is
//   summed by the CTA that writes its table row. A segment that crosses
//   blocks is summed block by block into fp32 pieces (at most two a block: the
//   run that began earlier and the run that goes on), which are then added in
//   order; so a token that fills half the batch is no one CTA's work. Sums
//   are fp32, in an order that the ids alone decide: no floating-point atomics.
//   What bounds it is the table: every row is written once, most as zeros.
//   On GB300, 8192 bf16 tokens into 128000 x 4096 fp32: 338 us, of which the
//   sort takes 10 and the pieces 9; 6.4 TB/s over the whole, 6.9 over the
//   table's launch. A few tokens: three launches, 13 us for a small table.
#include <cuda_bf16.h>

#include "act.cuh"
#include "ptx.cuh"
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

// N consecutive elements moved as one access where N sizeof(T) is a vector
// size (2, 4, 8 or 16 bytes), as two 16-byte ones for 32.
template <typename T, int N>
struct __align__(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Pack {
    T v[N];
};
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T* p) {
    return *reinterpret_cast<const Pack<T, N>*>(p);
}
template <typename T, int N>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, N>& x) {
    constexpr int B = N * sizeof(T);
    if constexpr (B == 16)
        __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&x));
    else if constexpr (B == 8)
        __stcs(reinterpret_cast<uint2*>(p), *reinterpret_cast<const uint2*>(&x));
    else
        *reinterpret_cast<Pack<T, N>*>(p) = x;
}

// ---------------------------------------------------------------- lookup --

struct LookupArgs {
    const int64_t* ids;
    const void* table[kMaxG];
    void* out;
    int64_t N, V, Vs, H;
    int packs;        // packs of a row
    int segs;         // CTAs of a row
    int log_lanes;    // threads of a row within a CTA, as a power of two
    float scale;
    int* err;
};

constexpr int LOOKUP_THREADS = 256;
constexpr int LOOKUP_UNROLL = 4;

// A row is taken by 2^log_lanes threads, LOOKUP_UNROLL packs each, their loads
// in flight together; short rows share a CTA, long ones take several. HBM
// bounds it: 8192 bf16 rows of 8192 in 29 us on GB300, 268 MB asked for, of
// which 131 come from DRAM or go there in that time (the rest stays in L2).
template <typename T, int N>
__global__ void __launch_bounds__(LOOKUP_THREADS) embedding_scaled_kernel(const LookupArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lanes = 1 << p.log_lanes;
    const int64_t group = blockIdx.x / (unsigned)p.segs;
    const int seg = (int)(blockIdx.x - (unsigned)group * (unsigned)p.segs);
    const int64_t n = group * (LOOKUP_THREADS >> p.log_lanes) + ((int)threadIdx.x >> p.log_lanes);
    if (n >= p.N) return;
    const int lane = (int)threadIdx.x & (lanes - 1);
    const int64_t id = p.ids[n];
    const bool good = id >= 0 && id < p.V;
    if (!good && lane == 0 && seg == 0) atomicCAS(p.err, 0, (int)TPMLP_ERR_ARG);
    const uint32_t k = good ? (uint32_t)id / (uint32_t)p.Vs : 0u;
    const T* src = static_cast<const T*>(p.table[k]) + (good ? (id - (int64_t)k * p.Vs) * p.H : 0);
    T* dst = static_cast<T*>(p.out) + n * p.H;
    const int c0 = seg * lanes * LOOKUP_UNROLL + lane;
    Pack<T, N> x[LOOKUP_UNROLL];
#pragma unroll
    for (int u = 0; u < LOOKUP_UNROLL; ++u)
        if (c0 + u * lanes < p.packs) x[u] = load_pack<T, N>(src + (int64_t)(c0 + u * lanes) * N);
#pragma unroll
    for (int u = 0; u < LOOKUP_UNROLL; ++u) {
        if (c0 + u * lanes >= p.packs) break;
#pragma unroll
        for (int j = 0; j < N; ++j) x[u].v[j] = from_f32<T>(good ? p.scale * to_f32(x[u].v[j]) : 0.f);
        store_pack<T, N>(dst + (int64_t)(c0 + u * lanes) * N, x[u]);
    }
}

// ------------------------------------------------------------------ sort --

constexpr int RADIX_BITS = 9;
constexpr int BINS = 1 << RADIX_BITS;
constexpr int SORT_ROUNDS = 8;                               // tokens per lane
constexpr int SORT_THREADS = 512;                            // of the sort over several CTAs
// Its rounds while the CTAs are few: ranking a round takes a warp up to 32 steps,
// one for every digit among its lanes, so more SMs have it sooner, until every
// CTA adds up too many others' counts. (Whole call into 32000 x 512 fp32 on
// GB300, CTAs of 1024 / 4096 tokens: 4096 tokens 26 / 38 us, 16384 39 / 53,
// 65536 77 / 88, 131072 126 / 126, 262144 223 / 210.)
constexpr int FEW_ROUNDS = 2;
constexpr int64_t FEW_TOKENS = 65536;
// The sort in one CTA, for a batch that small: all passes in one launch instead
// of two each. Up to 2048 tokens it was faster for every table (GB300, whole
// call, one CTA / several: 256 tokens into 2000 x 512 fp32 13.0 / 18.0 us, from
// a captured graph 11.7 / 13.0; 1024 into 9999 x 1030 23.4 / 26.4; 2048 into
// 38549 x 1464 54.8 / 55.5). Ranking more tokens on one SM is not: 4099 into
// 9999 x 1030 38.4 / 36.0, 8192 into 2000 x 512 32.1 / 23.9.
constexpr int ONE_THREADS = 1024;
constexpr int ONE_ROUNDS = 2;
constexpr int ONE_MAX = ONE_THREADS * ONE_ROUNDS;            // its tokens at most
constexpr int ONE_SMEM = (ONE_THREADS / 32) * BINS * 4 + ONE_MAX * 8;
static_assert(SORT_THREADS == BINS, "one thread per digit");

struct SortArgs {
    const int64_t* ids;     // first pass: the keys (in token order)
    const uint2* in;        // later passes: (key, token)
    uint2* out;
    int* hist;              // [CTAs][BINS]
    int2* seg;              // zeroed beside the first pass
    int64_t N, V;
    int shift, bits;
    int* err;
};

// Pair of position i before the first pass. An id outside [0, V) gets key V
// and lands behind every row's segment.
__device__ __forceinline__ uint2 first_pair(const SortArgs& p, int64_t i) {
    const int64_t id = p.ids[i];
    const bool good = id >= 0 && id < p.V;
    if (!good) atomicCAS(p.err, 0, (int)TPMLP_ERR_ARG);
    return make_uint2(good ? (uint32_t)id : (uint32_t)p.V, (uint32_t)i);
}
__device__ __forceinline__ uint2 sort_pair(const SortArgs& p, int64_t i) {
    return p.ids == nullptr ? p.in[i] : first_pair(p, i);
}

__device__ __forceinline__ void zero_segments(const SortArgs& p, int first, int ctas) {
    for (int64_t v = (int64_t)(blockIdx.x - first) * blockDim.x + threadIdx.x; v < p.V;
         v += (int64_t)ctas * blockDim.x)
        p.seg[v] = make_int2(0, 0);
}

// Ranks of a warp's 32 x R consecutive pairs within their digits: lanes
// with one digit rank themselves by lane, behind the warp's count so far.
template <int R>
__device__ __forceinline__ void warp_ranks(const uint2 (&item)[R], const bool (&in)[R], int shift, int* cnt,
                                           int (&rank)[R]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t digit = in[r] ? (item[r].x >> shift) & (BINS - 1) : (uint32_t)BINS;
        const uint32_t peers = __match_any_sync(0xffffffffu, digit);
        const int mine = __popc(peers & ((1u << lane) - 1u));
        const int seen = in[r] ? cnt[digit] : 0;
        rank[r] = seen + mine;
        __syncwarp();
        if (in[r] && mine == 0) cnt[digit] = seen + __popc(peers);
        __syncwarp();
    }
}

// Exclusive scan of one value a thread over the first BINS threads.
__device__ __forceinline__ int scan_bins(int x, int* warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
    }
    if (threadIdx.x < BINS && lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int start = inc - x;
    if (threadIdx.x < BINS)
        for (int w = 0; w < warp; ++w) start += warp_sum[w];
    return start;
}

// All passes in one CTA (N <= ONE_MAX), the pairs in registers and exchanged
// through shared memory; the other CTAs zero the segments.
__global__ void __launch_bounds__(ONE_THREADS) sort_one_kernel(const SortArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x > 0) {
        zero_segments(p, 1, (int)gridDim.x - 1);
        return;
    }
    extern __shared__ uint2 exchange[];   // [ONE_MAX], then the warps' counts
    int* cnt = reinterpret_cast<int*>(exchange + ONE_MAX);
    __shared__ int warp_sum[BINS / 32];
    const int warp = threadIdx.x >> 5;
    const int base = warp * 32 * ONE_ROUNDS + (threadIdx.x & 31);
    uint2 item[ONE_ROUNDS];
    bool in[ONE_ROUNDS];
    int rank[ONE_ROUNDS];
#pragma unroll
    for (int r = 0; r < ONE_ROUNDS; ++r) {
        in[r] = base + r * 32 < p.N;
        item[r] = in[r] ? first_pair(p, base + r * 32) : make_uint2(0u, 0u);
    }
    for (int shift = 0; shift < p.bits; shift += RADIX_BITS) {
        for (int i = threadIdx.x; i < (ONE_THREADS / 32) * BINS; i += ONE_THREADS) cnt[i] = 0;
        __syncthreads();
        warp_ranks(item, in, shift, cnt + warp * BINS, rank);
        __syncthreads();
        int total = 0;
        if (threadIdx.x < BINS)
#pragma unroll 8
            for (int w = 0; w < ONE_THREADS / 32; ++w) {   // each warp's first place within the digit
                const int c = cnt[w * BINS + threadIdx.x];
                cnt[w * BINS + threadIdx.x] = total;
                total += c;
            }
        const int start = scan_bins(total, warp_sum);
        if (threadIdx.x < BINS)
#pragma unroll 8
            for (int w = 0; w < ONE_THREADS / 32; ++w) cnt[w * BINS + threadIdx.x] += start;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ONE_ROUNDS; ++r)
            if (in[r]) exchange[cnt[warp * BINS + ((item[r].x >> shift) & (BINS - 1))] + rank[r]] = item[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ONE_ROUNDS; ++r)
            if (in[r]) item[r] = exchange[base + r * 32];
    }
#pragma unroll
    for (int r = 0; r < ONE_ROUNDS; ++r)
        if (in[r]) p.out[base + r * 32] = item[r];
}

template <int R>
__global__ void __launch_bounds__(SORT_THREADS) sort_hist_kernel(const SortArgs p, int ctas) {
    pdl_wait();
    pdl_launch_dependents();
    if ((int)blockIdx.x >= ctas) {   // first pass: the rest of the grid
        zero_segments(p, ctas, (int)gridDim.x - ctas);
        return;
    }
    __shared__ int cnt[BINS];
    cnt[threadIdx.x] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * (SORT_THREADS * R);
    for (int r = 0; r < R; ++r) {
        const int64_t i = base + r * SORT_THREADS + threadIdx.x;
        if (i >= p.N) break;
        atomicAdd(&cnt[(sort_pair(p, i).x >> p.shift) & (BINS - 1)], 1);
    }
    __syncthreads();
    p.hist[(int64_t)blockIdx.x * BINS + threadIdx.x] = cnt[threadIdx.x];
}

// Stable: a pair goes behind every smaller digit, its digit in earlier CTAs, in
// earlier warps, and in its warp's earlier pairs.
template <int R>
__global__ void __launch_bounds__(SORT_THREADS) sort_scatter_kernel(const SortArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int WARPS = SORT_THREADS / 32;
    __shared__ int cnt[WARPS][BINS];
    __shared__ int warp_sum[BINS / 32];
    const int warp = threadIdx.x >> 5;
    for (int w = 0; w < WARPS; ++w) cnt[w][threadIdx.x] = 0;
    // digit threadIdx.x: all its pairs, and those in CTAs before this one
    int total = 0, before = 0;
#pragma unroll 8
    for (int b = 0; b < (int)gridDim.x; ++b) {
        const int h = p.hist[(int64_t)b * BINS + threadIdx.x];
        total += h;
        if (b < (int)blockIdx.x) before += h;
    }
    int start = scan_bins(total, warp_sum) + before;

    const int64_t base = (int64_t)blockIdx.x * (SORT_THREADS * R) + warp * (32 * R) + (threadIdx.x & 31);
    uint2 item[R];
    bool in[R];
    int rank[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        in[r] = base + r * 32 < p.N;
        item[r] = in[r] ? sort_pair(p, base + r * 32) : make_uint2(0u, 0u);
    }
    warp_ranks(item, in, p.shift, cnt[warp], rank);
    __syncthreads();
    for (int w = 0; w < WARPS; ++w) {   // digit threadIdx.x: each warp's first place
        const int c = cnt[w][threadIdx.x];
        cnt[w][threadIdx.x] = start;
        start += c;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (in[r]) p.out[cnt[warp][(item[r].x >> p.shift) & (BINS - 1)] + rank[r]] = item[r];
}

// -------------------------------------------------------------- gradient --

constexpr int SPAN = 32;          // sorted positions of a block
constexpr int GRAD_THREADS = 256;
constexpr int GRAD_WARPS = GRAD_THREADS / 32;
constexpr int GRAD_ROWS = 64;     // table rows of a CTA at most
constexpr int GRAD_BYTES = 32768; // and of table, where rows are short
constexpr int WARP_ROW = 4096;    // bytes of a table row up to which a warp takes it, not the CTA
constexpr int JOIN_COLS = 128;    // columns that a CTA joins at a time
// CTAs that join pieces, unless a block's would be fewer than 8: most find
// nothing to join (8192 tokens into 128000 x 4096: one for every block and 128
// columns would be 9 us slower)
constexpr int JOIN_CTAS = 2048;

struct GradArgs {
    const uint2* sorted;
    int2* seg;                    // [V): a row's sorted positions {first, last + 1}; {0, 0}: none
    const void* dout;
    void* dtable[kMaxG];
    float* pieces;                // [2 blocks][Hp]
    int64_t N, V, Vs, H, Hp;
    int blocks;                   // of SPAN positions
    int rows;                     // table rows of a CTA
    int by_warp;                  // a warp to a row
    int packs;                    // packs of a row
    int join_ctas;                // CTAs per block that join pieces
    float scale;
    int accumulate;
};

template <typename T, int N>
__device__ __forceinline__ void add_rows(const GradArgs& p, const uint32_t* tok, int n, int64_t col,
                                         float (&acc)[N]) {
    const T* base = static_cast<const T*>(p.dout) + col;
    int i = 0;
    for (; i + 4 <= n; i += 4) {   // four rows in flight, added in order
        Pack<T, N> x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = load_pack<T, N>(base + (int64_t)tok[i + u] * p.H);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += to_f32(x[u].v[j]);
    }
    for (; i < n; ++i) {
        const Pack<T, N> x = load_pack<T, N>(base + (int64_t)tok[i] * p.H);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += to_f32(x.v[j]);
    }
}

// Segments' ends, and the pieces of segments that cross blocks. Block b of
// SPAN sorted positions: piece 2 b is the run that began in an earlier block,
// piece 2 b + 1 the run that goes on into the next (and began here).
template <typename T, int N>
__global__ void __launch_bounds__(GRAD_THREADS) embedding_grad_pieces_kernel(const GradArgs p) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ uint32_t key[SPAN + 2];   // with the neighbours on either side
    __shared__ uint32_t tok[SPAN];
    const int b = (int)blockIdx.x;
    const int64_t first = (int64_t)b * SPAN;
    const int n = (int)min((int64_t)SPAN, p.N - first);
    const uint32_t none = 0xffffffffu;
    for (int i = threadIdx.x; i < n + 2; i += GRAD_THREADS) {
        const int64_t at = first + i - 1;
        const uint2 x = at >= 0 && at < p.N ? p.sorted[at] : make_uint2(none, 0u);
        key[i] = x.x;
        if (i >= 1 && i <= n) tok[i - 1] = x.y;
    }
    __syncthreads();
    if (blockIdx.y == 0 && (int)threadIdx.x < n) {
        const int i = (int)threadIdx.x;
        const uint32_t k = key[i + 1];
        if (k < (uint32_t)p.V) {
            if (key[i] != k) p.seg[k].x = (int)(first + i);
            if (key[i + 2] != k) p.seg[k].y = (int)(first + i) + 1;
        }
    }
    int head = 0, tail = n;   // the two runs: [0, head) and [tail, n)
    if (key[0] == key[1] && key[1] < (uint32_t)p.V)
        while (head < n && key[head + 1] == key[0]) ++head;
    if (n == SPAN && key[n + 1] == key[n] && key[n] < (uint32_t)p.V)
        while (tail > head && key[tail] == key[n + 1]) --tail;
    const int c = (int)(blockIdx.y * GRAD_THREADS + threadIdx.x);
    if (c >= p.packs) return;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const int lo = side ? tail : 0, hi = side ? n : head;
        if (lo >= hi) continue;
        float acc[N];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = 0.f;
        add_rows<T, N>(p, tok + lo, hi - lo, (int64_t)c * N, acc);
        float* dst = p.pieces + (int64_t)(2 * b + side) * p.Hp + (int64_t)c * N;
#pragma unroll
        for (int j = 0; j < N; ++j) dst[j] = acc[j];
    }
}

template <typename GT>
__device__ __forceinline__ GT* table_row(const GradArgs& p, uint32_t v) {
    const uint32_t k = v / (uint32_t)p.Vs;
    return static_cast<GT*>(p.dtable[k]) + (int64_t)(v - k * (uint32_t)p.Vs) * p.H;
}

// Zeros over a row that may begin anywhere, by `nt` threads: whole 16-byte
// words, then the elements at the row's two ends.
template <typename GT>
__device__ __forceinline__ void zero_row(GT* dst, int H, int t, int nt) {
    constexpr int N = 16 / (int)sizeof(GT);
    const int off = (int)((16 - (reinterpret_cast<uintptr_t>(dst) & 15)) & 15) / (int)sizeof(GT);
    const int head = min(off, H), body = (H - head) / N;
    uint4* v = reinterpret_cast<uint4*>(dst + head);
#pragma unroll 4
    for (int c = t; c < body; c += nt) __stcs(v + c, make_uint4(0u, 0u, 0u, 0u));
    const int ends = H - body * N;   // fewer than 2 N
    if (t < ends) dst[t < head ? t : t + body * N] = from_f32<GT>(0.f);
}

// One row from its segment's tokens, by `nt` threads.
template <typename T, int N, typename GT>
__device__ __forceinline__ void sum_row(const GradArgs& p, GT* dst, const uint32_t* tok, int n, int t, int nt) {
    for (int c = t; c < p.packs; c += nt) {
        float acc[N];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = 0.f;
        add_rows<T, N>(p, tok, n, (int64_t)c * N, acc);
        GT* at = dst + (int64_t)c * N;
        Pack<GT, N> o;
        if (p.accumulate) o = load_pack<GT, N>(at);
#pragma unroll
        for (int j = 0; j < N; ++j)
            o.v[j] = from_f32<GT>(p.accumulate ? fmaf(p.scale, acc[j], to_f32(o.v[j])) : p.scale * acc[j]);
        if constexpr (N * sizeof(GT) == 32) {
            const uint4* w = reinterpret_cast<const uint4*>(&o);
            __stcs(reinterpret_cast<uint4*>(at), w[0]);
            __stcs(reinterpret_cast<uint4*>(at) + 1, w[1]);
        } else {
            store_pack<GT, N>(at, o);
        }
    }
}

// Table rows from segments inside one block of positions (zeros where there is
// none), and, in the grid's first CTAs, from the pieces of the others. Short
// rows go to a warp each.
template <typename T, int N, typename GT>
__global__ void __launch_bounds__(GRAD_THREADS) embedding_grad_kernel(const GradArgs p) {
    pdl_wait();
    __shared__ float4 part[GRAD_WARPS][32];
    __shared__ int2 segs[GRAD_ROWS];
    __shared__ uint32_t tok[GRAD_WARPS][SPAN];
    const unsigned joins = (unsigned)p.blocks * (unsigned)p.join_ctas;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x < joins) {
        // the segment that begins in block b and goes on
        const int b = (int)(blockIdx.x / (unsigned)p.join_ctas);
        const int64_t next = (int64_t)(b + 1) * SPAN;
        if (next >= p.N) return;
        const uint32_t key = p.sorted[next].x;
        if (key >= (uint32_t)p.V) return;
        const int2 sg = p.seg[key];
        if (sg.x / SPAN != b) return;
        const int last = (sg.y - 1) / SPAN;
        const int count = last - b + 1;
        const int lo = (int)((int64_t)count * warp / GRAD_WARPS), hi = (int)((int64_t)count * (warp + 1) / GRAD_WARPS);
        const unsigned in_block = blockIdx.x - (unsigned)b * (unsigned)p.join_ctas;
        for (int64_t col0 = (int64_t)in_block * JOIN_COLS; col0 < p.Hp; col0 += (int64_t)p.join_ctas * JOIN_COLS) {
            const int64_t col = col0 + lane * 4;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            if (col < p.Hp) {
#pragma unroll 4
                for (int i = lo; i < hi; ++i) {
                    const int64_t slot = 2 * (int64_t)(b + i) + (i == 0 ? 1 : 0);
                    const float4 x = *reinterpret_cast<const float4*>(p.pieces + slot * p.Hp + col);
                    acc.x += x.x;
                    acc.y += x.y;
                    acc.z += x.z;
                    acc.w += x.w;
                }
            }
            part[warp][lane] = acc;
            __syncthreads();
            if (warp == 0 && col < p.Hp) {
                for (int w = 1; w < GRAD_WARPS; ++w) {
                    const float4 x = part[w][lane];
                    acc.x += x.x;
                    acc.y += x.y;
                    acc.z += x.z;
                    acc.w += x.w;
                }
                GT* dst = table_row<GT>(p, key) + col;
                const float v[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col + j < p.H)
                        dst[j] = from_f32<GT>(p.accumulate ? fmaf(p.scale, v[j], to_f32(dst[j])) : p.scale * v[j]);
            }
            __syncthreads();   // `part` is read before the next columns' sums
        }
        return;
    }
    const int64_t v0 = (int64_t)(blockIdx.x - joins) * p.rows;
    const int rows = (int)min((int64_t)p.rows, p.V - v0);
    if ((int)threadIdx.x < rows) segs[threadIdx.x] = p.N > 0 ? p.seg[v0 + threadIdx.x] : make_int2(0, 0);
    __syncthreads();
    if (!p.by_warp) {   // at most GRAD_WARPS rows: every row's tokens at once, a warp to a row
        const int2 sg = warp < rows ? segs[warp] : make_int2(0, 0);
        if (sg.y - sg.x > lane && sg.x / SPAN == (sg.y - 1) / SPAN) tok[warp][lane] = p.sorted[sg.x + lane].y;
        __syncthreads();
    }
    for (int r = p.by_warp ? warp : 0; r < rows; r += p.by_warp ? GRAD_WARPS : 1) {
        const int2 sg = segs[r];
        const int n = sg.y - sg.x;
        if (n > 0 && sg.x / SPAN != (sg.y - 1) / SPAN) continue;   // joined from pieces
        if (n == 0 && p.accumulate) continue;
        GT* dst = table_row<GT>(p, (uint32_t)(v0 + r));
        if (p.by_warp) {
            if (n == 0) {
                zero_row(dst, (int)p.H, lane, 32);
                continue;
            }
            __syncwarp();
            if (lane < n) tok[warp][lane] = p.sorted[sg.x + lane].y;
            __syncwarp();
            sum_row<T, N, GT>(p, dst, tok[warp], n, lane, 32);
        } else if (n == 0) {
            zero_row(dst, (int)p.H, (int)threadIdx.x, GRAD_THREADS);
        } else {
            sum_row<T, N, GT>(p, dst, tok[r], n, (int)threadIdx.x, GRAD_THREADS);
        }
    }
}

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline int64_t sort_ctas(int64_t N) {
    const int64_t tile = (int64_t)SORT_THREADS * (N <= FEW_TOKENS ? FEW_ROUNDS : SORT_ROUNDS);
    return (N + tile - 1) / tile;
}
inline int64_t grad_blocks(int64_t N) { return (N + SPAN - 1) / SPAN; }
inline int64_t piece_pitch(int64_t H) { return (H + 3) / 4 * 4; }

// Workspace: two arrays of (key, token) pairs, the digit counts, the segments,
// the pieces.
struct GradLayout {
    size_t pairs[2], hist, seg, pieces, total;
};
GradLayout grad_layout(int64_t N, int64_t V, int64_t H) {
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
    l.pieces = o;
    o += round256((size_t)(2 * grad_blocks(N)) * piece_pitch(H) * sizeof(float));
    l.total = o;
    return l;
}

// Elements per access that pointers of `align` bytes' alignment and rows of H
// elements of `size` bytes allow, up to 16 bytes.
int pack_elems(uintptr_t align, int64_t H, int size) {
    int n = 16 / size;
    while (n > 1 && (H % n != 0 || align % (uintptr_t)(n * size) != 0)) n /= 2;
    return n;
}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
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
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int N, typename GT>
cudaError_t grad_launch(const GradArgs& g, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (g.N > 0) {
        LaunchScope ls("embedding_grad_pieces", s);
        e = launch_pdl(embedding_grad_pieces_kernel<T, N>,
                       dim3((unsigned)g.blocks, (unsigned)((g.packs + GRAD_THREADS - 1) / GRAD_THREADS)),
                       GRAD_THREADS, 0, s, g);
    }
    if (e != cudaSuccess) return e;
    LaunchScope ls("embedding_grad", s);
    // N, V < 2^31, at most 8 joining CTAs a block or 2048, at least 8 rows a CTA: below 2^30
    const int64_t grid = (int64_t)g.blocks * g.join_ctas + (g.V + g.rows - 1) / g.rows;
    return launch_pdl(embedding_grad_kernel<T, N, GT>, dim3((unsigned)grid), GRAD_THREADS, 0, s, g);
}

template <typename T, typename GT>
cudaError_t grad_dispatch(const GradArgs& g, int n, cudaStream_t s) {
    if (n == 8) {
        if constexpr (sizeof(T) == 2) return grad_launch<T, 8, GT>(g, s);
    }
    if (n >= 4) return grad_launch<T, 4, GT>(g, s);
    if (n == 2) return grad_launch<T, 2, GT>(g, s);
    return grad_launch<T, 1, GT>(g, s);
}

template <typename T>
cudaError_t lookup_dispatch(const LookupArgs& p, int n, unsigned grid, cudaStream_t s) {
    if (n == 8) {
        if constexpr (sizeof(T) == 2)
            return launch_pdl(embedding_scaled_kernel<T, 8>, dim3(grid), LOOKUP_THREADS, 0, s, p);
    }
    if (n >= 4) return launch_pdl(embedding_scaled_kernel<T, 4>, dim3(grid), LOOKUP_THREADS, 0, s, p);
    if (n == 2) return launch_pdl(embedding_scaled_kernel<T, 2>, dim3(grid), LOOKUP_THREADS, 0, s, p);
    return launch_pdl(embedding_scaled_kernel<T, 1>, dim3(grid), LOOKUP_THREADS, 0, s, p);
}

}  // namespace

tpmlp_status run_vocab_embedding_scaled(int f32, int64_t N, int64_t V, int64_t H, int T,
                                        const int64_t* ids, const void* const* table, float scale,
                                        void* out, cudaStream_t s) {
    if (N == 0) return TPMLP_OK;
    LookupArgs p{};
    const int size = f32 ? 4 : 2;
    uintptr_t align = reinterpret_cast<uintptr_t>(out);
    p.ids = ids;
    for (int k = 0; k < T; ++k) {
        p.table[k] = table[k];
        align |= reinterpret_cast<uintptr_t>(table[k]);
    }
    const int n = pack_elems(align, H, size);
    p.out = out;
    p.N = N;
    p.V = V;
    p.Vs = V / T;
    p.H = H;
    p.packs = (int)(H / n);
    p.log_lanes = 5;   // at least a warp a row
    while ((1 << p.log_lanes) < LOOKUP_THREADS && (LOOKUP_UNROLL << p.log_lanes) < p.packs) ++p.log_lanes;
    p.segs = (p.packs + (LOOKUP_UNROLL << p.log_lanes) - 1) / (LOOKUP_UNROLL << p.log_lanes);
    p.scale = scale;
    p.err = device_error_word();
    if (p.err == nullptr) return TPMLP_ERR_CUDA;
    const int64_t rows = LOOKUP_THREADS >> p.log_lanes;
    const int64_t grid = (N + rows - 1) / rows * p.segs;
    if (grid > 0x7fffffffLL) return TPMLP_ERR_SHAPE;
    cudaError_t e;
    {
        LaunchScope ls("vocab_embedding_scaled", s);
        e = f32 ? lookup_dispatch<float>(p, n, (unsigned)grid, s)
                : lookup_dispatch<__nv_bfloat16>(p, n, (unsigned)grid, s);
    }
    return e == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

size_t embedding_grad_bytes(int64_t N, int64_t V, int64_t H) { return grad_layout(N, V, H).total; }

tpmlp_status run_vocab_embedding_backward(int f32, int grad_f32, int64_t N, int64_t V, int64_t H,
                                          int T, const int64_t* ids, const void* dout, float scale,
                                          int accumulate, void* const* dtable, void* workspace,
                                          cudaStream_t s) {
    if (N == 0 && accumulate) return TPMLP_OK;
    GradArgs g{};
    uintptr_t in_align = reinterpret_cast<uintptr_t>(dout), out_align = 0;
    for (int k = 0; k < T; ++k) {
        g.dtable[k] = dtable[k];
        out_align |= reinterpret_cast<uintptr_t>(dtable[k]);
    }
    // the same elements per access on both sides (a bf16 pack of 8 is two
    // 16-byte stores of fp32)
    const int gsize = grad_f32 ? 4 : 2;
    const int zn = pack_elems(out_align, H, gsize);
    int n = pack_elems(in_align, H, f32 ? 4 : 2);
    if (n > zn && !(n == 8 && zn == 4 && grad_f32)) n = zn;
    g.packs = (int)(H / n);
    if ((g.packs + (int64_t)GRAD_THREADS - 1) / GRAD_THREADS > 65535) return TPMLP_ERR_SHAPE;   // the grid's y
    const GradLayout l = grad_layout(N, V, H);
    char* ws = static_cast<char*>(workspace);
    int* err = device_error_word();
    if (err == nullptr) return TPMLP_ERR_CUDA;
    g.seg = reinterpret_cast<int2*>(ws + l.seg);
    if (N > 0) {
        SortArgs p{};
        p.ids = ids;
        p.hist = reinterpret_cast<int*>(ws + l.hist);
        p.seg = g.seg;
        p.N = N;
        p.V = V;
        p.bits = 1;
        while ((V >> p.bits) != 0) ++p.bits;   // keys 0..V
        p.err = err;
        if (N <= ONE_MAX) {
            p.out = reinterpret_cast<uint2*>(ws + l.pairs[0]);
            if (cudaFuncSetAttribute(sort_one_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ONE_SMEM) !=
                cudaSuccess)
                return TPMLP_ERR_CUDA;
            const unsigned zero_ctas = (unsigned)(V / (ONE_THREADS * 4) + 1 < 64 ? V / (ONE_THREADS * 4) + 1 : 64);
            LaunchScope ls("embedding_grad_sort", s);
            if (launch_pdl(sort_one_kernel, dim3(1 + zero_ctas), ONE_THREADS, ONE_SMEM, s, p) != cudaSuccess)
                return TPMLP_ERR_CUDA;
            g.sorted = p.out;
        } else {
            const int ctas = (int)sort_ctas(N);
            const bool few = N <= FEW_TOKENS;
            int which = 0;
            for (p.shift = 0; p.shift < p.bits; p.shift += RADIX_BITS) {
                p.out = reinterpret_cast<uint2*>(ws + l.pairs[which]);
                {
                    LaunchScope ls("embedding_grad_sort", s);
                    if (launch_pdl(few ? sort_hist_kernel<FEW_ROUNDS> : sort_hist_kernel<SORT_ROUNDS>,
                                   dim3((unsigned)(ctas + (p.shift == 0 ? 64 : 0))), SORT_THREADS, 0, s, p,
                                   ctas) != cudaSuccess)
                        return TPMLP_ERR_CUDA;
                }
                {
                    LaunchScope ls("embedding_grad_sort", s);
                    if (launch_pdl(few ? sort_scatter_kernel<FEW_ROUNDS> : sort_scatter_kernel<SORT_ROUNDS>,
                                   dim3((unsigned)ctas), SORT_THREADS, 0, s, p) != cudaSuccess)
                        return TPMLP_ERR_CUDA;
                }
                g.sorted = p.out;
                p.ids = nullptr;
                p.in = p.out;
                which ^= 1;
            }
        }
    }
    g.dout = dout;
    g.pieces = reinterpret_cast<float*>(ws + l.pieces);
    g.N = N;
    g.V = V;
    g.Vs = V / T;
    g.H = H;
    g.Hp = piece_pitch(H);
    g.blocks = (int)grad_blocks(N);
    // a block's columns over up to 8 CTAs, and over more where the blocks are few
    const int64_t join_cols = (H + JOIN_COLS - 1) / JOIN_COLS;
    const int64_t most = g.blocks > 0 && JOIN_CTAS / g.blocks > 8 ? JOIN_CTAS / g.blocks : 8;
    g.join_ctas = (int)(join_cols < most ? join_cols : most);
    // long rows: eight a CTA, all its threads on one after the other
    const int64_t row_bytes = H * gsize;
    g.by_warp = row_bytes <= WARP_ROW;
    g.rows = !g.by_warp ? GRAD_WARPS : row_bytes * GRAD_ROWS <= GRAD_BYTES ? GRAD_ROWS : (int)(GRAD_BYTES / row_bytes);
    g.scale = scale;
    g.accumulate = accumulate;
    cudaError_t e;
    if (f32)
        e = grad_f32 ? grad_dispatch<float, float>(g, n, s) : grad_dispatch<float, __nv_bfloat16>(g, n, s);
    else
        e = grad_f32 ? grad_dispatch<__nv_bfloat16, float>(g, n, s)
                     : grad_dispatch<__nv_bfloat16, __nv_bfloat16>(g, n, s);
    return e == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

}  // namespace tpmlp
