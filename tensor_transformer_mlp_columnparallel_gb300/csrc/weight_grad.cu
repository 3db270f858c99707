// Weight gradients of few tokens: C[m, n] = sum_{k < K} A[k, m] (B + B2)[k, n] in
// bf16 with K (tokens) small against M and N, for a list of such products in
// one launch. B2 is what B's rounding to bf16 left over (or absent): a second
// walk over the tokens into the same accumulator.
//
// Writing C bounds it: at K = 16 a 128 x 256 tile reads 12 KB of operands
// (from L2) for 64 KB of output, and its product is one K step. So the CTA is
// built around its stores: one persistent CTA an SM, eight epilogue warps
// instead of four, each taking 32 rows x 128 columns of the accumulator out of
// tensor memory, and 4 KB tensor stores whose rows are whole 128-byte lines,
// two in flight a warp. Warp 8 loads (TMA, a ring of 64-token stages), one
// thread of warp 9 issues the MMAs (tcgen05, M = 128, N = 256) into one of two
// accumulators, so the next tile is ready when an epilogue ends. (GB300, D =
// 4096, F = 16384, T = 4, 403 MB of gradients: 61 us at N = 16, 6.6 TB/s; 70
// at N = 64.)
//
// Every wait is bounded in time, as in the block's GEMM: one that runs out
// records TPMLP_ERR_TIMEOUT and raises the CTA's abort flag; loads and MMAs in
// flight are waited for, tensor memory is freed.
#include <cuda_bf16.h>

#include "act.cuh"
#include "ptx.cuh"
#include "tc_desc.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int WG_M = 128, WG_N = 256, WG_BK = 64;
constexpr int WG_STAGES = 3;
constexpr int WG_A_BYTES = WG_M * WG_BK * 2, WG_B_BYTES = WG_N * WG_BK * 2;
constexpr int WG_STAGE = WG_A_BYTES + WG_B_BYTES;
constexpr int WG_EPI_WARPS = 8;
constexpr int WG_OUT = 4096;                             // 32 rows x 64 columns of bf16
constexpr int WG_THREADS = 32 * (WG_EPI_WARPS + 2);
constexpr int WG_SMEM = 1024 + WG_STAGES * WG_STAGE + WG_EPI_WARPS * 2 * WG_OUT + 256;
static_assert(WG_SMEM <= 232448, "shared memory");

struct WgParams {
    CUtensorMap maps[4 * kMaxWeightGrads];      // operands and outputs
    int16_t a_map[kMaxWeightGrads], b_map[kMaxWeightGrads], c_map[kMaxWeightGrads];
    int16_t b2_map[kMaxWeightGrads];            // -1: none
    int M[kMaxWeightGrads], N[kMaxWeightGrads];
    int first_tile[kMaxWeightGrads + 1];        // tiles in front of each product
    int products, K, bk;                        // bk: tokens of a stage (a multiple of 16)
    int* err;
    uint64_t timeout_ns, drain_ns;
    int inject;          // failure-detection self test: the role that stalls (0: none)
};

struct WgTile {
    int q, m0, n0;
};
__device__ __forceinline__ WgTile wg_tile(const WgParams& p, int t) {
    WgTile w;
    w.q = 0;
    while (w.q + 1 < p.products && t >= p.first_tile[w.q + 1]) ++w.q;
    const int local = t - p.first_tile[w.q];
    const int tiles_n = (p.N[w.q] + WG_N - 1) / WG_N;
    const int tm = local / tiles_n;
    w.m0 = tm * WG_M;
    w.n0 = (local - tm * tiles_n) * WG_N;
    return w;
}

__global__ void __launch_bounds__(WG_THREADS, 1) weight_grad_kernel(const __grid_constant__ WgParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t s0 = smem_u32(smem);
    const uint32_t out0 = s0 + WG_STAGES * WG_STAGE;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + WG_STAGES * WG_STAGE + WG_EPI_WARPS * 2 * WG_OUT);
    constexpr int FULL = 0, EMPTY = WG_STAGES, TFULL = 2 * WG_STAGES, TEMPTY = TFULL + 2, DRAIN = TEMPTY + 2,
                  STALL = DRAIN + 1, NUM_BARS = DRAIN + 2;   // STALL: never completed (self test)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NUM_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t bar0 = smem_u32(bars);
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < WG_STAGES; ++s) {
            mbar_init(bar(FULL + s), 1);
            mbar_init(bar(EMPTY + s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar(TFULL + a), 1);
            mbar_init(bar(TEMPTY + a), WG_EPI_WARPS);
        }
        mbar_init(bar(DRAIN), 1);
        mbar_init(bar(STALL), 1);
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == WG_EPI_WARPS + 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    const int tiles = p.first_tile[p.products];
    const int k_blocks = (p.K + p.bk - 1) / p.bk;
    const uint32_t box = 128u * (uint32_t)p.bk;   // bytes of a 64-wide box

    if (warp == WG_EPI_WARPS) {
        if (lane == 0) {
            // ---------------- TMA producer ----------------
            int s = 0;
            uint32_t ph = 0, issued = 0;
            bool ok = p.inject != 3 || wait_bounded(bar(STALL), 0, abort_flag, p.err, p.timeout_ns, true);
            for (int t = (int)blockIdx.x; ok && t < tiles; t += (int)gridDim.x) {
                const WgTile w = wg_tile(p, t);
                const CUtensorMap* ma = &p.maps[p.a_map[w.q]];
                const int walks = p.b2_map[w.q] >= 0 ? 2 : 1;
                for (int i = 0; i < k_blocks * walks; ++i) {
                    const CUtensorMap* mb = &p.maps[i < k_blocks ? p.b_map[w.q] : p.b2_map[w.q]];
                    const int kb = i < k_blocks ? i : i - k_blocks;
                    if (!wait_fast(bar(EMPTY + s), ph ^ 1u, abort_flag, p.err, p.timeout_ns, true)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(bar(FULL + s), 6u * box);
                    const uint32_t a = s0 + (uint32_t)(s * WG_STAGE), b = a + WG_A_BYTES;
#pragma unroll
                    for (int j = 0; j < WG_M / 64; ++j)
                        tma_load_2d(a + (uint32_t)j * box, ma, bar(FULL + s), w.m0 + 64 * j, kb * p.bk);
#pragma unroll
                    for (int j = 0; j < WG_N / 64; ++j)
                        tma_load_2d(b + (uint32_t)j * box, mb, bar(FULL + s), w.n0 + 64 * j, kb * p.bk);
                    ++issued;
                    if (++s == WG_STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // no load may be in flight when the CTA leaves
            for (uint32_t j = issued > WG_STAGES ? issued - WG_STAGES : 0u; j < issued; ++j)
                wait_bounded(bar(FULL + (int)(j % WG_STAGES)), (j / WG_STAGES) & 1u, abort_flag, p.err, p.drain_ns,
                             false);
        }
    } else if (warp == WG_EPI_WARPS + 1) {
        if (lane == 0) {
            // ---------------- MMA issuer ----------------
            const uint32_t idesc = instr_desc(WG_M, WG_N, 1, 1);   // both operands lie K by M (N)
            const uint64_t da = smem_desc(s0, box, 1024), db = smem_desc(s0 + WG_A_BYTES, box, 1024);
            int s = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = p.inject != 2 || wait_bounded(bar(STALL), 0, abort_flag, p.err, p.timeout_ns, true);
            for (int t = (int)blockIdx.x; ok && t < tiles; t += (int)gridDim.x) {
                if (!wait_fast(bar(TEMPTY + acc), aph ^ 1u, abort_flag, p.err, p.timeout_ns, true)) break;
                tc_fence_after();
                const int walks = p.b2_map[wg_tile(p, t).q] >= 0 ? 2 : 1;
                for (int i = 0; i < k_blocks * walks; ++i) {
                    const int kb = i < k_blocks ? i : i - k_blocks;
                    if (!wait_fast(bar(FULL + s), ph, abort_flag, p.err, p.timeout_ns, true)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t off = (uint64_t)((s * WG_STAGE) >> 4);
                    const int steps = (min(p.bk, p.K - kb * p.bk) + 15) / 16;
                    for (int k = 0; k < steps; ++k)   // 16 rows of 128 bytes a step
                        tc_mma_f16(tmem + (uint32_t)(acc * WG_N), da + off + (uint64_t)(k * 128),
                                   db + off + (uint64_t)(k * 128), idesc, (i | k) != 0 ? 1u : 0u);
                    tc_commit(bar(EMPTY + s));
                    if (++s == WG_STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                tc_commit(bar(TFULL + acc));
                if (++acc == 2) {
                    acc = 0;
                    aph ^= 1u;
                }
            }
            tc_commit(bar(DRAIN));
            wait_bounded(bar(DRAIN), 0, abort_flag, p.err, p.drain_ns, false);
        }
    } else {
        // ---------------- epilogue ----------------
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t buf0 = out0 + (uint32_t)(warp * 2 * WG_OUT);
        int acc = 0;
        uint32_t aph = 0;
        int live = 1;
        if (p.inject == 1) {
            if (lane == 0) live = wait_bounded(bar(STALL), 0, abort_flag, p.err, p.timeout_ns, true);
            live = __shfl_sync(0xffffffffu, live, 0);
        }
        for (int t = (int)blockIdx.x; live && t < tiles; t += (int)gridDim.x) {
            const WgTile w = wg_tile(p, t);
            int ok = 1;
            if (lane == 0) ok = wait_fast(bar(TFULL + acc), aph, abort_flag, p.err, p.timeout_ns, true);
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            tc_fence_after();
            const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * WG_N + half * 128);
            const int row = w.m0 + quarter * 32;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t r[2][32];
                tmem_ld_32cols(src + (uint32_t)(b * 64), r[0]);
                tmem_ld_32cols(src + (uint32_t)(b * 64 + 32), r[1]);
                tmem_ld_wait();
                if (b == 1) {   // the accumulator is read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(TEMPTY + acc));
                }
                // the store that last used this buffer has read it
                if (lane == 0) bulk_wait_read_all_but_one();
                __syncwarp();
                const uint32_t buf = buf0 + (uint32_t)(b * WG_OUT);
#pragma unroll
                for (int j = 0; j < 8; ++j) {   // 16-byte word j of row r at j ^ (r & 7): the map's swizzle
                    const uint32_t(&x)[32] = r[j >> 2];
                    const int o = (j & 3) * 8;
                    uint32_t v[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        v[h] = pack_bf16x2(__uint_as_float(x[o + 2 * h]), __uint_as_float(x[o + 2 * h + 1]));
                    st_shared_v4(buf + (uint32_t)lane * 128u + (uint32_t)((j ^ (lane & 7)) << 4), v[0], v[1], v[2],
                                 v[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                const int col = w.n0 + half * 128 + b * 64;
                if (lane == 0) {
                    if (row < p.M[w.q] && col < p.N[w.q]) tma_store_2d(&p.maps[p.c_map[w.q]], buf, col, row);
                    bulk_commit();
                }
            }
            if (++acc == 2) {
                acc = 0;
                aph ^= 1u;
            }
        }
        if (lane == 0) bulk_wait_all();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == WG_EPI_WARPS + 1) tmem_dealloc(tmem, 512);
}

}  // namespace

tpmlp_status run_weight_grads(const WeightGradProduct* products, int count, int K, cudaStream_t s,
                              const char* name) {
    if (count < 1) return TPMLP_OK;
    if (count > kMaxWeightGrads || K < 1) return TPMLP_ERR_SHAPE;
    static WgParams p;   // large; filled per call under the lock
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    p.bk = K < WG_BK ? (K + 15) / 16 * 16 : WG_BK;
    int64_t tiles = 0;
    int maps = 0;
    for (int q = 0; q < count; ++q) {
        const WeightGradProduct& w = products[q];
        // consecutive products often share an operand (X, dY)
        const bool same_a = q > 0 && w.A == products[q - 1].A && w.M == products[q - 1].M && w.lda == products[q - 1].lda;
        const bool same_b = q > 0 && w.B == products[q - 1].B && w.N == products[q - 1].N && w.ldb == products[q - 1].ldb;
        bool ok = true;
        if (!same_a) ok = make_map(&p.maps[maps], w.A, w.M, K, w.lda, 64, p.bk);
        p.a_map[q] = (int16_t)(same_a ? p.a_map[q - 1] : maps++);
        if (!same_b) ok = ok && make_map(&p.maps[maps], w.B, w.N, K, w.ldb, 64, p.bk);
        p.b_map[q] = (int16_t)(same_b ? p.b_map[q - 1] : maps++);
        if (w.B2 != nullptr) ok = ok && make_map(&p.maps[maps], w.B2, w.N, K, w.ldb, 64, p.bk);
        p.b2_map[q] = (int16_t)(w.B2 != nullptr ? maps++ : -1);
        ok = ok && make_map(&p.maps[maps], w.C, w.N, w.M, w.ldc, 64, 32);
        p.c_map[q] = (int16_t)maps++;
        if (!ok) return TPMLP_ERR_CUDA;
        p.M[q] = w.M;
        p.N[q] = w.N;
        p.first_tile[q] = (int)tiles;
        tiles += (int64_t)((w.M + WG_M - 1) / WG_M) * ((w.N + WG_N - 1) / WG_N);
        if (tiles > 0x7fffffffLL) return TPMLP_ERR_SHAPE;
    }
    p.first_tile[count] = (int)tiles;
    p.products = count;
    p.K = K;
    p.err = device_error_word();
    if (p.err == nullptr) return TPMLP_ERR_CUDA;
    p.timeout_ns = wait_timeout_ns();
    p.inject = weight_grad_stall_role();
    p.drain_ns = p.timeout_ns > 100000000ull ? p.timeout_ns : 100000000ull;
    if (cudaFuncSetAttribute(weight_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, WG_SMEM) != cudaSuccess)
        return TPMLP_ERR_CUDA;
    const int64_t sms = device_sm_count();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)(tiles < sms ? tiles : sms));
    cfg.blockDim = dim3(WG_THREADS);
    cfg.dynamicSmemBytes = WG_SMEM;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    {
        LaunchScope ls(name, s);
        e = cudaLaunchKernelEx(&cfg, weight_grad_kernel, p);
    }
    if (e != cudaSuccess) return TPMLP_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

}  // namespace tpmlp
