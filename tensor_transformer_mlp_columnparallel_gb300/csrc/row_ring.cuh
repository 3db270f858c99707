// Rows in turn: CTAs that stay on their SM, whose groups of threads each take one
// row after the other, the next ones on their way to shared memory; and the
// launches of kernels that wait for what runs before them.
#pragma once
#include <atomic>
#include <type_traits>

#include "access.cuh"
#include "ptx.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int LONGEST = 8192;    // elements of a row that is taken in turn

// The lanes of this thread's group of NT threads, a power of two, in its warp.
template <int NT> __device__ __forceinline__ uint32_t group_lanes() {
    if constexpr (NT >= 32) return 0xffffffffu;
    else return ((1u << NT) - 1u) << (threadIdx.x & 31 & ~(NT - 1));
}

// A barrier of a group of NT threads.
template <int NT> __device__ __forceinline__ void group_sync(int group) {
    if constexpr (NT > 32)
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(NT) : "memory");
    else
        __syncwarp(group_lanes<NT>());
}

// wait_bounded without the call: one in the loop would have the threads' columns
// saved around it.
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t phase, volatile int* flag, int* err,
                                            uint64_t timeout_ns) {
    if (mbar_try_wait(bar, phase)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait(bar, phase)) return true;
        if (*flag) return false;
        if (globaltimer_ns() - t0 > timeout_ns) {
            *flag = 1;
            atomicCAS(err, 0, (int)TPMLP_ERR_TIMEOUT);
            return false;
        }
    }
}

// CTAs of TH threads that stay, in groups of as many threads, NT, as a row needs at
// LONGEST / TH elements a thread (FULL: exactly). A thread keeps its columns'
// parameters in registers; a group's next rows (Q matrices of STAGES rows) are on
// their way to shared memory. Rows of whole 16-byte accesses come by bulk copies,
// one instruction a row (copies by every thread were what the layer norm's gradient
// waited for: 8192 x 8192 bf16, 107 us against 87), others by 4-byte copies of the threads' own elements.
template <typename T, int B, int Q, int STAGES, int TH, int NT, bool FULL>
struct RowRing {
    using A = Access<T, B>;
    using Word = typename A::Word;
    static constexpr bool BULK = B == 16;
    static constexpr int R = LONGEST / TH / A::N, GROUPS = TH / NT;
    Word* rows;          // of this group
    uint64_t* bars;      // BULK: STAGES of this group
    int t, accesses, group;
    int k;               // the current row's stage
    uint32_t phase;

    static constexpr int MOST = GROUPS * STAGES * Q * NT * R * B;
    __device__ __forceinline__ RowRing(void* memory, uint64_t* barriers, int64_t D) {
        group = threadIdx.x / NT;
        t = threadIdx.x & (NT - 1);
        accesses = FULL ? NT * R : (int)(D / A::N);
        rows = static_cast<Word*>(memory) + group * STAGES * Q * NT * R;
        bars = barriers + group * STAGES;
        k = 0;
        phase = 0;
        if (BULK) {
            if (t == 0)
                for (int s = 0; s < STAGES; ++s) mbar_init(smem_u32(bars + s), 1);
            fence_mbar_init();
            fence_proxy_async_smem();
            group_sync<NT>(group);
        }
    }
    __device__ __forceinline__ bool mine(int i) const { return FULL || t + i * NT < accesses; }
    // access i of matrix q of the current row; zeros beyond it
    __device__ __forceinline__ Word at(int q, int i) const {
        return mine(i) ? rows[(k * Q + q) * (NT * R) + t + i * NT] : Word{};
    }
    // into stage s: BULK: thread 0's work, once the group is done with the stage
    __device__ __forceinline__ void fetch(int s, int q, const void* base, int64_t row, int64_t ld) const {
        const T* src = static_cast<const T*>(base) + row * ld;
        Word* dst = rows + (s * Q + q) * (NT * R);
        if constexpr (BULK) {
            bulk_load_g2s(smem_u32(dst), src, (uint32_t)accesses * B, smem_u32(bars + s));
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (mine(i)) {
                    const Word* from = reinterpret_cast<const Word*>(src) + t + i * NT;
                    if constexpr (B == 4)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst + t + i * NT)),
                                     "l"(from) : "memory");
                    else   // there is no copy of 2 bytes
                        dst[t + i * NT] = *from;
                }
        }
    }
    // copy(s): the fetches of one row into stage s, if there is such a row
    template <typename Copy> __device__ __forceinline__ void ask(int s, bool there, Copy copy) const {
        if constexpr (BULK) {
            if (t == 0 && there) {
                mbar_arrive_expect_tx(smem_u32(bars + s), (uint32_t)(Q * accesses * B));
                copy(s);
            }
        } else {
            if (there) copy(s);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    // The current row has arrived; false: not within the limit (flag, the group's
    // for this turn, is set).
    __device__ __forceinline__ bool wait(volatile int* flag, int* err, uint64_t timeout_ns) const {
        if constexpr (BULK) {
            const bool ok = wait_inline(smem_u32(bars + k), phase, flag, err, timeout_ns);
            return NT > 32 ? ok : __all_sync(0xffffffffu, ok);
        } else {
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
            return true;
        }
    }
    __device__ __forceinline__ void next() {
        if (++k == STAGES) {
            k = 0;
            phase ^= 1u;
        }
    }
    // The self test's stall: a wait for `spare`, a barrier of the group that nothing
    // completes.
    __device__ __forceinline__ bool stall(uint64_t* spare, volatile int* flag, int* err, uint64_t timeout_ns) const {
        if (t == 0) mbar_init(smem_u32(spare), 1);
        fence_mbar_init();
        group_sync<NT>(group);
        return wait_inline(smem_u32(spare), 0, flag, err, timeout_ns);
    }
    // After a wait that ran out: no copy may be in flight into a CTA that leaves.
    // `left` rows from the current one on were asked for.
    __device__ __forceinline__ void drain(uint32_t left, volatile int* flag, int* err, uint64_t timeout_ns) {
        if (!BULK || t != 0) return;
        const uint64_t limit = timeout_ns > 100000000ull ? timeout_ns : 100000000ull;
        for (uint32_t i = 0; i < left && i < STAGES; ++i, next()) wait_bounded(smem_u32(bars + k), phase, flag, err, limit, false);
    }
};

template <typename... P, typename... A>
tpmlp_status launch_smem(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
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
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return TPMLP_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

template <typename... P, typename... A>
tpmlp_status launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
    return launch_smem(kernel, grid, threads, 0, s, args...);
}

// The kernel may use `bytes` of dynamic shared memory: asked for once a device
// (`asked`: one bit each; devices beyond ask every time).
template <typename K>
bool allow_smem(K kernel, int bytes, std::atomic<uint64_t>& asked) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (asked.load() & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    asked.fetch_or(bit);
    return true;
}

// f(NT, FULL) as constants: the group of NT to TH threads that rows of D elements take
template <int TH, int NT, typename F> tpmlp_status with_group(int64_t D, F f) {
    constexpr int ELEMS = LONGEST / TH;
    const std::integral_constant<int, NT> nt;
    if constexpr (NT < TH)
        if (D > NT * ELEMS) return with_group<TH, 2 * NT>(D, f);
    return D == NT * ELEMS ? f(nt, std::true_type()) : f(nt, std::false_type());
}

}  // namespace
}  // namespace tpmlp
