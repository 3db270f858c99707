// Accesses of 16, 4 or 2 bytes to rows of fp32 or bf16 elements, as fp32 values:
// the widest access that divides a row, its pitch and its address serves all
// of the row.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "act.cuh"
#include "f32x2.cuh"

namespace tpmlp {

template <int B> struct AccessWord;
template <> struct AccessWord<16> { using type = uint4; };
template <> struct AccessWord<8> { using type = uint2; };
template <> struct AccessWord<4> { using type = uint32_t; };
template <> struct AccessWord<2> { using type = unsigned short; };

template <int N> struct PairOf { using type = F2; };
template <> struct PairOf<1> { using type = float; };

// N elements of T in one access of B bytes.
template <typename T, int B>
struct Access {
    using Word = typename AccessWord<B>::type;
    static constexpr int N = B / (int)sizeof(T);
    static_assert(N >= 1, "an access holds an element");

    static __device__ __forceinline__ void unpack(const Word& x, float (&v)[N]) {
        if constexpr (sizeof(T) == 4) {
            const float* f = reinterpret_cast<const float*>(&x);
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = f[j];
        } else if constexpr (B == 2) {
            v[0] = __uint_as_float((uint32_t)x << 16);
        } else {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    }
    // the same as packed pairs (a single element: as itself)
    using Pair = typename PairOf<N>::type;
    static constexpr int PAIRS = N > 1 ? N / 2 : 1;
    static __device__ __forceinline__ Pair both(float x) {
        if constexpr (N > 1) return f2(x, x);
        else return x;
    }
    static __device__ __forceinline__ void unpack(const Word& x, F2 (&v)[N > 1 ? PAIRS : 2]) {
        float e[N];
        unpack(x, e);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) v[j] = f2(e[2 * j], e[2 * j + 1]);
    }
    static __device__ __forceinline__ Word pack(const F2 (&v)[N > 1 ? PAIRS : 2]) {
        float e[N];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) split2(v[j], e[2 * j], e[2 * j + 1]);
        return pack(e);
    }
    static __device__ __forceinline__ float total(F2 v) {   // of a sum kept in pairs
        float a, b;
        split2(v, a, b);
        return a + b;
    }
    static __device__ __forceinline__ float total(float v) { return v; }
    static __device__ __forceinline__ Word pack(const float (&v)[N]) {
        Word x;
        if constexpr (sizeof(T) == 4) {
            float* f = reinterpret_cast<float*>(&x);
#pragma unroll
            for (int j = 0; j < N; ++j) f[j] = v[j];
        } else if constexpr (B == 2) {
            x = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
        } else {
            uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        }
        return x;
    }
};

// N consecutive elements of T from an address that is aligned to
// min(16, N sizeof(T)) bytes (parameters, which many rows read: cached).
template <typename T, int N>
__device__ __forceinline__ void load_params(const T* p, float (&v)[N]) {
    constexpr int BYTES = N * (int)sizeof(T), B = BYTES < 16 ? BYTES : 16;
    using A = Access<T, B>;
#pragma unroll
    for (int k = 0; k < BYTES / B; ++k) {
        float t[A::N];
        A::unpack(__ldg(reinterpret_cast<const typename A::Word*>(p) + k), t);
#pragma unroll
        for (int j = 0; j < A::N; ++j) v[k * A::N + j] = t[j];
    }
}

template <typename T, int N>
__device__ __forceinline__ void load_params(const T* p, F2 (&v)[N / 2]) {
    float e[N];
    load_params<T, N>(p, e);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) v[j] = f2(e[2 * j], e[2 * j + 1]);
}

// Host side: whether accesses of `bytes` fit an address and (for several rows)
// a pitch in bytes.
inline bool access_fits(const void* p, int64_t pitch, int bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && pitch % bytes == 0;
}

}  // namespace tpmlp
