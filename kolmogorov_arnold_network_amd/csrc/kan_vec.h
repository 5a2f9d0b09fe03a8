// Vector loads and stores of the token-side kernels: VEC consecutive elements
// of a row in storage type TS, as floats.  Rows start at any element (odd
// widths, halves of a wider array), so the vectors claim only the alignment
// of one element; the hardware takes such accesses at full width.
#pragma once

#include "kan_device.h"

namespace kan {

typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

// BYTES of a row as 32-bit words
template <int BYTES>
struct words;
template <>
struct words<4> {
    typedef uint32_t type;
};
template <>
struct words<8> {
    typedef u32x2v type;
};
template <>
struct words<16> {
    typedef u32x4v type;
};

// The raw words of VEC elements, and their values.
template <typename TS, int VEC>
struct Raw {
    static constexpr int W = VEC * (int)sizeof(TS) / 4;
    uint32_t w[W];
};
template <>
struct Raw<uint16_t, 1> {
    uint32_t w[1];
};

template <typename TS, int VEC>
__device__ __forceinline__ Raw<TS, VEC> load_raw(const TS* p) {
    Raw<TS, VEC> r;
    if constexpr (sizeof(TS) * VEC == 2) {
        r.w[0] = *p;
    } else {
        typedef typename words<(int)sizeof(TS) * VEC>::type W;
        typedef W Wu __attribute__((aligned(sizeof(TS))));
        const W v = *reinterpret_cast<const Wu*>(p);
        __builtin_memcpy(r.w, &v, sizeof(v));
    }
    return r;
}

// The same, for data that is read once: the caches keep it no longer than needed.
template <typename TS, int VEC>
__device__ __forceinline__ Raw<TS, VEC> load_once(const TS* p) {
    static_assert(sizeof(TS) * VEC > 2, "a vector");
    Raw<TS, VEC> r;
    typedef typename words<(int)sizeof(TS) * VEC>::type W;
    typedef W Wu __attribute__((aligned(sizeof(TS))));
    const W v = __builtin_nontemporal_load(reinterpret_cast<const Wu*>(p));
    __builtin_memcpy(r.w, &v, sizeof(v));
    return r;
}

template <typename TS, int VEC>
__device__ __forceinline__ float raw_value(const Raw<TS, VEC>& r, int i) {
    if constexpr (sizeof(TS) == 4) return __uint_as_float(r.w[i]);
    else return __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
}

// STREAM: the caches keep what is written no longer than needed.
template <int VEC, bool STREAM = false>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
    typedef typename words<4 * VEC>::type W;
    typedef W Wu __attribute__((aligned(4)));
    W w;
    __builtin_memcpy(&w, v, sizeof(w));
    if constexpr (STREAM) __builtin_nontemporal_store(w, reinterpret_cast<Wu*>(p));
    else *reinterpret_cast<Wu*>(p) = w;
}
// Two floats rounded to nearest even bf16, in one instruction (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const f32x2 f = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

template <int VEC, bool STREAM = false>
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        *p = f2bf(v[0]);
    } else {
        typedef typename words<2 * VEC>::type W;
        typedef W Wu __attribute__((aligned(2)));
        uint32_t u[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) u[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        W w;
        __builtin_memcpy(&w, u, sizeof(w));
        if constexpr (STREAM) __builtin_nontemporal_store(w, reinterpret_cast<Wu*>(p));
        else *reinterpret_cast<Wu*>(p) = w;
    }
}

}  // namespace kan
