// zf_vec.h -- device helpers shared by the kernels that work on rows of fp32,
// fp16 or bf16 elements at any element offset (zeroflat_embed.hip,
// zeroflat_act.hip, zeroflat_wgrad.hip): groups of eight elements per lane,
// formats, and division by a fixed number.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zf_launch.h"

namespace zf {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
// Words of any element alignment: global memory is read and written at any byte
// address on gfx950 (the compiler emits the full-width instructions), so that a
// view inside a flat buffer needs no path of its own.
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int v4u_any __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int v2u_any __attribute__((ext_vector_type(2), aligned(1)));

template <int DT>
struct Elem { using type = uint16_t; };
template <>
struct Elem<ZERO_F32> { using type = float; };

template <int DT>
__device__ __forceinline__ float to_f32(typename Elem<DT>::type x) {
    if constexpr (DT == ZERO_F32) return x;
    else if constexpr (DT == ZERO_F16) return (float)__builtin_bit_cast(_Float16, x);
    else return __uint_as_float((uint32_t)x << 16);
}
// to nearest, ties to even (one instruction per value or pair on gfx950)
template <int DT>
__device__ __forceinline__ typename Elem<DT>::type from_f32(float x) {
    if constexpr (DT == ZERO_F32) return x;
    else if constexpr (DT == ZERO_F16) return __builtin_bit_cast(uint16_t, (_Float16)x);
    else return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// Eight consecutive elements at p, the first `n` of which exist (the others
// read as 0); n >= 8 is the common case.
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t i, int n, float (&x)[8]) {
    using T = typename Elem<DT>::type;
    const T* p = static_cast<const T*>(base) + i;
    if (n >= 8) {
        if constexpr (DT == ZERO_F32) {
            const v4f a = *reinterpret_cast<const v4f_any*>(p);
            const v4f b = *reinterpret_cast<const v4f_any*>(p + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) { x[k] = a[k]; x[4 + k] = b[k]; }
        } else {
            const v4u a = *reinterpret_cast<const v4u_any*>(p);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[2 * k] = to_f32<DT>((uint16_t)(a[k] & 0xffffu));
                x[2 * k + 1] = to_f32<DT>((uint16_t)(a[k] >> 16));
            }
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < n ? to_f32<DT>(p[k]) : 0.0f;
}
// STREAM: past the caches, for what is not read again while it would be there.
template <int DT, bool STREAM>
__device__ __forceinline__ void store8_as(void* base, int64_t i, int n, const float (&x)[8]) {
    using T = typename Elem<DT>::type;
    T* p = static_cast<T*>(base) + i;
    if (n >= 8) {
        if constexpr (DT == ZERO_F32) {
            v4f_any* q = reinterpret_cast<v4f_any*>(p);
            const v4f_any a = {x[0], x[1], x[2], x[3]}, b = {x[4], x[5], x[6], x[7]};
            if constexpr (STREAM) {
                __builtin_nontemporal_store(a, q);
                __builtin_nontemporal_store(b, q + 1);
            } else {
                q[0] = a;
                q[1] = b;
            }
        } else {
            v4u_any a;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                a[k] = (uint32_t)from_f32<DT>(x[2 * k]) | (uint32_t)from_f32<DT>(x[2 * k + 1]) << 16;
            if constexpr (STREAM) __builtin_nontemporal_store(a, reinterpret_cast<v4u_any*>(p));
            else *reinterpret_cast<v4u_any*>(p) = a;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = from_f32<DT>(x[k]);
}
// Eight consecutive elements as they lie in memory, to be converted later: loads
// that nothing waits for between them.
template <int DT>
struct Raw8 {
    v4u lo, hi;                            // hi: fp32 only
};
template <int DT, bool STREAM = false>
__device__ __forceinline__ Raw8<DT> fetch8(const void* base, int64_t i) {
    const auto* p = static_cast<const typename Elem<DT>::type*>(base) + i;
    Raw8<DT> r;
    if constexpr (DT == ZERO_F32) {
        const v4f_any* q = reinterpret_cast<const v4f_any*>(p);
        r.lo = __builtin_bit_cast(v4u, STREAM ? __builtin_nontemporal_load(q) : q[0]);
        r.hi = __builtin_bit_cast(v4u, STREAM ? __builtin_nontemporal_load(q + 1) : q[1]);
    } else {
        const v4u_any* q = reinterpret_cast<const v4u_any*>(p);
        r.lo = STREAM ? __builtin_nontemporal_load(q) : q[0];
    }
    return r;
}
template <int DT>
__device__ __forceinline__ float element(const Raw8<DT>& r, int k) {
    if constexpr (DT == ZERO_F32) {
        const uint32_t w = k < 4 ? r.lo[k] : r.hi[k - 4];
        return __uint_as_float(w);
    } else {
        const uint32_t w = r.lo[k / 2];
        if constexpr (DT == ZERO_BF16) return __uint_as_float(k & 1 ? w & 0xffff0000u : w << 16);
        else return to_f32<DT>((uint16_t)(k & 1 ? w >> 16 : w));
    }
}

// The compiler would make one plain store of the two branches: empty statements
// that it cannot move keep them apart.
#define ZF_APART asm volatile("" ::: "memory")
template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t i, int n, const float (&x)[8], int stream) {
    if (stream) {
        ZF_APART;
        store8_as<DT, true>(base, i, n, x);
        ZF_APART;
    } else {
        store8_as<DT, false>(base, i, n, x);
    }
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31, by a product: with 2^s >= d the
// least such power and m = floor(2^32 (2^s - d) / d) + 1, the quotient is
// (mulhi(m, n) + n) >> s (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994); the sum stays below 2^32.
inline Div make_div(uint32_t d) {
    uint32_t s = 0;
    while (((uint64_t)1 << s) < d) ++s;
    const uint64_t m = ((((uint64_t)1 << s) - d) << 32) / d + 1;
    return Div{d, (uint32_t)m, s};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const Div& v) {
    return (__umulhi(v.m, n) + n) >> v.s;
}

}  // namespace zf
