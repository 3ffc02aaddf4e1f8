// lmkv_rotary.cuh -- rotary position encoding: what the append kernel and the
// shifted scatter share.
//
// Angles.  t = p * f radians is p * (f / 2 pi) turns, and only the fraction of
// a turn matters.  With F = round(f / 2 pi * 2^64) the product p * F modulo
// 2^64 is that fraction exactly as far as F goes (2^-53 of f, or 2^-64 of a turn), for any
// int64 p, negative ones included: three 32-bit multiplications and no
// 64-bit floating point, where an fp32 product p * f is off by p * f * 2^-24
// radians (0.008 at p = 131072, f = 1).  The top 32 bits, as a signed number
// of half turns, go to sincospif, whose argument needs no further reduction.
#pragma once

#include "lmkv_paged.cuh"

namespace lmkv_rotary_detail {

using lmkv_paged::Elem;

// By-value kernel parameter.
struct Rotary {
    int32_t half;          // pairs: rot_dim / 2
    int32_t interleaved;
    float magnitude;
    uint64_t turns[LMKV_ROTARY_MAX_PAIRS];
};

// INVALID_ARG for a rotary that does not fit the head or holds a value that
// is not finite.
int make_rotary(const lmkv_rotary_t* in, int32_t head_dim, Rotary* out);

// For 16-bit rows the special function unit's sine and cosine will do: on
// [-pi, pi] they are within 2^-21.1, less than a hundredth of those types' half step.
template <class T>
__device__ __forceinline__ float2 cos_sin(uint64_t turns, int64_t pos) {
    const uint64_t frac = turns * (uint64_t)pos;
    const float half_turns = (float)(int32_t)(uint32_t)(frac >> 32) * 4.656612873077393e-10f;   // 2^-31
    float s, c;
    if constexpr (sizeof(T) == 2) __sincosf(half_turns * 3.14159265358979f, &s, &c);
    else sincospif(half_turns, &s, &c);
    return make_float2(c, s);
}

// V elements of T in one register vector of 16 bytes (V = 16 / sizeof(T)), or
// a single element (V = 1).
template <class T, int V>
struct Vec {
    T x[V];
};
// Rows are read once: past L1.  kStream: they are not this kernel's own output
// either, and what is written is not needed soon.
template <class T, int V, bool kStream>
__device__ __forceinline__ Vec<T, V> ld_vec(const T* p) {
    Vec<T, V> v;
    if constexpr (V * sizeof(T) == 16) {
        int4& r = *reinterpret_cast<int4*>(v.x);
        if constexpr (kStream)
            asm("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
                : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
        else
            asm volatile("ld.global.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v.x[i] = p[i];
    }
    return v;
}
template <class T, int V, bool kStream>
__device__ __forceinline__ void st_vec(T* p, const Vec<T, V>& v) {
    if constexpr (V * sizeof(T) == 16) {
        const int4 r = *reinterpret_cast<const int4*>(v.x);
        if constexpr (kStream)
            asm volatile("st.global.cs.v4.s32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
                         : "memory");
        else *reinterpret_cast<int4*>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = v.x[i];
    }
}

// A head is worked on in units.  Half layout: unit u < half / V turns V pairs,
// the vectors at u * V and half + u * V; interleaved: unit u < 2 * half / V
// turns the V / 2 pairs of the vector at u * V.  The units after these copy
// the vectors behind rot_dim.  V is 16 bytes' worth where pointers, strides,
// half and head_dim allow it, else 1: a unit is then one pair of either layout,
// or one element (head_dim may be odd).
// (cos, sin) of the pairs lie in shared memory as [pair of the unit][unit], so
// that the units of a warp read consecutive places.
template <class T, int V, bool kInterleaved, bool kStream = false>
struct Units {
    static constexpr bool kTwo = !kInterleaved || V == 1;        // a turning unit is two vectors
    static constexpr int kPairs = kTwo ? V : V / 2;              // of a unit
    // The place of pair i's (cos, sin).
    static __device__ __forceinline__ int place(int i, int half) {
        return (i % kPairs) * turning(half) + i / kPairs;
    }
    static __device__ __host__ __forceinline__ int turning(int half) { return half / kPairs; }
    static __device__ __host__ __forceinline__ int count(int half, int head_dim) {
        return turning(half) + (head_dim - 2 * half) / V;
    }
    // Where a turning unit's vectors are.
    static __device__ __forceinline__ int first(int u) { return kInterleaved && kTwo ? 2 * u : u * V; }
    static __device__ __forceinline__ int second(int u, int half) { return kInterleaved ? 2 * u + 1 : half + u * V; }
    Vec<T, V> a, b;

    __device__ __forceinline__ void load(const T* head, int u, int half) {
        const int nt = turning(half);
        if (!kTwo || u >= nt) {
            a = ld_vec<T, V, kStream>(head + (u < nt ? u * V : 2 * half + (u - nt) * V));
        } else {
            a = ld_vec<T, V, kStream>(head + first(u));
            b = ld_vec<T, V, kStream>(head + second(u, half));
        }
    }
    // cs: this token's (cos, sin) table.
    __device__ __forceinline__ void turn(const float2* cs, int u, int half) {
        const int nt = turning(half);
        if (u >= nt) return;
        if constexpr (!kTwo) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 w = cs[i * nt + u];
                const float x = Elem<T>::to_float(a.x[2 * i]), y = Elem<T>::to_float(a.x[2 * i + 1]);
                a.x[2 * i] = Elem<T>::from_float(x * w.x - y * w.y);
                a.x[2 * i + 1] = Elem<T>::from_float(x * w.y + y * w.x);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 w = cs[i * nt + u];
                const float x = Elem<T>::to_float(a.x[i]), y = Elem<T>::to_float(b.x[i]);
                a.x[i] = Elem<T>::from_float(x * w.x - y * w.y);
                b.x[i] = Elem<T>::from_float(x * w.y + y * w.x);
            }
        }
    }
    __device__ __forceinline__ void store(T* head, int u, int half) const {
        const int nt = turning(half);
        if (!kTwo || u >= nt) {
            st_vec<T, V, kStream>(head + (u < nt ? u * V : 2 * half + (u - nt) * V), a);
        } else {
            st_vec<T, V, kStream>(head + first(u), a);
            st_vec<T, V, kStream>(head + second(u, half), b);
        }
    }
};

// Whether 16-byte vectors of `elem` bytes divide a head's parts.
inline bool vector_fits(int32_t half, int32_t interleaved, int32_t head_dim, int32_t elem) {
    const int v = 16 / elem;
    return (interleaved ? 2 * half : half) % v == 0 && head_dim % v == 0;
}

}  // namespace lmkv_rotary_detail
