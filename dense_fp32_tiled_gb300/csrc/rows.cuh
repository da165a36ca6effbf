// rows.cuh -- whole rows in the widest access that their addresses allow: the
// packs of values that kernels move, and the host's choice among them.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "linear.h"
#include "linear_types.cuh"

namespace rows {

using lt::from_f;
using lt::to_f;

// V values (16, 8, 4 or 2 bytes) of a row, as the word they travel in: a load
// that may not happen is then one predicated instruction, and the next ones
// follow it at once.
template <int BYTES>
struct Word;
template <>
struct Word<16> {
    using type = uint4;
};
template <>
struct Word<8> {
    using type = uint2;
};
template <>
struct Word<4> {
    using type = uint32_t;
};
template <>
struct Word<2> {
    using type = uint16_t;
};
template <typename T, int V>
struct Pack {
    static constexpr int BYTES = V * static_cast<int>(sizeof(T));
    using Raw = typename Word<BYTES>::type;
    Raw raw;
    __device__ __forceinline__ void clear() { raw = Raw{}; }
    __device__ __forceinline__ uint32_t word(int i) const {
        if constexpr (BYTES == 16) return i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w;
        if constexpr (BYTES == 8) return i == 0 ? raw.x : raw.y;
        if constexpr (BYTES <= 4) return raw;
    }
    __device__ __forceinline__ void get(float (&f)[V]) const {
        if constexpr (BYTES == 2) {
            f[0] = to_f(*reinterpret_cast<const T *>(&raw));
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = __uint_as_float(word(i));
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 v = lt::unpack2<T>(word(i));
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[V]) {
        if constexpr (BYTES == 2) {
            const T v = from_f<T>(f[0]);
            raw = *reinterpret_cast<const Raw *>(&v);
        } else {
            uint32_t w[BYTES / 4];
#pragma unroll
            for (int i = 0; i < BYTES / 4; ++i) {
                if constexpr (sizeof(T) == 4)
                    w[i] = __float_as_uint(f[i]);
                else
                    w[i] = lt::pack2<T>(f[2 * i], f[2 * i + 1]);
            }
            if constexpr (BYTES == 16) raw = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (BYTES == 8) raw = make_uint2(w[0], w[1]);
            if constexpr (BYTES == 4) raw = w[0];
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load(const T *p) {
    Pack<T, V> v;
    v.raw = *reinterpret_cast<const typename Pack<T, V>::Raw *>(p);
    return v;
}
// The values at p, or zeros.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_if(bool in, const T *p) {
    Pack<T, V> v;
    v.clear();
    if (in) v.raw = *reinterpret_cast<const typename Pack<T, V>::Raw *>(p);
    return v;
}
template <typename T, int V>
__device__ __forceinline__ void store(T *p, const Pack<T, V> &v) {
    *reinterpret_cast<typename Pack<T, V>::Raw *>(p) = v.raw;
}

// ---- two values at a time ------------------------------------------------------------
// FP32 arithmetic on pairs: one instruction for two, each rounded as by itself.  A pack of V values is V / 2 pairs, or one float.
using Pair = float2;
template <int V>
struct Lanes {
    using Num = Pair;
    static constexpr int N = V / 2;
};
template <>
struct Lanes<1> {
    using Num = float;
    static constexpr int N = 1;
};
__device__ __forceinline__ Pair add(Pair a, Pair b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ Pair mul(Pair a, Pair b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ Pair fma_of(Pair a, Pair b, Pair c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma_of(float a, float b, float c) { return fmaf(a, b, c); }
template <typename Num>
__device__ __forceinline__ Num all(float v) {
    if constexpr (sizeof(Num) == 8)
        return make_float2(v, v);
    else
        return v;
}
__device__ __forceinline__ float sum_of(Pair p) {
    return p.x + p.y;
}
__device__ __forceinline__ float sum_of(float v) { return v; }
template <typename T, int V>
__device__ __forceinline__ void get(const Pack<T, V> &p, typename Lanes<V>::Num (&f)[Lanes<V>::N]) {
    if constexpr (V == 1) {
        float v[1];
        p.get(v);
        f[0] = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (sizeof(T) == 4)
                f[i] = make_float2(__uint_as_float(p.word(2 * i)), __uint_as_float(p.word(2 * i + 1)));
            else if constexpr (std::is_same<T, __nv_bfloat16>::value)  // an instruction each
                f[i] = make_float2(__uint_as_float(p.word(i) << 16), __uint_as_float(p.word(i) & 0xffff0000u));
            else
                f[i] = lt::unpack2<T>(p.word(i));
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack_of(const typename Lanes<V>::Num (&f)[Lanes<V>::N]) {
    float v[V];
    if constexpr (V == 1) {
        v[0] = f[0];
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            v[2 * i] = f[i].x;
            v[2 * i + 1] = f[i].y;
        }
    }
    Pack<T, V> p;
    p.set(v);
    return p;
}
// The values at p, or ones.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_or_ones(bool in, const T *p) {
    if (in) return load<T, V>(p);
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 1.0f;
    Pack<T, V> o;
    o.set(v);
    return o;
}

// ---- host ----------------------------------------------------------------------------
struct Span {
    uintptr_t lo = 0, hi = 0;
};
inline Span span(const void *p, long long rows, long long width, long long ld, long long bytes) {
    Span s;
    if (p == nullptr || rows <= 0 || width <= 0) return s;
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + static_cast<uintptr_t>(((rows - 1) * ld + width) * bytes);
    return s;
}
inline bool overlap(const Span &a, const Span &b) { return a.lo < b.hi && b.lo < a.hi; }
inline bool misaligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// The widest access (16, 8, 4 or 2 bytes) that rows of this address and stride allow.
inline int width_of(const void *p, long long ld, int type) {
    if (p == nullptr) return 16;
    const unsigned long long bits = reinterpret_cast<uintptr_t>(p) | static_cast<unsigned long long>(ld) * lt::type_bytes(type) | 16;
    return static_cast<int>(bits & (0 - bits));
}
inline int narrower(int a, int b) { return a < b ? a : b; }
inline int launched(cudaError_t err) {
    if (err == cudaSuccess) return SGEMM_OK;
    (void)cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
}
// f(element, values per access) for the type and the bytes of an access.
template <typename F>
int with_rows(int type, int bytes, F &&f) {
    if (type == LINEAR_F32)
        return bytes == 16 ? f(float(), lt::Int<4>{}) : bytes == 8 ? f(float(), lt::Int<2>{}) : f(float(), lt::Int<1>{});
    auto half = [&](auto el) {
        return bytes == 16  ? f(el, lt::Int<8>{})
               : bytes == 8 ? f(el, lt::Int<4>{})
               : bytes == 4 ? f(el, lt::Int<2>{})
                            : f(el, lt::Int<1>{});
    };
    return type == LINEAR_BF16 ? half(__nv_bfloat16()) : half(__half());
}

}  // namespace rows
