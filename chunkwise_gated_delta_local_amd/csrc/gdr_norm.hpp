// Rows in 16-byte pieces, shared by the norms (gdr_norm.hip, gdr_block_norm.hip).
#pragma once

#include <type_traits>

#include "gdr_mixer.hpp"

namespace gdr {

// elements c .. c + V - 1 of a row of C, zero past its end
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ typename Raw<T, V>::type load_piece(const T* row, int c, int C) {
    typename Raw<T, V>::type r;
    if (c + V <= C) return load_raw<T, V, ONCE>(row + c);
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = c + v < C ? row[c + v] : to_t<T>(0.f);
    return r;
}
// a parameter's elements, which are T or fp32; `none` where there is no parameter
template <typename T, int V>
__device__ __forceinline__ void load_param(const void* p, int c, int C, int f32, float none, float (&f)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = none;
    if (!p || c >= C) return;
    if (f32) unpack<float, V>(load_piece<float, V>((const float*)p, c, C), f);
    else unpack<T, V>(load_piece<T, V>((const T*)p, c, C), f);
}
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void store_piece(T* row, int c, int C, const float (&f)[V]) {
    typename Raw<T, V>::type r;
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = to_t<T>(f[v]);
    if (c + V <= C) {
        store_raw<T, V, ONCE>(row + c, r);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c + v < C) row[c + v] = r[v];
    }
}

// V elements of a tensor that is fp32 or T, as they were read: the choice is the same
// for a whole launch, and the values are not looked at before they are unpacked, so
// that the loads of several tensors are on their way together.
typedef float f32x2 __attribute__((ext_vector_type(2)));
template <int V> struct AnyPiece {
    f32x4 x[V / 4];
};
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void load_any(AnyPiece<V>& r, const void* p, int64_t row, int c, int C, int f32) {
    if (sizeof(T) == 4 || f32) {
        const float* q = (const float*)p + row;
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            if (c + i < C) r.x[i / 4] = load_piece<float, 4, ONCE>(q, c + i, C);
            else r.x[i / 4] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    } else if constexpr (sizeof(T) == 2) {
        typedef typename Raw<T, V>::type raw;
        const raw x = load_piece<T, V, ONCE>((const T*)p + row, c, C);
        if constexpr (sizeof(raw) == 16) r.x[0] = __builtin_bit_cast(f32x4, x);
        else r.x[0] = __builtin_shufflevector(__builtin_bit_cast(f32x2, x), f32x2{}, 0, 1, 2, 3);
    }
}
template <typename T, int V>
__device__ __forceinline__ void unpack_any(const AnyPiece<V>& r, int f32, float (&f)[V]) {
    if (sizeof(T) == 4 || f32) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = r.x[i / 4][i % 4];
    } else if constexpr (sizeof(T) == 2) {
        typedef typename Raw<T, V>::type raw;
        if constexpr (sizeof(raw) == 16) unpack<T, V>(__builtin_bit_cast(raw, r.x[0]), f);
        else unpack<T, V>(__builtin_bit_cast(raw, __builtin_shufflevector(r.x[0], r.x[0], 0, 1)), f);
    }
}
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void store_any(void* p, int64_t row, int c, int C, int f32, const float (&f)[V]) {
    if (sizeof(T) == 4 || f32) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float g[4] = {f[i], f[i + 1], f[i + 2], f[i + 3]};
            if (c + i < C) store_piece<float, 4, ONCE>((float*)p + row, c + i, C, g);
        }
    } else if constexpr (sizeof(T) == 2) {
        store_piece<T, V, ONCE>((T*)p + row, c, C, f);
    }
}

}  // namespace gdr
