// Element types of the label-learning operators (embed.hip, norm.hip,
// labelloss.hip): float32 and bfloat16 rows, widened to float32 in registers
// and rounded once (to nearest even) where a result is stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gs {

using bf16 = __bf16;
typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Elements of one 16-byte access.
template <class T>
constexpr int WIDE = 16 / (int)sizeof(T);

// 16 bytes at an address that is aligned to the element only: gfx950 takes
// 16-byte global accesses at any address, so rows of odd lengths and strides
// need no narrower ones.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef bf16 bf16x8_any __attribute__((ext_vector_type(8), aligned(2)));

// The WIDE<T> elements of a row at p, of which `left` are inside the row (the
// others read as 0). FULL: the row is whole accesses (left is not looked at).
// room: elements from p to the end of the matrix. Where that is enough the
// access may reach behind the row, and what it finds there is masked, so that
// a row's end costs no branch; only the matrix's last elements take one.
template <bool FULL>
__device__ __forceinline__ void load_row(const float* p, int left, int64_t room, float (&v)[4]) {
    if (FULL || room >= 4) {
        const f32x4_any t = *reinterpret_cast<const f32x4_any*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = FULL || i < left ? t[i] : 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < left ? p[i] : 0.f;
    }
}

template <bool FULL>
__device__ __forceinline__ void load_row(const bf16* p, int left, int64_t room, float (&v)[8]) {
    if (FULL || room >= 8) {
        const bf16x8_any t = *reinterpret_cast<const bf16x8_any*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = FULL || i < left ? (float)t[i] : 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? (float)p[i] : 0.f;
    }
}

// Stores the first `left` (FULL: all) of WIDE<T> elements.
template <bool FULL>
__device__ __forceinline__ void store_row(float* p, int left, const float (&v)[4]) {
    if (FULL || left >= 4) {
        f32x4_any t;
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = v[i];
        *reinterpret_cast<f32x4_any*>(p) = t;
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < left) p[i] = v[i];
    }
}

template <bool FULL>
__device__ __forceinline__ void store_row(bf16* p, int left, const float (&v)[8]) {
    if (FULL || left >= 8) {
        bf16x8_any t;
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = (bf16)v[i];
        *reinterpret_cast<bf16x8_any*>(p) = t;
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < left) p[i] = (bf16)v[i];
    }
}

// Row i of a table index array (int32, or int64 with `wide`), or -1 where it
// names none of the `rows` rows.
__device__ __forceinline__ int row_index(const void* ids, bool wide, int64_t i, int rows) {
    const int64_t v = wide ? static_cast<const int64_t*>(ids)[i] : (int64_t)static_cast<const int32_t*>(ids)[i];
    return v >= 0 && v < rows ? (int)v : -1;
}

}  // namespace gs
