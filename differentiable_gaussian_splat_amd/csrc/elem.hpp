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
template <class T>
using wide_t = T __attribute__((ext_vector_type(WIDE<T>)));
template <class T>
using wide_any = T __attribute__((ext_vector_type(WIDE<T>), aligned(sizeof(T))));

// The WIDE<T> elements of a row at p, as they are in memory. left: of them
// inside the row; room: from p to the end of the matrix. Where the room is
// enough the access may reach behind the row; what it finds there is masked by
// `widen` or `clip`, so that a row's end costs no branch (only the matrix's
// last elements do). Masked later and not here, where it would wait for the
// load. FULL: the row is whole accesses, and none of this is looked at.
template <bool FULL, class T>
__device__ __forceinline__ wide_t<T> load_row(const T* p, int left, int64_t room) {
    wide_t<T> t;
    if (FULL || room >= WIDE<T>) {
        t = *reinterpret_cast<const wide_any<T>*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < WIDE<T>; ++i) t[i] = i < left ? p[i] : (T)0.f;
    }
    return t;
}

template <bool FULL, class T>
__device__ __forceinline__ wide_t<T> clip(wide_t<T> t, int left) {
#pragma unroll
    for (int i = 0; i < WIDE<T>; ++i) t[i] = FULL || i < left ? t[i] : (T)0.f;
    return t;
}

template <bool FULL, class T, int V>
__device__ __forceinline__ void widen(wide_t<T> t, int left, float (&v)[V]) {
    static_assert(V == WIDE<T>, "");
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = FULL || i < left ? (float)t[i] : 0.f;
}

// Stores the first `left` (FULL: all) of WIDE<T> elements.
template <bool FULL>
__device__ __forceinline__ void store_row(float* p, int left, const float (&v)[4]) {
    if (FULL || left >= 4) {
        wide_any<float> t;
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = v[i];
        *reinterpret_cast<wide_any<float>*>(p) = t;
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < left) p[i] = v[i];
    }
}

template <bool FULL>
__device__ __forceinline__ void store_row(bf16* p, int left, const float (&v)[8]) {
    if (FULL || left >= 8) {
        wide_any<bf16> t;
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = (bf16)v[i];
        *reinterpret_cast<wide_any<bf16>*>(p) = t;
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
