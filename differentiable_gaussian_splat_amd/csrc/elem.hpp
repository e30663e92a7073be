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

// V consecutive elements; V is 1 or WIDE<T> (then p is 16-byte aligned).
template <int V>
__device__ __forceinline__ void load_row(const float* p, float (&v)[V]) {
    if constexpr (V == 4) {
        const float4 t = *reinterpret_cast<const float4*>(p);
        v[0] = t.x;
        v[1] = t.y;
        v[2] = t.z;
        v[3] = t.w;
    } else {
        static_assert(V == 1, "");
        v[0] = *p;
    }
}

template <int V>
__device__ __forceinline__ void load_row(const bf16* p, float (&v)[V]) {
    if constexpr (V == 8) {
        const bf16x8 t = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)t[i];
    } else {
        static_assert(V == 1, "");
        v[0] = (float)*p;
    }
}

template <int V>
__device__ __forceinline__ void store_row(float* p, const float (&v)[V]) {
    if constexpr (V == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        static_assert(V == 1, "");
        *p = v[0];
    }
}

template <int V>
__device__ __forceinline__ void store_row(bf16* p, const float (&v)[V]) {
    if constexpr (V == 8) {
        bf16x8 t;
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = (bf16)v[i];
        *reinterpret_cast<bf16x8*>(p) = t;
    } else {
        static_assert(V == 1, "");
        *p = (bf16)v[0];
    }
}

// Row i of a table index array (int32, or int64 with `wide`), or -1 where it
// names none of the `rows` rows.
__device__ __forceinline__ int row_index(const void* ids, bool wide, int64_t i, int rows) {
    const int64_t v = wide ? static_cast<const int64_t*>(ids)[i] : (int64_t)static_cast<const int32_t*>(ids)[i];
    return v >= 0 && v < rows ? (int)v : -1;
}

// Whether rows of `dim` elements at p, `stride` apart, can be read 16 bytes at a time.
template <class T>
inline bool wide_rows(const void* p, int64_t stride, int dim) {
    return p == nullptr || ((uintptr_t)p % 16 == 0 && stride % WIDE<T> == 0 && dim % WIDE<T> == 0);
}

}  // namespace gs
