// Rows in 8 bits: e4m3 values with a power of two for each row and block of 128
// columns.
//
//   e = the least with max |v| <= 448 2^e over the block's finite values
//       (0 where all are 0; -126 at least),   q = v / 2^e in e4m3, to nearest even
//
// A floating-point format loses nothing by the scale being a power of two: the
// quotients keep their bits, and only what falls below e4m3's smallest normal
// number depends on the scale at all. So the matrix units can apply it (they take
// an 8-bit exponent per row and 32 columns of either operand), and products need
// no arithmetic beside theirs. Infinities and NaN become e4m3's NaN: a score that
// one of them enters is no number.
//
// Memory: values [n][cols], cols = dim rounded up to 128, zero from dim on; scales
// [n][groups], the exponents plus 127, groups = cols / 128 rounded up to 4, of
// which those past the blocks are 127.
#pragma once

#include "elem.hpp"

namespace gs {

constexpr int Q8_BLOCK = 128;

__host__ __device__ constexpr int q8_cols(int dim) { return (dim + Q8_BLOCK - 1) / Q8_BLOCK * Q8_BLOCK; }
__host__ __device__ constexpr int q8_groups(int dim) { return (q8_cols(dim) / Q8_BLOCK + 3) / 4 * 4; }

// Lanes that share a block where each holds an access of T.
template <class T>
constexpr int Q8_LANES = Q8_BLOCK / WIDE<T>;

// The magnitude that counts for the scale: 0 for infinities and NaN.
__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < INFINITY ? a : 0.f;
}

// The biased exponent (1 to 247) of the scale for a largest magnitude: 448 is 1.75 2^8.
__device__ __forceinline__ int scale_exponent(float top) {
    const uint32_t u = __float_as_uint(top);
    const int e = (int)((u + 0x1fffffu) >> 23) - 8;
    return u == 0 ? 127 : e < 1 ? 1 : e;
}

// 2^-(e - 127)
__device__ __forceinline__ float scale_inverse(int e) { return __uint_as_float((uint32_t)(254 - e) << 23); }

// Four values over the scale in e4m3, the first in the lowest byte.
__device__ __forceinline__ uint32_t pack_q8(const float* v, float inverse) {
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        q[k] = v[k] * inverse;
        q[k] = fabsf(q[k]) < INFINITY ? q[k] : __builtin_nanf("");
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
}

// Stores an access's values (4 float32 or 8 bfloat16 as float32) in e4m3.
__device__ __forceinline__ void store_q8(uint8_t* p, const float (&v)[4], float inverse) {
    *reinterpret_cast<uint32_t*>(p) = pack_q8(v, inverse);
}
__device__ __forceinline__ void store_q8(uint8_t* p, const float (&v)[8], float inverse) {
    uint2 w;
    w.x = pack_q8(v, inverse);
    w.y = pack_q8(v + 4, inverse);
    *reinterpret_cast<uint2*>(p) = w;
}

}  // namespace gs
