// Scores of rows in 8 bits against a vocabulary in 8 bits (rows8.hpp):
//
//   out[i][v] = sum over blocks b of 2^(ea_ib + ew_vb) sum_{k in b} a_ik w_vk
//
// on the matrix units. Which of their products is taken goes by the result's type:
//   bfloat16  e4m3 operands with an 8-bit exponent per row and 32 columns. The sums
//             are float32, but of eight columns' products beside each other each is
//             cut off at 2^-13 of the largest's power of two before they are added
//             (seen by products of single powers of two), which leaves 1.4e-5 of a
//             score's size on normal data: nothing beside the result's own rounding.
//   float32   the operands widened to bfloat16 with their scale, which is exact, and
//             bfloat16 products, at less than a third of the rate: 1.4e-8 to 2e-7.
// The vocabulary's rows stand for the rows of a unit's tile and the features for its
// columns, so that a lane holds runs of one feature row's scores; which vocabulary
// row stands in which row of the tile is chosen so that a lane's runs join.
#include <type_traits>

#include "launch.hpp"
#include "rows8.hpp"

namespace gs {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Stores C scores from out on, `left` of them in the row (out is aligned to its elements only).
template <int C>
__device__ __forceinline__ void store_scores(float* out, int64_t left, const float (&v)[C]) {
#pragma unroll
    for (int c = 0; c < C; c += 4) {
        if (left >= c + 4) {
            wide_any<float> t;
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = v[c + k];
            *reinterpret_cast<wide_any<float>*>(out + c) = t;
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (c + k < left) out[c + k] = v[c + k];
        }
    }
}

template <int C>
__device__ __forceinline__ void store_scores(bf16* out, int64_t left, const float (&v)[C]) {
    constexpr int S = C < 8 ? C : 8;
    typedef bf16 run __attribute__((ext_vector_type(S)));
    typedef bf16 run_any __attribute__((ext_vector_type(S), aligned(2)));
#pragma unroll
    for (int c = 0; c < C; c += S) {
        if (left >= c + S) {
            run t;
#pragma unroll
            for (int k = 0; k < S; ++k) t[k] = (bf16)v[c + k];
            *reinterpret_cast<run_any*>(out + c) = t;
        } else {
#pragma unroll
            for (int k = 0; k < S - 1; ++k)
                if (c + k < left) out[c + k] = (bf16)v[c + k];
        }
    }
}

// 32 bytes of a lane's row: the two halves of a 128-byte block, 16 bytes of each.
__device__ __forceinline__ i32x8 block_of(const uint8_t* row) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(row), hi = *reinterpret_cast<const i32x4*>(row + 64);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Block B of four blocks' scales, as a number.
template <int B>
__device__ __forceinline__ float scale_of(int four) {
    return __uint_as_float((uint32_t)((four >> (8 * B)) & 255) << 23);
}

// Eight of a lane's values (words 2 s and 2 s + 1) times their scale in bfloat16.
__device__ __forceinline__ bf16x8 widen8(const i32x8& q, int s, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * s], scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * s], scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * s + 1], scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * s + 1], scale, true);
    bf16x8 v;
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
    return v;
}

// Straight from memory to registers: a wave takes 16 XT feature rows and 16 VT vocabulary rows over its share of the
// depth (every KS-th four blocks); the KS waves of a tile join their sums in LDS.
template <class T, int XT, int VT, int KS>
__global__ __launch_bounds__(256) void k_scores_direct(ScoreArgs a) {
    constexpr int VW = 4 / KS;  // tiles side by side
    __shared__ float s_join[KS > 1 ? VW * (KS - 1) * XT * VT * 256 : 1];
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int share = w % KS, side = w / KS;
    const int64_t x0 = (int64_t)blockIdx.y * (16 * XT), v0 = ((int64_t)blockIdx.x * VW + side) * (16 * VT);
    const int blocks = a.cols / Q8_BLOCK, fours = (blocks + 3) / 4;
    const uint8_t *xp[XT], *vp[VT], *xs[XT], *vs[VT];
#pragma unroll
    for (int i = 0; i < XT; ++i) {
        const int64_t r = min(x0 + 16 * i + l % 16, a.n - 1);
        xp[i] = a.q + r * a.qs + (l / 16) * 16;
        xs[i] = a.qscales + r * a.qss;
    }
#pragma unroll
    for (int j = 0; j < VT; ++j) {
        const int m = l % 16;
        const int64_t r = min(v0 + (m / 4) * (4 * VT) + 4 * j + m % 4, a.vocab - 1);
        vp[j] = a.w + r * a.ws + (l / 16) * 16;
        vs[j] = a.wscales + r * a.wss;
    }
    f32x4 acc[XT][VT];
#pragma unroll
    for (int i = 0; i < XT; ++i)
#pragma unroll
        for (int j = 0; j < VT; ++j) acc[i][j] = 0.f;
    for (int f = share; f < fours; f += KS) {
        int sx[XT], sv[VT];
#pragma unroll
        for (int i = 0; i < XT; ++i) sx[i] = *reinterpret_cast<const int*>(xs[i] + 4 * f);
#pragma unroll
        for (int j = 0; j < VT; ++j) sv[j] = *reinterpret_cast<const int*>(vs[j] + 4 * f);
        auto block = [&](auto which) {
            constexpr int B = decltype(which)::value;
            if (4 * f + B >= blocks) return;
            const int64_t at = (int64_t)(4 * f + B) * Q8_BLOCK;
            i32x8 fx[XT], fv[VT];
#pragma unroll
            for (int i = 0; i < XT; ++i) fx[i] = block_of(xp[i] + at);
#pragma unroll
            for (int j = 0; j < VT; ++j) fv[j] = block_of(vp[j] + at);
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < XT; ++i)
#pragma unroll
                    for (int j = 0; j < VT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fv[j], fx[i], acc[i][j], 0, 0, B,
                                                                                   sv[j], B, sx[i]);
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    bf16x8 hx[XT], hv[VT];
#pragma unroll
                    for (int i = 0; i < XT; ++i) hx[i] = widen8(fx[i], s, scale_of<B>(sx[i]));
#pragma unroll
                    for (int j = 0; j < VT; ++j) hv[j] = widen8(fv[j], s, scale_of<B>(sv[j]));
#pragma unroll
                    for (int i = 0; i < XT; ++i)
#pragma unroll
                        for (int j = 0; j < VT; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hv[j], hx[i], acc[i][j], 0, 0, 0);
                }
            }
        };
        block(std::integral_constant<int, 0>{});
        block(std::integral_constant<int, 1>{});
        block(std::integral_constant<int, 2>{});
        block(std::integral_constant<int, 3>{});
    }
    if constexpr (KS > 1) {
        float* s = s_join + side * (KS - 1) * XT * VT * 256;
        if (share > 0) {
#pragma unroll
            for (int i = 0; i < XT; ++i)
#pragma unroll
                for (int j = 0; j < VT; ++j)
                    *reinterpret_cast<f32x4*>(s + (((share - 1) * XT + i) * VT + j) * 256 + l * 4) = acc[i][j];
        }
        __syncthreads();
        if (share > 0) return;
#pragma unroll
        for (int k = 0; k < KS - 1; ++k)
#pragma unroll
            for (int i = 0; i < XT; ++i)
#pragma unroll
                for (int j = 0; j < VT; ++j)
                    acc[i][j] += *reinterpret_cast<const f32x4*>(s + ((k * XT + i) * VT + j) * 256 + l * 4);
    }
    const int64_t v = v0 + (l / 16) * (4 * VT);
#pragma unroll
    for (int i = 0; i < XT; ++i) {
        const int64_t r = x0 + 16 * i + l % 16;
        if (r >= a.n || v >= a.vocab) continue;
        float t[4 * VT];
#pragma unroll
        for (int j = 0; j < VT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) t[4 * j + k] = acc[i][j][k];
        store_scores((T*)a.out + r * a.os + v, a.vocab - v, t);
    }
}

template <class T, int XT, int VT, int KS>
hipError_t scores_direct(const ScoreArgs& a, hipStream_t s) {
    const int64_t per = 16 * VT * (4 / KS);
    const int64_t bx = (a.vocab + per - 1) / per;
    // a grid's second axis holds 65535 blocks
    const int64_t most = (int64_t)65535 * 16 * XT;
    for (int64_t r = 0; r < a.n; r += most) {
        ScoreArgs p = a;
        p.n = a.n - r < most ? a.n - r : most;
        p.q += r * a.qs;
        p.qscales += r * a.qss;
        p.out = (T*)a.out + r * a.os;
        const dim3 grid((unsigned)bx, (unsigned)((p.n + 16 * XT - 1) / (16 * XT)));
        k_scores_direct<T, XT, VT, KS><<<grid, 256, 0, s>>>(p);
        if (hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

template <class T>
hipError_t scores(const ScoreArgs& a, hipStream_t s) {
    return scores_direct<T, 2, 2, 1>(a, s);
}

}  // namespace

hipError_t launch_label_scores(const ScoreArgs& a, hipStream_t stream) {
    return a.half ? scores<bf16>(a, stream) : scores<float>(a, stream);
}

}  // namespace gs
