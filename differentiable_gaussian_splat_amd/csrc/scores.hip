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
//             Of large products that cancel, small ones among the same eight are lost:
//             a choice for up to 1.8 times the speed, which the caller makes with the type.
//   float32   the operands widened to bfloat16 with their scale, and bfloat16
//             products, at less than a third of the rate: 1.4e-8 to 2e-7. The widening
//             is exact for scales of 2^-111 to 2^112. A wave that meets others takes
//             the 8-bit products for them, one of each eight columns at a time: there
//             is nothing beside it then that a product could be cut off by.
#include <type_traits>

#include "launch.hpp"
#include "rows8.hpp"

namespace gs {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
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

// Whether one of a lane's four scales, of `used` blocks of columns, is too far from 1 for widen8. With a byte of 16 to
// 239 the least value times its scale (2^-9 2^-111) and the greatest (448 2^112) are normal bfloat16 numbers.
__device__ __forceinline__ bool far_scales(int four, int used) {
    const uint32_t in = used >= 4 ? ~0u : (1u << (8 * used)) - 1;
    const uint32_t s = ((uint32_t)four & in) | (0x7f7f7f7fu & ~in);
    // a byte's upper half is 0 or 15: one more, it is 0 but for its lowest bit (and the 16)
    const uint32_t near = (((s >> 4) & 0x0f0f0f0fu) + 0x01010101u) & 0x0e0e0e0eu;
    return (near - 0x01010101u) & 0x80808080u;
}

// Of a lane's values those in place m of each eight, zeros in the others' places.
__device__ __forceinline__ i32x8 one_of_eight(const i32x8& q, int m) {
    const int byte = 0xff << (8 * (m & 3)), even = m < 4 ? byte : 0, odd = m < 4 ? 0 : byte;
    i32x8 v;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = q[k] & (k % 2 ? odd : even);
    return v;
}

constexpr int DIRECT_WAVES = 8;  // of a block

// Straight from memory to registers: a wave takes 16 XT feature rows and 16 VT vocabulary rows over its share of the
// depth (every KS-th four blocks); the KS waves of a tile join their sums in LDS. The vocabulary's rows stand for the
// rows of a unit's tile and the features for its columns, so that a lane holds runs of one feature row's scores; which
// vocabulary row stands in which row of the tile is chosen so that a lane's runs join.
template <class T, int XT, int VT, int KS>
__global__ __launch_bounds__(64 * DIRECT_WAVES) void k_scores_direct(ScoreArgs a) {
    constexpr int VW = DIRECT_WAVES / KS;  // tiles side by side
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
        bool far = false;  // float32: whether a scale is, of this wave's and these four blocks
        auto block = [&](auto which) {
            constexpr int B = decltype(which)::value;
            if (4 * f + B >= blocks) return;
            const int64_t at = (int64_t)(4 * f + B) * Q8_BLOCK;
            i32x8 fx[XT], fv[VT];
#pragma unroll
            for (int i = 0; i < XT; ++i) fx[i] = block_of(xp[i] + at);
#pragma unroll
            for (int j = 0; j < VT; ++j) fv[j] = block_of(vp[j] + at);
            auto product = [&](const i32x8& x, int i, int j) {
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fv[j], x, acc[i][j], 0, 0, B, sv[j], B,
                                                                           sx[i]);
            };
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < XT; ++i)
#pragma unroll
                    for (int j = 0; j < VT; ++j) product(fx[i], i, j);
            } else {
                if (B == 0) {  // behind the first block's loads, which do not wait for it
#pragma unroll
                    for (int i = 0; i < XT; ++i) far |= far_scales(sx[i], blocks - 4 * f);
#pragma unroll
                    for (int j = 0; j < VT; ++j) far |= far_scales(sv[j], blocks - 4 * f);
                    far = __ballot(far) != 0;
                }
                if (far) {
#pragma unroll 1
                    for (int m = 0; m < 8; ++m)
#pragma unroll
                        for (int i = 0; i < XT; ++i) {
                            const i32x8 one = one_of_eight(fx[i], m);
#pragma unroll
                            for (int j = 0; j < VT; ++j) product(one, i, j);
                        }
                    return;
                }
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
#pragma unroll 1
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
    const int64_t per = 16 * VT * (DIRECT_WAVES / KS);
    // the rules of `scores` send no more than 12160 rows here: a grid's second axis holds 65535 blocks
    const dim3 grid((unsigned)((a.vocab + per - 1) / per), (unsigned)((a.n + 16 * XT - 1) / (16 * XT)));
    k_scores_direct<T, XT, VT, KS><<<grid, 64 * DIRECT_WAVES, 0, s>>>(a);
    return hipGetLastError();
}

// The depth is split over as many of a block's waves as it takes to have two to a SIMD, and as there are four blocks of
// columns (LEAST: so many at least, as the caller has seen).
template <class T, int XT, int VT, int LEAST>
hipError_t scores_split(const ScoreArgs& a, hipStream_t s) {
    const int64_t tiles = ((a.n + 16 * XT - 1) / (16 * XT)) * ((a.vocab + 16 * VT - 1) / (16 * VT));
    const int fours = (a.cols / Q8_BLOCK + 3) / 4;
    int ks = LEAST;
    while (ks < DIRECT_WAVES && ks < fours && tiles * ks < 2048) ks *= 2;
    if constexpr (LEAST == 1) {
        if (ks == 1) return scores_direct<T, XT, VT, 1>(a, s);
        if (ks == 2) return scores_direct<T, XT, VT, 2>(a, s);
    }
    if (ks == 4) return scores_direct<T, XT, VT, 4>(a, s);
    return scores_direct<T, XT, VT, 8>(a, s);
}

// ------------------------------------------------------------------ tiles through LDS

constexpr int STEP = 64;     // columns of a staged step: one e4m3 product deep, half a block
constexpr int GROUP_X = 4;   // rows of tiles that follow one another along the vocabulary

// How a row's four 16-byte chunks are exchanged, so that the sixteen lanes that read one depth's chunks together find
// them spread over all banks.
__device__ __forceinline__ int chunk_turn(int r) { return (r >> 2) & 3; }

// The vocabulary row (of a block's) that stands in row s of its tiles: column c of a wave's tile j is its VT c + j, so
// that a lane's scores in a row join, and the 32 lanes of a row write without gaps. (Runs of a lane's own, 16 bytes at
// a time with other lanes' between them, cost four times the requests: 8192 x 128 x 65536 437 us, so 287.)
template <int VT>
__device__ __forceinline__ int vocab_row(int s) {
    return s / (32 * VT) * (32 * VT) + s % 32 * VT + s / 32 % VT;
}

// Where a tile's scores go, said to be global memory: through a pointer of any memory they would be flat accesses,
// which LDS waits count too, and which end in no said order with the loads beside them.
template <class T>
using scores_at = T __attribute__((address_space(1)))*;

// Stores C scores side by side (out is aligned to its elements only). PAST: past the caches, which the operands need.
template <bool PAST, class T, int C>
__device__ __forceinline__ void store_run(scores_at<T> out, const float (&v)[C]) {
    typedef T run __attribute__((ext_vector_type(C)));
    typedef T run_any __attribute__((ext_vector_type(C), aligned(sizeof(T))));
    run t;
#pragma unroll
    for (int c = 0; c < C; ++c) t[c] = (T)v[c];
    if (PAST)
        __builtin_nontemporal_store(t, (scores_at<run_any>)out);
    else
        *(scores_at<run_any>)out = t;
}

// A descriptor of `bytes` bytes from p on; reads beyond them give 0. (A step's offset, which is added to a lane's,
// stays below `bytes`, and a lane's own lies beyond them for every row past the last.)
__device__ __forceinline__ i32x4 extent(const uint8_t* p, int bytes) {
    const uint64_t at = (uint64_t)p;
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)at);
    r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32)) & 0xffff;
    r[2] = __builtin_amdgcn_readfirstlane(bytes);
    r[3] = 0x00020000;
    return r;
}

// Loads straight to LDS: lane l's 16 bytes at off + step (4 bytes at from) go to lds + 16 l (4 l). They write no
// register, so that nothing of them is the compiler's to keep: step_barrier waits for their arrival. The wait state is
// what a write of m0 needs before them; those that a vector write of the descriptor needs are settle's.
__device__ __forceinline__ void load_lds16(uint32_t lds, uint32_t off, i32x4 from, int step) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(off),
                 "s"(from), "s"(step)
                 : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(uint32_t lds, const uint8_t* from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(from) : "memory", "m0");
}
__device__ __forceinline__ void settle(i32x4& a, i32x4& b) { asm volatile("s_nop 4" : "+s"(a), "+s"(b)); }

// Waits until all but the last LEFT of this wave's memory accesses are done and its LDS reads too, then for the block.
template <int LEFT>
__device__ __forceinline__ void step_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// A wave's part of a tile in which a scale is far from 1, again from memory, by one of eight columns at a time: feature
// rows from x0 on, 32 rows of them each, against the rows of the vocabulary's tile at v0 that stand from s0 on. 32 x 32
// scores at a time, which need few registers: next to the tile's next operands there are no more. (Every tile so:
// 8192 x 1024 x 8192 833 us, with near scales 129; 5003 x 256 x 8191 127, 38. Straight from memory 5 to 15 % more.)
template <int VT, class Args>
__device__ __forceinline__ void far_tile(const Args& a, int x0, int rows, int v0, int s0) {
    const int l = threadIdx.x & 63;
    const int cols = a.cols;
#pragma unroll 1
    for (int t = 0; t < rows * VT; ++t) {
        const int x = x0 + t / VT * 32, v = v0 + vocab_row<VT>(s0 + t % VT * 32 + l % 32);
        const int64_t xr = min(x + l % 32, (int)a.n - 1), vr = min(v, (int)a.vocab - 1);
        const uint8_t *q = a.q + xr * a.qs + l / 32 * 32, *w = a.w + vr * a.ws + l / 32 * 32;
        const uint8_t *qs = a.qscales + xr * a.qss, *ws = a.wscales + vr * a.wss;
        f32x16 c;
#pragma unroll
        for (int e = 0; e < 16; ++e) c[e] = 0.f;
#pragma unroll 1
        for (int k = 0; k < cols; k += STEP) {
            const auto at = [&](const uint8_t* p) {
                const i32x4 lo = *reinterpret_cast<const i32x4*>(p + k);
                const i32x4 hi = *reinterpret_cast<const i32x4*>(p + k + 16);
                return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            };
            const i32x8 fx = at(q), fv = at(w);
            const int sx = qs[k / Q8_BLOCK], sv = ws[k / Q8_BLOCK];
#pragma unroll 1
            for (int m = 0; m < 8; ++m)
                c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(one_of_eight(fx, m), fv, c, 0, 0, 0, sx, 0, sv);
        }
        if (v < a.vocab) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int r = x + 4 * (l / 32) + 8 * (e / 4) + e % 4;
                if (r < a.n) ((scores_at<float>)a.out)[r * a.os + v] = c[e];
            }
        }
    }
}

// Tiles of 32 XT WX feature rows and 32 VT WV vocabulary rows by WX x WV waves. Blocks stay: each goes through its
// tiles' steps as one sequence, in which the loads run ahead over the tiles' ends and the scores of one tile are
// written while the next one's operands arrive.
//
// STAGES steps are in LDS. In step s a wave multiplies the operands it holds, reads those of step s + 1 from LDS and
// loads step s + STAGES into the place of step s. A barrier a step both publishes the arrived step and frees the one
// before it. Loads past the last step are made all the same, which keeps their count per step. Memory accesses are
// counted off in order: LOADS to a step, and behind a whole tile's last step its STORES, which the two steps after it
// let pass. (The scales' loads, one to four blocks of columns, are counted with nothing: a wait is then for a little
// more, never for less.)
//
// 8192 x 8192 x 8192 bfloat16 430 to 455 us (2.4 to 2.55 PFLOP/s): the units are busy 73 % of the cycles, at 1.7 GHz
// of 2.4: it is power that bounds them (products alone, from registers, reach 3.8). LDS is read without bank
// conflicts. With the step's reads and loads all behind its barrier 524; with a descriptor formed for each load
// 30 % more. Four waves of 128 x 128 with a third less to read from LDS 458 where eight had 441.
// 8192 x 1024 x 65536 bfloat16 530 to 625 us: a gigabyte of scores beside it, which alone takes 225. The stores stand
// in the same queue as the loads and hold them up (units busy 49 to 59 % of the cycles, at 1.9 to 1.4 GHz); past the
// caches they take 90 us less than through them. Blocks that start a part of a tile's time apart gain 3 % of it, and
// lose 10 % where tiles are deep.
template <class T, int WX, int WV, int XT, int VT, int STAGES>
__global__ __launch_bounds__(64 * WX * WV, 8 / (WX * WV)) void k_scores_tiles(ScoreArgs a, int tiles_x, int tiles_v) {
    constexpr int NW = WX * WV, BX = 32 * XT * WX, BV = 32 * VT * WV, ROWS = BX + BV;
    constexpr int LOADS = ROWS / 16 / NW;          // of 16 rows each, per wave and step
    constexpr int STORES = XT * 16;                // of VT scores, per lane and whole tile
    // (float32 by 256 x 256 lets none pass: two ways into a tile, and its widened operands, do not fit the registers.)
    constexpr bool LET = sizeof(T) == 2 || XT * VT < 8;
    static_assert(ROWS % (16 * NW) == 0 && BX % (16 * NW) == 0 && BX % 64 == 0, "");
    static_assert((STAGES - 2) * LOADS + STORES < 64 && (STAGES - 1) * LOADS < 64, "what a wait can count");
    __shared__ alignas(1024) uint8_t s_rows[STAGES * ROWS * STEP];
    __shared__ alignas(1024) int s_scales[4 * ROWS];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
    const uint32_t rows0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)s_rows;
    const uint32_t scales0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)s_scales;

    // Consecutive blocks go to the eight dies in turn: each die takes a run of tiles, in groups of GROUP_X rows of
    // them, so that its cache serves both operands. A block's places in the order are apart by a constant.
    const int tiles = tiles_x * tiles_v;
    const int die = blockIdx.x & 7, slots = gridDim.x >> 3;
    const int first = (int)((int64_t)tiles * die / 8) + (int)(blockIdx.x >> 3);
    const int last = (int)((int64_t)tiles * (die + 1) / 8);
    const int mine = first < last ? (last - first + slots - 1) / slots : 0;
    if (mine == 0) return;
    const int nk = a.cols / STEP;
    // the arguments read again where they are used once a tile: kept over the steps they would not fit the registers
    auto again = []() {
        auto p = (const __attribute__((address_space(4))) ScoreArgs*)__builtin_amdgcn_kernarg_segment_ptr();
        asm volatile("" : "+s"(p));
        return p;
    };
    struct Place {
        int group, in;
    };
    auto advance = [&](Place& p) {
        p.in += slots;
        while (p.in >= GROUP_X * tiles_v) {
            p.in -= GROUP_X * tiles_v;
            ++p.group;
        }
    };
    auto corner = [&](const Place& p, int& x0, int& v0) {
        const int rows = min(GROUP_X, tiles_x - p.group * GROUP_X);
        const int third = (int)__umulhi((uint32_t)p.in, 0x55555556u);
        const int v = rows == 4 ? p.in >> 2 : rows == 3 ? third : p.in >> (rows - 1);
        x0 = (p.group * GROUP_X + p.in - v * rows) * BX;
        v0 = v * BV;
    };
    static_assert(GROUP_X == 4, "the divisions by a group's rows");

    // what this lane loads first: a quarter of a row's step of either operand (then of rows apart by multiples of
    // NW * 16, which turns no chunks and keeps the order of the vocabulary's rows apart from the lane's)
    static_assert(NW * 16 % 32 == 0 && (VT % (NW / 2) == 0 || NW / 2 % VT == 0), "");
    const int row = w * 16 + l / 4, chunk = ((l % 4) ^ chunk_turn(row)) * 16;
    int off_x = row * (int)a.qs + chunk, off_v = vocab_row<VT>(row) * (int)a.ws + chunk;

    // the tile to load next: its place and corner, its rows; the step in it and its places in LDS
    Place load_place{first / (GROUP_X * tiles_v), first % (GROUP_X * tiles_v)}, place = load_place;
    int load_tile = 0, load_k = 0, load_at = 0, load_four = 0, load_x = 0, load_v = 0;
    i32x4 from_x, from_v;
    auto turn = [&](i32x4& to_x, i32x4& to_v) {
        load_x = load_v = 0;  // past the last tile the first one of all again, which nothing reads
        if (load_tile < mine) corner(load_place, load_x, load_v);
        const auto* p = again();
        to_x = extent(p->q + load_x * p->qs, (min(BX, (int)p->n - load_x) - 1) * (int)p->qs + p->cols);
        to_v = extent(p->w + load_v * p->ws, (min(BV, (int)p->vocab - load_v) - 1) * (int)p->ws + p->cols);
        settle(to_x, to_v);
    };
    auto issue_scales = [&](int k) {  // where four blocks of columns begin, ahead of their values
        if ((k & 7) == 0) {
            const auto* p = again();
#pragma unroll 1
            for (int r0 = w * 64; r0 < ROWS; r0 += NW * 64) {  // 64 rows, of one operand
                const int r = r0 + l;
                const int64_t x = min(load_x + r, (int)p->n - 1);
                const int64_t v = min(load_v + vocab_row<VT>(r - BX), (int)p->vocab - 1);
                load_lds4(scales0 + (load_four * ROWS + r0) * 4,
                          k / 2 + (r0 < BX ? p->qscales + x * p->qss : p->wscales + v * p->wss));
            }
            load_four = (load_four + 1) & 3;
        }
    };
    auto issue = [&](int i) {  // the i-th of the step's loads
        constexpr int LX = BX / 16 / NW;
        asm volatile("" : "+v"(off_x), "+v"(off_v));  // added anew in each step: the sums would not fit the registers
        load_lds16(rows0 + load_at * (ROWS * STEP) + (i * NW + w) * 1024,
                   i < LX ? off_x + i * NW * 16 * (int)a.qs : off_v + vocab_row<VT>((i - LX) * NW * 16) * (int)a.ws,
                   i < LX ? from_x : from_v, load_k * STEP);
    };
    auto issued = [&]() {
        load_at = load_at == STAGES - 1 ? 0 : load_at + 1;
        ++load_k;
    };
    auto next_tile = [&](i32x4& to_x, i32x4& to_v) {
        ++load_tile;
        advance(load_place);
        turn(to_x, to_v);
    };

    const int wx = w % WX * (32 * XT), wv = BX + w / WX * (32 * VT);  // the wave's first rows in LDS
    // where a lane's rows of its first tiles begin (the others are 32 rows on, where the chunks' turn is the same)
    const int turned = ((l / 32 * 2) ^ chunk_turn(l % 32)) * 16;
    const int at_x = (wx + l % 32) * STEP + turned, at_v = (wv + l % 32) * STEP + turned;
    int read_at = 0;  // the next step to read
    auto read = [&](i32x8 (&fx)[XT], i32x8 (&fv)[VT], int f) {  // the f-th of the step's fragments
        const uint8_t* at = s_rows + read_at * (ROWS * STEP);
        const int lo = f < VT ? at_v : at_x, r = 32 * (f < VT ? f : f - VT);
        const i32x4 a0 = *reinterpret_cast<const i32x4*>(at + lo + r * STEP);
        const i32x4 a1 = *reinterpret_cast<const i32x4*>(at + (lo ^ 16) + r * STEP);
        (f < VT ? fv[f < VT ? f : 0] : fx[f < VT ? 0 : f - VT]) =
            __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    f32x16 acc[XT][VT];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < XT; ++i)
#pragma unroll
            for (int j = 0; j < VT; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    };
    int sx[XT], sv[VT];  // the scales of four blocks, the current one's lowest
    // a product stays in its place: left to the compiler they sink past the next barriers, and the operands of several
    // steps do not fit the registers
    auto stay = [](f32x16& c) { asm volatile("" : "+v"(c)); };
    // between(part, parts): what is done between the products
    auto multiply = [&](const i32x8 (&fx)[XT], const i32x8 (&fv)[VT], auto between) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < XT; ++i)
#pragma unroll
                for (int j = 0; j < VT; ++j) {
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fx[i], fv[j], acc[i][j], 0, 0, 0, sx[i],
                                                                              0, sv[j]);
                    stay(acc[i][j]);
                    between(i * VT + j, XT * VT);
                }
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                bf16x8 hx[XT];
#pragma unroll
                for (int i = 0; i < XT; ++i) hx[i] = widen8(fx[i], s, scale_of<0>(sx[i]));
#pragma unroll
                for (int j = 0; j < VT; ++j) {
                    const bf16x8 hv = widen8(fv[j], s, scale_of<0>(sv[j]));
#pragma unroll
                    for (int i = 0; i < XT; ++i) {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hx[i], hv, acc[i][j], 0, 0, 0);
                        stay(acc[i][j]);
                    }
                }
                between(s, 4);
            }
        }
    };

    turn(from_x, from_v);
    i32x8 fx[2][XT], fv[2][VT];
#pragma unroll 1
    for (int i = 0; i < STAGES; ++i) {
        if (load_k == nk) {
            load_k = 0;
            next_tile(from_x, from_v);
        }
        issue_scales(load_k);
#pragma unroll
        for (int j = 0; j < LOADS; ++j) issue(j);
        issued();
    }
    step_barrier<(STAGES - 1) * LOADS>();
#pragma unroll
    for (int f = 0; f < XT + VT; ++f) read(fx[0], fv[0], f);
    ++read_at;
    clear();
    int four = 0;        // the place of the four blocks' scales
    bool quiet = false;  // whether a whole tile's stores may still be under way
    bool far = false;    // float32: whether a scale of this lane's rows of the tile is
    // a block of columns: two steps
    auto block = [&](int kb, auto stores) {
        if ((kb & 3) == 0) {
            const int* at = s_scales + four * ROWS;
#pragma unroll
            for (int i = 0; i < XT; ++i) sx[i] = at[wx + 32 * i + l % 32];
#pragma unroll
            for (int j = 0; j < VT; ++j) sv[j] = at[wv + 32 * j + l % 32];
            four = (four + 1) & 3;
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < XT; ++i) far |= far_scales(sx[i], nk / 2 - kb);
#pragma unroll
                for (int j = 0; j < VT; ++j) far |= far_scales(sv[j], nk / 2 - kb);
            }
        }
        // whichever of the block's two loads begins a tile or four blocks is prepared here, so that nothing branches
        // between the steps
        i32x4 to_x = from_x, to_v = from_v;
        const int ahead = STAGES % 2;  // steps until then
        int k = load_k + ahead;
        if (k == nk) {
            k = 0;
            next_tile(to_x, to_v);
        }
        issue_scales(k);
        if (ahead == 0) from_x = to_x, from_v = to_v, load_k = k;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            // step s + 1 is here, the later ones are under way
            step_barrier<(STAGES - 2) * LOADS + decltype(stores)::value>();
            // the next operands' reads and the loads spread over the products: all waves' at once would keep each
            // other, and the products behind them, waiting
            multiply(fx[half], fv[half], [&](int part, int parts) {
#pragma unroll
                for (int f = part * (XT + VT) / parts; f < (part + 1) * (XT + VT) / parts; ++f)
                    read(fx[1 - half], fv[1 - half], f);
#pragma unroll
                for (int i = part * LOADS / parts; i < (part + 1) * LOADS / parts; ++i) issue(i);
            });
            read_at = read_at == STAGES - 1 ? 0 : read_at + 1;
            issued();
            if (ahead == 1 && half == 0) from_x = to_x, from_v = to_v, load_k = k;
        }
#pragma unroll
        for (int i = 0; i < XT; ++i) sx[i] = (int)((uint32_t)sx[i] >> 8);
#pragma unroll
        for (int j = 0; j < VT; ++j) sv[j] = (int)((uint32_t)sv[j] >> 8);
    };
    for (int k = 0; k < mine; ++k) {
        if (LET && quiet)
            block(0, std::integral_constant<int, STORES>{});
        else
            block(0, std::integral_constant<int, 0>{});
        for (int kb = 1; kb < nk / 2; ++kb) block(kb, std::integral_constant<int, 0>{});
        // the last products' wait states before their results are read: behind `stay` the compiler need not see them
        asm volatile("s_nop 15\n\ts_nop 3");
#pragma unroll
        for (int i = 0; i < XT; ++i)
#pragma unroll
            for (int j = 0; j < VT; ++j) stay(acc[i][j]);
        int x0, v0;
        corner(place, x0, v0);
        advance(place);
        // element e of acc[i][j]: feature row x + 32 i + 8 (e / 4) + e % 4, score v + j
        const auto* p = again();
        const int n = (int)p->n, vocab = (int)p->vocab;
        const int64_t os = p->os;
        const int x = x0 + wx + 4 * (l / 32), v = v0 + (wv - BX) + l % 32 * VT;
        auto out = (scores_at<T>)((T*)p->out + x * os + v);
        const bool whole = n - x0 >= BX && vocab - v0 >= BV;
        int rows = n - x;  // from out on
        const int left = vocab - v;
        auto store = [&](auto past) {
#pragma unroll
            for (int i = 0; i < XT; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float t[VT];
#pragma unroll
                    for (int j = 0; j < VT; ++j) t[j] = acc[i][j][e];
                    if (whole || (rows > 0 && left >= VT)) {
                        store_run<decltype(past)::value, T>(out, t);
                    } else if (rows > 0) {
#pragma unroll
                        for (int j = 0; j < VT - 1; ++j)
                            if (j < left) out[j] = (T)t[j];
                    }
                    // row by row: all rows' places together would not fit the registers
                    const int on = e % 4 == 3 ? 5 : 1;
                    out += on * os;
                    rows -= on;
                    asm volatile("" : "+v"(out), "+v"(rows));
                }
        };
        if (sizeof(T) == 4 && __ballot(far)) {
            far_tile<VT>(*p, x0 + wx, XT, v0, wv - BX);
            quiet = far = false;
        } else {
            if (whole && p->past)
                store(std::true_type{});
            else
                store(std::false_type{});
            quiet = LET && whole;
        }
        clear();
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the loads past the last step
}

template <class T, int WX, int WV, int XT, int VT, int STAGES>
hipError_t scores_tiles(ScoreArgs a, hipStream_t s) {
    constexpr int BX = 32 * XT * WX, BV = 32 * VT * WV;
    // rows of whole cache lines only: of others past the caches the lines' parts go to memory one by one
    a.past = (uintptr_t)a.out % 128 == 0 && a.os * sizeof(T) % 128 == 0;
    // at most 2^27 tiles: there are at most 2^40 scores
    const int64_t tx = (a.n + BX - 1) / BX, tv = (a.vocab + BV - 1) / BV, blocks = 256 * (8 / (WX * WV));
    const int64_t grid = tx * tv < blocks ? (tx * tv + 7) / 8 * 8 : blocks;
    k_scores_tiles<T, WX, WV, XT, VT, STAGES><<<(unsigned)grid, 64 * WX * WV, 0, s>>>(a, (int)tx, (int)tv);
    return hipGetLastError();
}

// Which way a product takes. Straight to registers where there are few rows, or too few tiles for the units; through
// LDS otherwise. us, straight and by tiles of 128 x 128 (float32 in brackets):
//   4 x 1024 x 65536     13, 14.5 (13, 17.5)    16 x 1024 x 65536   17, 15 (17, 18)
//   16 x 1024 x 8192     8, 8 (8, 12)           32 x 1024 x 65536   18, 15 (18.7, 19.1)
//   64 x 1024 x 65536    32, 16.5 (34, 21)      300 x 1024 x 300    10, 9 (10, 12.5)
//   1024 x 1024 x 1024   10, 8 (11, 11)         1280 x 6528 x 576   39, 31 (42, 48)
//   512 x 8192 x 1000    28, 32 (29, 58)        2048 x 4096 x 512   27, 18 (29, 30.5)
//   4000 x 512 x 400     10, 8 (11, 10)         128 x 65536 x 128   126, 214 (127, 412)
// Straight, 64 x 32 to a wave reads a quarter less than 32 x 32, and fills the units where the depth can be split over
// eight waves: 512 x 8192 x 1000 27, with 32 x 32 34; 512 x 2048 x 1000 15, 11.
// Tiles of 256 x 256 have the operands' bytes from LDS for half the products of 128 x 128; with few columns to a tile
// two blocks to a unit hide each other's stores: 256 x 256 and two blocks of 128 x 256, 8192 x 256 x 65536 282, 242;
// x 384 323, 294; x 512 349, 352; x 1024 547, 605; 8192 x 8192 x 8192 438, 533 (128 x 128 633).
// In float32, where the products take four times as long, 256 x 256 gains little and loses where rounds are not full:
// 128 x 128 and 256 x 256, 8192 x 8192 x 8192 920, 797; 16384 x 512 x 16384 327, 287; 3000 x 4096 x 5000 116, 102;
// 8192 x 1024 x 65536 1084, 942; 5000 x 2048 x 5000 100, 101; 45414 x 1280 x 550 75, 100; 5003 x 256 x 8192 37, 43.
template <class T>
hipError_t scores(const ScoreArgs& a, hipStream_t s) {
    auto tiles = [&](int64_t bx, int64_t bv) { return ((a.n + bx - 1) / bx) * ((a.vocab + bv - 1) / bv); };
    const bool deep = a.cols >= 4096;
    if constexpr (sizeof(T) == 2) {
        if (a.n > 8) {
            if (a.cols <= 384 && tiles(128, 256) >= 256) return scores_tiles<T, 2, 2, 2, 4, 3>(a, s);
            if (tiles(256, 256) >= 192) return scores_tiles<T, 4, 2, 2, 4, 4>(a, s);
            if (tiles(128, 128) >= (a.n <= 16 ? 256 : deep ? 48 : 8)) return scores_tiles<T, 2, 2, 2, 2, 4>(a, s);
        }
    } else if (a.n > 32 && tiles(128, 128) >= 96) {
        // three quarters at least of the units' rounds of 256 x 256 are scores
        const int64_t rounds = (tiles(256, 256) + 255) / 256;
        if (a.cols >= 512 && a.n * a.vocab / (3 * 256 * 65536 / 4) >= rounds)
            return scores_tiles<T, 4, 2, 2, 4, 4>(a, s);
        return scores_tiles<T, 2, 2, 2, 2, 4>(a, s);
    }
    if (a.n <= 16) return scores_split<T, 1, 1, 1>(a, s);
    // here less than 96 tiles of 128 x 128 are at most 760 of these: 4 waves to each at least
    if (deep && a.n > 32 && tiles(64, 32) >= 128) return scores_split<T, 4, 2, 4>(a, s);
    return scores_split<T, 2, 2, 1>(a, s);
}

}  // namespace

hipError_t launch_label_scores(const ScoreArgs& a, hipStream_t stream) {
    return a.half ? scores<bf16>(a, stream) : scores<float>(a, stream);
}

}  // namespace gs
