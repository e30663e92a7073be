// Root-mean-square normalisation of feature rows after a residual's addition,
// forward and backward, and with the result in 8 bits (rows8.hpp).
//
//   h = x + residual (rounded to the rows' type, as it is handed on)
//   rstd = (sum_j h_j^2 / D + eps)^-1/2,  y = h rstd w
//   g = dy w,  dx = rstd (g - h rstd^2 mean_j(g h)) + dh      (dh: h's own gradient)
//   dw_j = sum_i dy_ij h_ij rstd_i
//
// Bound by memory: the forward reads x and the residual and writes h and y once,
// the backward reads h, dy and dh and writes dx once. A row lies in the registers
// of LPR lanes (from one lane to a block of 1024 threads for the longest rows), so
// that its statistic costs no second read. Blocks walk over the rows. The column
// sums of dw go to the workspace, one row per block, and a second launch adds them
// in a fixed order (norm.hip); a single block writes dw itself (64 x 6 float32 with
// gradients 14 us, 19 with the second launch).
//
// With inputs that change from call to call: 1M x 64 float32 with residual and
// gradients 333 us (1.79 GB read or written once: 5.4 TB/s; a large copy has 4.8);
// 32771 rows of 771 bfloat16 in a wider matrix 87 (4.1 TB/s: forward 40, backward 39,
// column sums 5; where the backward loaded the sum's gradient behind its row's sum it
// took 66). 65536 x 1024 bfloat16 with residual into 8 bits 93 (5.1 TB/s), the rows as
// they are 42 (4.8). Short rows share a wave: 636224 x 13 float32 into 8 bits 24 us, 40
// with residual and norm (on one set of buffers 22 and 31; with a row to the 32 lanes of
// a block of columns 250 and 88).
#include "elem.hpp"
#include "launch.hpp"
#include "rows8.hpp"

// Products are rounded before they are added (fused only where fmaf says so).
#pragma clang fp contract(off)

namespace gs {

namespace {

// load_row and store_row of whole rows; PAST: past the caches.
template <bool FULL, bool PAST, class T>
__device__ __forceinline__ wide_t<T> load_part(const T* p, int left, int64_t room) {
    static_assert(FULL || !PAST, "");
    if constexpr (PAST) return __builtin_nontemporal_load(reinterpret_cast<const wide_any<T>*>(p));
    return load_row<FULL>(p, left, room);
}

template <bool FULL, bool PAST, class T, int V>
__device__ __forceinline__ void store_part(T* p, int left, const float (&v)[V]) {
    if constexpr (PAST) {
        wide_t<T> t;
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = (T)v[i];
        __builtin_nontemporal_store(t, reinterpret_cast<wide_any<T>*>(p));
    } else {
        store_row<FULL>(p, left, v);
    }
}

// Sum over the LPR lanes that share a row (all of them get it). s: NT / 64 floats, for rows of a whole block.
template <int NT, int LPR>
__device__ __forceinline__ float rms_row_sum(float v, float* s) {
    constexpr int W = LPR < 64 ? LPR : 64;
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
    if constexpr (LPR > 64) {
        static_assert(LPR == NT, "a row of more than a wave is the block's");
        __syncthreads();  // earlier readers of s are done
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int k = 0; k < LPR / 64; ++k) v += s[k];
    }
    return v;
}

struct RmsArgs {
    int64_t n;
    int dim;
    const void *x, *residual, *weight;  // x: h in the backward
    int64_t xs, rs;
    float eps;
    void *sum, *y;
    int64_t ss, ys;
    float* rstd;  // written by the forward, read by the backward
    uint8_t *q, *scales;
    int64_t qs, scs;
    const void *dy, *dsum;
    int64_t dys, dss;
    void* dx;
    int64_t dxs;
    float* part;    // [blocks][dim]: the blocks' column sums
    void* dweight;  // they themselves, of one block
    bool plain;     // into 8 bits without the norm
};

// Stores a wave's 64 / LPR rows of a block or less in 8 bits, of which a lane has VEC columns: 16 bytes to a lane, side
// by side over the rows, zeros behind the columns. first: the wave's first row.
template <int LPR, int VEC>
__device__ __forceinline__ void store_short(const RmsArgs& a, int64_t first, const float (&v)[VEC], float inverse) {
    constexpr int ROWS = 64 / LPR, PER = VEC / 4, WORDS = LPR * PER;  // words of a row, PER to a lane
    const int lane = threadIdx.x & 63;
    uint32_t have[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) have[p] = pack_q8(v + 4 * p, inverse);
#pragma unroll
    for (int i = 0; i < (ROWS * 8 + 63) / 64; ++i) {
        const int row = (i * 64 + lane) / 8, chunk = lane % 8;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int word = 4 * chunk + k, from = row * LPR + word / PER;
            uint32_t got = __shfl(have[0], from & 63);
            if (PER == 2) {
                const uint32_t odd = __shfl(have[PER - 1], from & 63);
                got = word % 2 ? odd : got;
            }
            w[k] = word < WORDS ? got : 0u;
        }
        if (row < ROWS && first + row < a.n)
            *reinterpret_cast<uint4*>(a.q + (first + row) * a.qs + chunk * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// The accesses of a row whose weights stay in registers over the block's rows.
constexpr int KEPT = 4;

template <class T, int NT, int LPR, int EPL, bool FULL, bool Q8, bool PAST>
__global__ __launch_bounds__(NT) void k_rms_fwd(RmsArgs a) {
    __shared__ float s_red[NT / 64];
    constexpr int RPB = NT / LPR, VEC = WIDE<T>;
    constexpr bool KEEP = EPL <= KEPT;
    const int l = threadIdx.x % LPR, dim = a.dim;
    const T *x = (const T*)a.x, *residual = (const T*)a.residual, *weight = (const T*)a.weight;
    wide_t<T> w[KEEP ? EPL : 1];
    if (KEEP && weight) {
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int c = (e * LPR + l) * VEC;
            w[KEEP ? e : 0] = (T)0.f;
            if (c < dim) w[KEEP ? e : 0] = load_row<FULL>(weight + c, dim - c, dim - c);
        }
    }
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.n; r0 += (int64_t)gridDim.x * RPB) {
        const int64_t r = r0 + threadIdx.x / LPR;
        const bool live = r < a.n;  // a row past the end is computed from zeros and not stored
        wide_t<T> raw[EPL];
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int c = (e * LPR + l) * VEC;
            raw[e] = (T)0.f;
            if (live && c < dim)
                raw[e] = load_part<FULL, PAST>(x + r * a.xs + c, dim - c, (a.n - 1 - r) * a.xs + dim - c);
        }
        if (residual) {
            wide_t<T> more[EPL];
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                const int c = (e * LPR + l) * VEC;
                more[e] = (T)0.f;
                if (live && c < dim)
                    more[e] = load_part<FULL, PAST>(residual + r * a.rs + c, dim - c, (a.n - 1 - r) * a.rs + dim - c);
            }
#pragma unroll
            for (int e = 0; e < EPL; ++e)
#pragma unroll
                for (int k = 0; k < VEC; ++k) raw[e][k] = (T)((float)raw[e][k] + (float)more[e][k]);
        }
        auto squares = [&](float by) {
            float sq = 0.f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                const int left = dim - (e * LPR + l) * VEC;
                float v[VEC];
                widen<FULL, T>(raw[e], left, v);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    v[k] *= by;
                    sq = (FULL ? left > 0 : k < left) ? fmaf(v[k], v[k], sq) : sq;
                }
            }
            return rms_row_sum<NT, LPR>(sq, s_red);
        };
        // A row whose squares float32 does not hold (values of 1e18 and more, or with an eps below 1e-24 of 1e-12 and
        // less) is summed again times a power of two, from its registers. All lanes of a row go the same way. (Of rows
        // as they are nothing is asked.)
        float by = 1.f, root = 1.f;
        if (!(Q8 && a.plain)) {
            float sum = squares(1.f);
            if (sum > 0x1p120f || (sum < 0x1p-80f && a.eps < 0x1p-80f)) {
                by = sum > 1.f ? 0x1p-80f : 0x1p100f;
                sum = squares(by);
            }
            root = 1.0f / sqrtf(sum / (float)dim + a.eps * by * by);
        }
        if (a.rstd && live && l == 0) a.rstd[r] = root * by;
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int c = (e * LPR + l) * VEC, left = dim - c;
            float v[VEC];
            widen<FULL, T>(raw[e], left, v);
            if (a.sum && live && left > 0) store_row<FULL>((T*)a.sum + r * a.ss + c, left, v);
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] = v[k] * by * root;
            if (weight) {
                float f[VEC];
                wide_t<T> wr = (T)0.f;
                if (KEEP)
                    wr = w[KEEP ? e : 0];
                else if (left > 0)
                    wr = load_row<FULL>(weight + c, left, left);
                widen<FULL, T>(wr, left, f);
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[k] *= f[k];
            }
            if constexpr (Q8) {
                constexpr int LANES = LPR < Q8_LANES<T> ? LPR : Q8_LANES<T>;
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    v[k] = (FULL ? left > 0 : k < left) ? v[k] : 0.f;
                    top = fmaxf(top, finite_abs(v[k]));
                }
#pragma unroll
                for (int off = LANES / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
                const int ex = scale_exponent(top);
                if constexpr (LPR >= Q8_LANES<T>) {
                    if (live && c < q8_cols(dim)) {
                        store_q8(a.q + r * a.qs + c, v, scale_inverse(ex));
                        if (l % LANES == 0) a.scales[r * a.scs + c / Q8_BLOCK] = (uint8_t)ex;
                    }
                } else {
                    store_short<LPR>(a, r0 + (threadIdx.x >> 6) * (64 / LPR), v, scale_inverse(ex));
                    if (live && l == 0) *reinterpret_cast<uint32_t*>(a.scales + r * a.scs) = 0x7f7f7f00u | ex;
                }
            } else if (live && left > 0) {
                store_part<FULL, PAST>((T*)a.y + r * a.ys + c, left, v);
            }
        }
        if constexpr (Q8 && LPR >= Q8_LANES<T>) {
            const int at = q8_cols(dim) / Q8_BLOCK + l;
            if (live && at < q8_groups(dim)) a.scales[r * a.scs + at] = 127;
        }
    }
}

// A row's h, dy and dh are loaded together, before the row's sum, where registers hold them (and the weights) all;
// longer rows are read again from the cache for their second use.
template <class T, int NT, int LPR, int EPL, bool FULL, bool PAST>
__global__ __launch_bounds__(NT) void k_rms_bwd(RmsArgs a) {
    constexpr int RPB = NT / LPR, VEC = WIDE<T>;
    constexpr bool AGAIN = EPL > KEPT;
    __shared__ float s_red[NT / 64];
    __shared__ float s_acc[LPR < NT ? LPR * EPL * VEC : 1];
    const int l = threadIdx.x % LPR, dim = a.dim;
    const T *h = (const T*)a.x, *weight = (const T*)a.weight, *dy = (const T*)a.dy, *dsum = (const T*)a.dsum;
    float aw[EPL][VEC];
#pragma unroll
    for (int e = 0; e < EPL; ++e)
#pragma unroll
        for (int k = 0; k < VEC; ++k) aw[e][k] = 0.f;
    wide_t<T> w[AGAIN ? 1 : EPL];
    auto load_weight = [&](int e) {
        const int left = dim - (e * LPR + l) * VEC;
        wide_t<T> v = (T)0.f;
        if (weight && left > 0) v = load_row<FULL>(weight + (dim - left), left, left);
        return v;
    };
    if (!AGAIN) {
#pragma unroll
        for (int e = 0; e < EPL; ++e) w[AGAIN ? 0 : e] = load_weight(e);
    }
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.n; r0 += (int64_t)gridDim.x * RPB) {
        const int64_t r = r0 + threadIdx.x / LPR;
        const bool live = r < a.n;
        wide_t<T> rh[AGAIN ? 1 : EPL], rg[AGAIN ? 1 : EPL], rs[AGAIN ? 1 : EPL];
        auto load = [&](const T* p, int64_t stride, int e) {
            const int c = (e * LPR + l) * VEC;
            wide_t<T> v = (T)0.f;
            if (p && live && c < dim)
                v = load_part<FULL, PAST>(p + r * stride + c, dim - c, (a.n - 1 - r) * stride + dim - c);
            return v;
        };
        if (!AGAIN) {
#pragma unroll
            for (int e = 0; e < EPL; ++e) rh[AGAIN ? 0 : e] = load(h, a.xs, e);
#pragma unroll
            for (int e = 0; e < EPL; ++e) rg[AGAIN ? 0 : e] = load(dy, a.dys, e);
#pragma unroll
            for (int e = 0; e < EPL; ++e) rs[AGAIN ? 0 : e] = load(dsum, a.dss, e);
        }
        const float rstd = live ? a.rstd[r] : 0.f;
        // hh: h rstd; g: dy w; d: dy
        auto values = [&](int e, float (&hh)[VEC], float (&g)[VEC], float (&d)[VEC]) {
            const int left = dim - (e * LPR + l) * VEC;
            widen<FULL, T>(rh[AGAIN ? 0 : e], left, hh);
            widen<FULL, T>(rg[AGAIN ? 0 : e], left, d);
            float f[VEC];
            widen<FULL, T>(AGAIN ? load_weight(e) : w[AGAIN ? 0 : e], left, f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                hh[k] *= rstd;
                g[k] = weight ? d[k] * f[k] : d[k];
            }
        };
        float sx = 0.f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            if (AGAIN) rh[0] = load(h, a.xs, e), rg[0] = load(dy, a.dys, e);
            float hh[VEC], g[VEC], d[VEC];
            values(e, hh, g, d);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {  // a column past the row has d = 0
                aw[e][k] = fmaf(d[k], hh[k], aw[e][k]);
                sx = fmaf(g[k], hh[k], sx);
            }
        }
        if (!a.dx) continue;  // the same for the whole launch
        const float mx = rms_row_sum<NT, LPR>(sx, s_red) / (float)dim;
        if (!live) continue;
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            if (AGAIN) rh[0] = load(h, a.xs, e), rg[0] = load(dy, a.dys, e), rs[0] = load(dsum, a.dss, e);
            const int c = (e * LPR + l) * VEC, left = dim - c;
            float hh[VEC], g[VEC], d[VEC];
            values(e, hh, g, d);
            widen<FULL, T>(rs[AGAIN ? 0 : e], left, d);
#pragma unroll
            for (int k = 0; k < VEC; ++k) g[k] = rstd * (g[k] - hh[k] * mx) + d[k];  // d: dh, zeros without one
            if (left > 0) store_part<FULL, PAST>((T*)a.dx + r * a.dxs + c, left, g);
        }
    }
    if (!a.part && !a.dweight) return;
    // the block's column sums: over the row groups of a wave, then over the waves in turn
#pragma unroll
    for (int e = 0; e < EPL; ++e)
#pragma unroll
        for (int k = 0; k < VEC; ++k)
#pragma unroll
            for (int off = LPR; off < 64; off <<= 1) aw[e][k] += __shfl_xor(aw[e][k], off);
    auto store = [&](int c, float v) {
        if (a.dweight)
            ((T*)a.dweight)[c] = (T)v;
        else
            a.part[(size_t)blockIdx.x * dim + c] = v;
    };
    if constexpr (LPR < NT) {
        const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
        for (int turn = 0; turn < NT / 64; ++turn) {
            if (wv == turn && lane < LPR) {
#pragma unroll
                for (int e = 0; e < EPL; ++e)
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        const int c = (e * LPR + l) * VEC + k;
                        s_acc[c] = turn ? s_acc[c] + aw[e][k] : aw[e][k];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < dim; c += NT) store(c, s_acc[c]);
    } else {
#pragma unroll
        for (int e = 0; e < EPL; ++e)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const int c = (e * LPR + l) * VEC + k;
                if (c < dim) store(c, aw[e][k]);
            }
    }
}

enum RmsCall { RMS_FWD, RMS_BWD, RMS_Q8 };

// Of 256 threads, and as many fewer of more. The backward's are rows of the column sums.
constexpr int RMS_BLOCKS_FWD = 2048, RMS_BLOCKS_BWD = 1024;
template <int CALL>
constexpr int rms_blocks(int threads) {
    return (CALL == RMS_BWD ? RMS_BLOCKS_BWD : RMS_BLOCKS_FWD) * 256 / threads;
}
// The accesses of the longest rows that blocks of 256 threads take; 1024 threads take longer ones.
constexpr int LONGEST_256 = 1024;

// What a call reads and writes in all beyond which it goes past the caches, except for the sum, which the backward
// reads next: nothing else of it would still be there for who comes next, but it would put the sum out. (What the
// last-level cache holds. 1M x 64 float32 with gradients 400 us through the caches, 332 past them; smaller calls gain
// nothing by it, 32768 x 1024 bfloat16, and leave their result in the cache for its reader.)
constexpr int64_t CACHED = (int64_t)256 << 20;

template <class T, int CALL, int NT, int LPR, int EPL, bool FULL>
hipError_t rms_rows(RmsArgs a, int& blocks, hipStream_t s) {
    const int64_t want = (a.n + NT / LPR - 1) / (NT / LPR);
    const int cap = rms_blocks<CALL>(NT);
    blocks = (int)(want < cap ? want : cap);
    const int matrices = CALL == RMS_BWD ? 3 + (a.dsum != nullptr) : 2 + (a.residual ? 2 : 0);
    const bool past = FULL && CALL != RMS_Q8 && a.n * a.dim * (int64_t)sizeof(T) * matrices > CACHED;
    constexpr bool CAN = FULL && CALL != RMS_Q8;
    if constexpr (CALL == RMS_BWD) {
        if (blocks > 1) a.dweight = nullptr;
        if (past)
            k_rms_bwd<T, NT, LPR, EPL, FULL, CAN><<<blocks, NT, 0, s>>>(a);
        else
            k_rms_bwd<T, NT, LPR, EPL, FULL, false><<<blocks, NT, 0, s>>>(a);
    } else {
        if (past)
            k_rms_fwd<T, NT, LPR, EPL, FULL, CALL == RMS_Q8, CAN><<<blocks, NT, 0, s>>>(a);
        else
            k_rms_fwd<T, NT, LPR, EPL, FULL, CALL == RMS_Q8, false><<<blocks, NT, 0, s>>>(a);
    }
    return hipGetLastError();
}

// The lanes of a row and their accesses: the fewest lanes that hold it with one access each up to a wave, then more
// accesses, then a block of four waves, then of sixteen.
template <class T, int CALL, bool FULL>
hipError_t rms_pick(const RmsArgs& a, int& blocks, hipStream_t s) {
    const int v = (a.dim + WIDE<T> - 1) / WIDE<T>;
    if (v <= 1) return rms_rows<T, CALL, 256, 1, 1, FULL>(a, blocks, s);
    if (v <= 2) return rms_rows<T, CALL, 256, 2, 1, FULL>(a, blocks, s);
    if (v <= 4) return rms_rows<T, CALL, 256, 4, 1, FULL>(a, blocks, s);
    if (v <= 8) return rms_rows<T, CALL, 256, 8, 1, FULL>(a, blocks, s);
    if (v <= 16) return rms_rows<T, CALL, 256, 16, 1, FULL>(a, blocks, s);
    if (v <= 32) return rms_rows<T, CALL, 256, 32, 1, FULL>(a, blocks, s);
    if (v <= 64) return rms_rows<T, CALL, 256, 64, 1, FULL>(a, blocks, s);
    if (v <= 128) return rms_rows<T, CALL, 256, 64, 2, FULL>(a, blocks, s);
    if (v <= 256) return rms_rows<T, CALL, 256, 64, 4, FULL>(a, blocks, s);
    if (v <= 512) return rms_rows<T, CALL, 256, 256, 2, FULL>(a, blocks, s);
    if (v <= LONGEST_256) return rms_rows<T, CALL, 256, 256, 4, FULL>(a, blocks, s);
    if (v <= 2048) return rms_rows<T, CALL, 1024, 1024, 2, FULL>(a, blocks, s);
    if (v <= 4096) return rms_rows<T, CALL, 1024, 1024, 4, FULL>(a, blocks, s);
    if (v <= 8192) return rms_rows<T, CALL, 1024, 1024, 8, FULL>(a, blocks, s);
    if constexpr (sizeof(T) == 4) return rms_rows<T, CALL, 1024, 1024, 16, FULL>(a, blocks, s);
    return hipErrorInvalidValue;  // 65536 bfloat16 are 8192 accesses
}

template <int CALL>
hipError_t rms_launch(bool half, const RmsArgs& a, int& blocks, hipStream_t s) {
    if (half)
        return a.dim % WIDE<bf16> == 0 ? rms_pick<bf16, CALL, true>(a, blocks, s)
                                       : rms_pick<bf16, CALL, false>(a, blocks, s);
    return a.dim % WIDE<float> == 0 ? rms_pick<float, CALL, true>(a, blocks, s)
                                    : rms_pick<float, CALL, false>(a, blocks, s);
}

}  // namespace

size_t rms_bwd_workspace(int64_t n, int dim, bool half) {
    const int wide = half ? WIDE<bf16> : WIDE<float>;
    const int64_t most = rms_blocks<RMS_BWD>((dim + wide - 1) / wide <= LONGEST_256 ? 256 : 1024);
    const int64_t rows = n < most ? n : most;
    return ((size_t)rows * dim * sizeof(float) + 255) & ~(size_t)255;
}

hipError_t launch_rms_fwd(int64_t n, int dim, bool half, const void* x, int64_t xs, const void* residual, int64_t rs,
                          const void* weight, float eps, void* sum, int64_t ss, void* y, int64_t ys, float* rstd,
                          hipStream_t stream) {
    RmsArgs a{};
    a.n = n;
    a.dim = dim;
    a.x = x;
    a.xs = xs;
    a.residual = residual;
    a.rs = rs;
    a.weight = weight;
    a.eps = eps;
    a.sum = sum;
    a.ss = ss;
    a.y = y;
    a.ys = ys;
    a.rstd = rstd;
    int blocks;
    return rms_launch<RMS_FWD>(half, a, blocks, stream);
}

hipError_t launch_rms_bwd(int64_t n, int dim, bool half, const void* h, int64_t hs, const void* weight,
                          const float* rstd, const void* dy, int64_t dys, const void* dsum, int64_t dss, void* dx,
                          int64_t dxs, void* dweight, float* part, hipStream_t stream) {
    RmsArgs a{};
    a.n = n;
    a.dim = dim;
    a.x = h;
    a.xs = hs;
    a.weight = weight;
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.dys = dys;
    a.dsum = dsum;
    a.dss = dss;
    a.dx = dx;
    a.dxs = dxs;
    a.part = dweight ? part : nullptr;
    a.dweight = dweight;
    int blocks = 0;
    if (n > 0 && (dx || dweight))
        if (hipError_t e = rms_launch<RMS_BWD>(half, a, blocks, stream)) return e;
    if (!dweight || blocks == 1) return hipSuccess;
    return launch_column_sums(half, blocks, dim, dim, part, dweight, nullptr, stream);
}

hipError_t launch_rms_q8(int64_t n, int dim, bool half, const void* x, int64_t xs, const void* residual, int64_t rs,
                         const void* weight, float eps, void* sum, int64_t ss, uint8_t* q, int64_t qs,
                         uint8_t* scales, int64_t scs, hipStream_t stream) {
    RmsArgs a{};
    a.n = n;
    a.dim = dim;
    a.x = x;
    a.xs = xs;
    a.residual = residual;
    a.rs = rs;
    a.weight = weight;
    a.eps = eps;
    a.sum = sum;
    a.ss = ss;
    a.q = q;
    a.qs = qs;
    a.scales = scales;
    a.scs = scs;
    int blocks;
    return rms_launch<RMS_Q8>(half, a, blocks, stream);
}

hipError_t launch_quantize_q8(int64_t n, int dim, bool half, const void* x, int64_t xs, uint8_t* q, int64_t qs,
                              uint8_t* scales, int64_t scs, hipStream_t stream) {
    RmsArgs a{};
    a.n = n;
    a.dim = dim;
    a.x = x;
    a.xs = xs;
    a.q = q;
    a.qs = qs;
    a.scales = scales;
    a.scs = scs;
    a.plain = true;
    int blocks;
    return rms_launch<RMS_Q8>(half, a, blocks, stream);
}

}  // namespace gs
