// Layer normalisation of feature rows, forward and backward.
//
//   mean = sum_j x_j / D,  rstd = (sum_j (x_j - mean)^2 / D + eps)^-1/2
//   xh = (x - mean) rstd,  y = xh w + b
//   g = dy w,  dx = rstd (g - mean_j(g) - xh mean_j(g xh))
//   dw_j = sum_i dy_ij xh_ij,  db_j = sum_i dy_ij
//
// Both directions are bound by memory: the forward reads x and writes y once,
// the backward reads x and dy and writes dx once. A row lies in the registers
// of LPR lanes (one lane up to a whole block), so that its statistics
// cost no second read; the variance is the mean square of x - mean, not a
// difference of sums. Blocks walk over the rows with the weights (and, in the
// backward, the column sums of dw and db) in registers. Column sums go to the
// workspace, one row per block, and a second launch adds them in a fixed
// order, so the result is the same bit for bit from run to run. Rows beyond
// what a block's registers hold are read again from the cache instead.
//
// A million rows of 64 float32: forward 90 us (512 MB, 5.7 TB/s), backward 155
// (768 MB, 5.0 TB/s), column sums 5; 32768 x 1024 bfloat16: 28, 39 and 6 (a
// large copy: 4.8 TB/s; part of these inputs is still in the last-level cache).
// Rows of odd length and stride run as fast: 77777 x 771 bfloat16 45 us, x 768
// 46 (with the accesses an element wide 771 columns cost twice as much). Rows past
// what registers hold take an access per element: 4000 x 16000 forward and
// backward 0.96 ms in float32 (1.3 TB/s), 0.77 in bfloat16, 4000 x 8000 0.12.
#include "elem.hpp"
#include "launch.hpp"

// Products are rounded before they are subtracted (fused only where fmaf says
// so): a difference that is zero in the formula, as dx of rows of one column, is zero.
#pragma clang fp contract(off)

namespace gs {

namespace {

constexpr int NB = 256;           // threads per block
constexpr int NORM_REG_DIM = 8192;  // longest row held in registers
constexpr int RED_COLS = 16;      // columns per block of the column-sum join
constexpr int RED_T = 1024;

// Sum over the LPR lanes that share a row (all of them get it). s: NB / 64 floats, for LPR = NB.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* s) {
    constexpr int W = LPR < 64 ? LPR : 64;
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
    if constexpr (LPR > 64) {
        const int w = threadIdx.x >> 6;
        __syncthreads();  // earlier readers of s are done
        if ((threadIdx.x & 63) == 0) s[w] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int k = 0; k < LPR / 64; ++k) v += s[k];
    }
    return v;
}

template <class T, int LPR, int EPL, bool FULL>
__global__ __launch_bounds__(NB) void k_norm_fwd(int64_t n, int dim, const T* __restrict__ x, int64_t xs,
                                                 const T* __restrict__ weight, const T* __restrict__ bias, float eps,
                                                 T* __restrict__ y, int64_t ys, float* __restrict__ mean_out,
                                                 float* __restrict__ rstd_out) {
    __shared__ float s_red[NB / 64];
    constexpr int RPB = NB / LPR, VEC = WIDE<T>;
    const int l = threadIdx.x % LPR;
    const float D = (float)dim;  // divided by, not multiplied by its reciprocal: the mean of equal values stays exact
    float w[EPL][VEC], b[EPL][VEC];
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
        const int c = (e * LPR + l) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            w[e][k] = 1.f;
            b[e][k] = 0.f;
        }
        if (c < dim) {
            if (weight) widen<FULL, T>(load_row<FULL>(weight + c, dim - c, dim - c), dim - c, w[e]);
            if (bias) widen<FULL, T>(load_row<FULL>(bias + c, dim - c, dim - c), dim - c, b[e]);
        }
    }
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < n; r0 += (int64_t)gridDim.x * RPB) {
        const int64_t r = r0 + threadIdx.x / LPR;
        const bool live = r < n;  // a row past the end is computed from zeros and not stored
        const T* xr = x + r * xs;
        wide_t<T> raw[EPL];
        float v[EPL][VEC];
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int c = (e * LPR + l) * VEC;
            raw[e] = (T)0.f;
            if (live && c < dim) raw[e] = load_row<FULL>(xr + c, dim - c, (n - 1 - r) * xs + dim - c);
        }
#pragma unroll
        for (int e = 0; e < EPL; ++e) widen<FULL, T>(raw[e], dim - (e * LPR + l) * VEC, v[e]);
#pragma unroll
        for (int e = 0; e < EPL; ++e)
#pragma unroll
            for (int k = 0; k < VEC; ++k) sum += v[e][k];
        const float mean = row_sum<LPR>(sum, s_red) / D;
        float sq = 0.f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int left = dim - (e * LPR + l) * VEC;
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                v[e][k] -= mean;
                sq = (FULL ? left > 0 : k < left) ? fmaf(v[e][k], v[e][k], sq) : sq;
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<LPR>(sq, s_red) / D + eps);
        if (!live) continue;
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int c = (e * LPR + l) * VEC;
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[e][k] = fmaf(v[e][k] * rstd, w[e][k], b[e][k]);
            if (c < dim) store_row<FULL>(y + r * ys + c, dim - c, v[e]);
        }
        if (l == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
    }
}

// One row per block, read from memory three times (the cache serves the later two).
template <class T>
__global__ __launch_bounds__(NB) void k_norm_fwd_long(int64_t n, int dim, const T* __restrict__ x, int64_t xs,
                                                      const T* __restrict__ weight, const T* __restrict__ bias,
                                                      float eps, T* __restrict__ y, int64_t ys,
                                                      float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    __shared__ float s_red[NB / 64];
    for (int64_t r = blockIdx.x; r < n; r += gridDim.x) {
        const T* xr = x + r * xs;
        float sum = 0.f;
        for (int c = threadIdx.x; c < dim; c += NB) sum += (float)xr[c];
        const float mean = row_sum<NB>(sum, s_red) / (float)dim;
        float sq = 0.f;
        for (int c = threadIdx.x; c < dim; c += NB) {
            const float d = (float)xr[c] - mean;
            sq = fmaf(d, d, sq);
        }
        const float rstd = 1.0f / sqrtf(row_sum<NB>(sq, s_red) / (float)dim + eps);
        for (int c = threadIdx.x; c < dim; c += NB) {
            const float xh = ((float)xr[c] - mean) * rstd;
            y[r * ys + c] = (T)fmaf(xh, weight ? (float)weight[c] : 1.f, bias ? (float)bias[c] : 0.f);
        }
        if (threadIdx.x == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
    }
}

// part (nullable): [gridDim.x][2][dim] column sums of dy xh and dy over the block's rows.
template <class T, int LPR, int EPL, bool FULL>
__global__ __launch_bounds__(NB) void k_norm_bwd(int64_t n, int dim, const T* __restrict__ x, int64_t xs,
                                                 const T* __restrict__ weight, const float* __restrict__ mean_in,
                                                 const float* __restrict__ rstd_in, const T* __restrict__ dy,
                                                 int64_t dys, T* __restrict__ dx, int64_t dxs,
                                                 float* __restrict__ part) {
    constexpr int RPB = NB / LPR, VEC = WIDE<T>;
    constexpr int COLS = LPR * EPL * VEC;
    __shared__ float s_red[NB / 64];
    __shared__ float s_acc[LPR < NB ? 2 * COLS : 1];
    const int l = threadIdx.x % LPR;
    const float inv = 1.0f / (float)dim;
    float w[EPL][VEC], aw[EPL][VEC], ab[EPL][VEC];
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
        const int c = (e * LPR + l) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            w[e][k] = 1.f;
            aw[e][k] = ab[e][k] = 0.f;
        }
        if (weight && c < dim) widen<FULL, T>(load_row<FULL>(weight + c, dim - c, dim - c), dim - c, w[e]);
    }
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < n; r0 += (int64_t)gridDim.x * RPB) {
        const int64_t r = r0 + threadIdx.x / LPR;
        const bool live = r < n;
        wide_t<T> rx[EPL], rg[EPL];
        float xv[EPL][VEC], gv[EPL][VEC];
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int c = (e * LPR + l) * VEC;
            rx[e] = rg[e] = (T)0.f;
            if (live && c < dim) {
                rx[e] = load_row<FULL>(x + r * xs + c, dim - c, (n - 1 - r) * xs + dim - c);
                rg[e] = load_row<FULL>(dy + r * dys + c, dim - c, (n - 1 - r) * dys + dim - c);
            }
        }
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            widen<FULL, T>(rx[e], dim - (e * LPR + l) * VEC, xv[e]);
            widen<FULL, T>(rg[e], dim - (e * LPR + l) * VEC, gv[e]);
        }
        const float mean = live ? mean_in[r] : 0.f, rstd = live ? rstd_in[r] : 0.f;
        float sg = 0.f, sx = 0.f;
#pragma unroll
        for (int e = 0; e < EPL; ++e)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float xh = (xv[e][k] - mean) * rstd;  // a column past the row has gv = 0
                aw[e][k] = fmaf(gv[e][k], xh, aw[e][k]);
                ab[e][k] += gv[e][k];
                const float g = gv[e][k] * w[e][k];
                sg += g;
                sx = fmaf(g, xh, sx);
                xv[e][k] = xh;
                gv[e][k] = g;
            }
        if (!dx) continue;  // the same for the whole launch
        const float mg = row_sum<LPR>(sg, s_red) * inv;
        const float mx = row_sum<LPR>(sx, s_red) * inv;
        if (!live) continue;
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int c = (e * LPR + l) * VEC;
#pragma unroll
            for (int k = 0; k < VEC; ++k) gv[e][k] = rstd * (gv[e][k] - fmaf(xv[e][k], mx, mg));
            if (c < dim) store_row<FULL>(dx + r * dxs + c, dim - c, gv[e]);
        }
    }
    if (!part) return;
    // the block's column sums: over the row groups of a wave, then over the waves in turn
#pragma unroll
    for (int e = 0; e < EPL; ++e)
#pragma unroll
        for (int k = 0; k < VEC; ++k)
#pragma unroll
            for (int off = LPR; off < 64; off <<= 1) {
                aw[e][k] += __shfl_xor(aw[e][k], off);
                ab[e][k] += __shfl_xor(ab[e][k], off);
            }
    float* pw = part + (size_t)blockIdx.x * 2 * dim;
    if constexpr (LPR < NB) {
        const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
        for (int turn = 0; turn < NB / 64; ++turn) {
            if (wv == turn && lane < LPR) {
#pragma unroll
                for (int e = 0; e < EPL; ++e)
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        const int c = (e * LPR + l) * VEC + k;
                        s_acc[c] = turn ? s_acc[c] + aw[e][k] : aw[e][k];
                        s_acc[COLS + c] = turn ? s_acc[COLS + c] + ab[e][k] : ab[e][k];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < dim; c += NB) {
            pw[c] = s_acc[c];
            pw[dim + c] = s_acc[COLS + c];
        }
    } else {
#pragma unroll
        for (int e = 0; e < EPL; ++e)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const int c = (e * LPR + l) * VEC + k;
                if (c < dim) {
                    pw[c] = aw[e][k];
                    pw[dim + c] = ab[e][k];
                }
            }
    }
}

template <class T>
__global__ __launch_bounds__(NB) void k_norm_bwd_long(int64_t n, int dim, const T* __restrict__ x, int64_t xs,
                                                      const T* __restrict__ weight, const float* __restrict__ mean_in,
                                                      const float* __restrict__ rstd_in, const T* __restrict__ dy,
                                                      int64_t dys, T* __restrict__ dx, int64_t dxs,
                                                      float* __restrict__ part) {
    __shared__ float s_red[NB / 64];
    float* pw = part ? part + (size_t)blockIdx.x * 2 * dim : nullptr;
    bool first = true;  // the block's first row writes its column sums, later ones add to them
    for (int64_t r = blockIdx.x; r < n; r += gridDim.x) {
        const T* xr = x + r * xs;
        const T* dr = dy + r * dys;
        const float mean = mean_in[r], rstd = rstd_in[r];
        float sg = 0.f, sx = 0.f;
        for (int c = threadIdx.x; c < dim; c += NB) {
            const float d = (float)dr[c], xh = ((float)xr[c] - mean) * rstd;
            const float g = d * (weight ? (float)weight[c] : 1.f);
            sg += g;
            sx = fmaf(g, xh, sx);
            if (pw) {  // column c is this thread's in every row
                pw[c] = first ? d * xh : fmaf(d, xh, pw[c]);
                pw[dim + c] = first ? d : pw[dim + c] + d;
            }
        }
        first = false;
        if (!dx) continue;
        const float mg = row_sum<NB>(sg, s_red) / (float)dim;
        const float mx = row_sum<NB>(sx, s_red) / (float)dim;
        for (int c = threadIdx.x; c < dim; c += NB) {
            const float xh = ((float)xr[c] - mean) * rstd;
            const float g = (float)dr[c] * (weight ? (float)weight[c] : 1.f);
            dx[r * dxs + c] = (T)(rstd * (g - fmaf(xh, mx, mg)));
        }
    }
}

// Adds the blocks' column sums: RED_COLS columns per block, the rows of part
// over RED_T / RED_COLS threads, joined in LDS in a fixed order.
template <class T>
__global__ __launch_bounds__(RED_T) void k_norm_cols(int nblk, int dim, const float* __restrict__ part,
                                                     T* __restrict__ dweight, T* __restrict__ dbias) {
    constexpr int G = RED_T / RED_COLS;
    __shared__ float s[G][RED_COLS];
    const int j = threadIdx.x % RED_COLS, g = threadIdx.x / RED_COLS;
    const int c = blockIdx.x * RED_COLS + j;  // over the 2 dim columns of part
    float a = 0.f;
    if (c < 2 * dim) {
#pragma unroll 8
        for (int b = g; b < nblk; b += G) a += part[(size_t)b * 2 * dim + c];
    }
    s[g][j] = a;
    __syncthreads();
    for (int h = G / 2; h > 0; h >>= 1) {
        if (g < h) s[g][j] += s[g + h][j];
        __syncthreads();
    }
    if (g == 0 && c < 2 * dim) {
        if (c < dim) {
            if (dweight) dweight[c] = (T)s[0][j];
        } else if (dbias) {
            dbias[c - dim] = (T)s[0][j];
        }
    }
}

struct NormArgs {
    int64_t n;
    int dim;
    const void *x, *weight, *bias, *dy;
    void *y, *dx;
    int64_t xs, ys, dys, dxs;
    float eps;
    float *mean, *rstd;  // written by the forward, read by the backward
    float* part;
    int blocks;
    bool backward;
};

template <class T, int LPR, int EPL, bool FULL>
hipError_t norm_rows(NormArgs& a, int cap, hipStream_t s) {
    const int64_t want = (a.n + NB / LPR - 1) / (NB / LPR);
    a.blocks = (int)(want < cap ? want : cap);
    const T *x = (const T*)a.x, *w = (const T*)a.weight;
    if (a.backward)
        k_norm_bwd<T, LPR, EPL, FULL><<<a.blocks, NB, 0, s>>>(a.n, a.dim, x, a.xs, w, a.mean, a.rstd, (const T*)a.dy,
                                                        a.dys, (T*)a.dx, a.dxs, a.part);
    else
        k_norm_fwd<T, LPR, EPL, FULL><<<a.blocks, NB, 0, s>>>(a.n, a.dim, x, a.xs, w, (const T*)a.bias, a.eps, (T*)a.y,
                                                        a.ys, a.mean, a.rstd);
    return hipGetLastError();
}

// The lanes of a row and their accesses: the fewest lanes that hold it with one
// access each up to a wave, then more accesses, then a block.
template <class T, bool FULL>
hipError_t norm_pick(NormArgs& a, int cap, hipStream_t s) {
    const int v = (a.dim + WIDE<T> - 1) / WIDE<T>;
    if (v <= 1) return norm_rows<T, 1, 1, FULL>(a, cap, s);
    if (v <= 2) return norm_rows<T, 2, 1, FULL>(a, cap, s);
    if (v <= 4) return norm_rows<T, 4, 1, FULL>(a, cap, s);
    if (v <= 8) return norm_rows<T, 8, 1, FULL>(a, cap, s);
    if (v <= 16) return norm_rows<T, 16, 1, FULL>(a, cap, s);
    if (v <= 32) return norm_rows<T, 32, 1, FULL>(a, cap, s);
    if (v <= 64) return norm_rows<T, 64, 1, FULL>(a, cap, s);
    if (v <= 128) return norm_rows<T, 64, 2, FULL>(a, cap, s);
    if (v <= 256) return norm_rows<T, 64, 4, FULL>(a, cap, s);
    if (v <= 512) return norm_rows<T, NB, 2, FULL>(a, cap, s);
    if (v <= 1024) return norm_rows<T, NB, 4, FULL>(a, cap, s);
    return norm_rows<T, NB, 8, FULL>(a, cap, s);  // float32 only: NORM_REG_DIM is 1024 accesses of bfloat16
}

constexpr int NORM_BLOCKS_FWD = 2048;
constexpr int NORM_BLOCKS_BWD = 1024;  // rows of the column-sum array

template <class T>
hipError_t norm_launch(NormArgs& a, hipStream_t s) {
    const int cap = a.backward ? NORM_BLOCKS_BWD : NORM_BLOCKS_FWD;
    if (a.dim <= NORM_REG_DIM)
        return a.dim % WIDE<T> == 0 ? norm_pick<T, true>(a, cap, s) : norm_pick<T, false>(a, cap, s);
    a.blocks = (int)(a.n < cap ? a.n : cap);
    const T *x = (const T*)a.x, *w = (const T*)a.weight;
    if (a.backward)
        k_norm_bwd_long<T><<<a.blocks, NB, 0, s>>>(a.n, a.dim, x, a.xs, w, a.mean, a.rstd, (const T*)a.dy, a.dys,
                                                   (T*)a.dx, a.dxs, a.part);
    else
        k_norm_fwd_long<T><<<a.blocks, NB, 0, s>>>(a.n, a.dim, x, a.xs, w, (const T*)a.bias, a.eps, (T*)a.y, a.ys,
                                                   a.mean, a.rstd);
    return hipGetLastError();
}

template <class T>
hipError_t norm_bwd(NormArgs a, void* dweight, void* dbias, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (a.n > 0 && (a.dx || a.part)) e = norm_launch<T>(a, s);
    if (e != hipSuccess || (!dweight && !dbias)) return e;
    const int nblk = a.n > 0 ? a.blocks : 0;
    k_norm_cols<T><<<(2 * a.dim + RED_COLS - 1) / RED_COLS, RED_T, 0, s>>>(nblk, a.dim, a.part, (T*)dweight,
                                                                          (T*)dbias);
    return hipGetLastError();
}

}  // namespace

size_t norm_bwd_workspace(int64_t n, int dim) {
    const int64_t rows = n < NORM_BLOCKS_BWD ? n : NORM_BLOCKS_BWD;
    return ((size_t)rows * 2 * dim * sizeof(float) + 255) & ~(size_t)255;
}

hipError_t launch_norm_fwd(int64_t n, int dim, bool half, const void* x, int64_t xs, const void* weight,
                           const void* bias, float eps, void* y, int64_t ys, float* mean, float* rstd,
                           hipStream_t stream) {
    NormArgs a{};
    a.n = n;
    a.dim = dim;
    a.x = x;
    a.xs = xs;
    a.weight = weight;
    a.bias = bias;
    a.eps = eps;
    a.y = y;
    a.ys = ys;
    a.mean = mean;
    a.rstd = rstd;
    return half ? norm_launch<bf16>(a, stream) : norm_launch<float>(a, stream);
}

hipError_t launch_norm_bwd(int64_t n, int dim, bool half, const void* x, int64_t xs, const void* weight,
                           const float* mean, const float* rstd, const void* dy, int64_t dys, void* dx, int64_t dxs,
                           void* dweight, void* dbias, float* part, hipStream_t stream) {
    NormArgs a{};
    a.n = n;
    a.dim = dim;
    a.backward = true;
    a.x = x;
    a.xs = xs;
    a.weight = weight;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.dys = dys;
    a.dx = dx;
    a.dxs = dxs;
    a.part = dweight || dbias ? part : nullptr;
    return half ? norm_bwd<bf16>(a, dweight, dbias, stream) : norm_bwd<float>(a, dweight, dbias, stream);
}

}  // namespace gs
