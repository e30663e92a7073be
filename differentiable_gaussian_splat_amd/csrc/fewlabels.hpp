// The vocabulary loss of few labels (closed label sets), for labelloss.hip.
//
// With up to FEW_LABELS labels the products are too flat for tiles: the call
// is bound by reading x and writing dx. So nothing is packed: a block takes 32
// labelled rows and walks along them, its four waves each with a quarter of the
// columns (float32 products in float32, bfloat16 in bfloat16); their sums meet
// in LDS, where a row's whole softmax is formed. The gradients take a column of w and of dw's sum per thread in
// registers and walk over the rows: 2 x labels operations for each element of
// x read once and of dx written once, in float32 and without rounding dz.
// dw's sums of the blocks' row chunks are joined in order by a second launch.
//
// 46272 x 896 x 3 float32 with gradients: 864 us by the tiled products.
#pragma once

#include "elem.hpp"

namespace gs {

namespace {

constexpr int FEW_LABELS = 64;
constexpr int FT = 256;      // threads
constexpr int FR = 32;       // labelled rows of a block
constexpr int FG = 32;       // rows staged at a time by the gradient

struct FewArgs {
    int64_t n;
    int dim, vocab;
    const void *x, *w, *labels;
    int64_t xs, ws;
    int wide_labels;
    const int32_t *rows, *place, *count;
    float *loss, *lse, *mean;
    int32_t *done, *count_out;
    double* block_sum;
    const float *dmean, *dloss;
    float* g;            // [labelled rows][ldg]
    int ldg;
    void* dx;
    int64_t dxs;
    float* dw;           // [chunk][vocab][kp] sums, or null
    int kp;
    int64_t chunk;       // rows of a chunk
};

// Sixteen depth elements of a 32 x 32 product; lane: row l % 32, elements 8 (l / 32) to + 7 of each operand.
__device__ __forceinline__ f32x16 few_product(const float* a, const float* b, f32x16 c) {
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(a + i);
        *reinterpret_cast<float4*>(y + i) = *reinterpret_cast<const float4*>(b + i);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[i], y[i], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ f32x16 few_product(const bf16* a, const bf16* b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8*>(a),
                                                   *reinterpret_cast<const bf16x8*>(b), c, 0, 0, 0);
}

// The logits of 32 labelled rows, then (FORWARD) their losses and, by the block
// that ends last, the mean, or dz. VT: 32-label tiles. 128 columns at a time of
// x's rows and of w go through LDS (read along the rows; a lane per row would
// touch a line per lane), the next ones on their way in registers meanwhile.
template <class T, int VT, bool FORWARD>
__global__ __launch_bounds__(FT) void k_few_logits(FewArgs a) {
    constexpr int VP = 32 * VT, V = WIDE<T>;
    constexpr int KC = 128, PITCH = KC + V, CH = KC / V;  // columns, their row in LDS, 16-byte accesses of a row
    constexpr int RS = FT / CH;                           // rows that the block's threads read at once
    constexpr int NX = FR / RS, NW = VP / RS;
    constexpr int TILES = (FR + VP) * PITCH * (int)sizeof(T), SUMS = FT / 64 * FR * (VP + 1) * 4;
    __shared__ __align__(16) char s_mem[TILES > SUMS ? TILES : SUMS];
    __shared__ double s_loss[FR];
    __shared__ int s_last;
    T* s_x = reinterpret_cast<T*>(s_mem);
    T* s_w = s_x + FR * PITCH;
    float(*s_z)[FR][VP + 1] = reinterpret_cast<float(*)[FR][VP + 1]>(s_mem);
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int cnt = *a.count, n0 = blockIdx.x * FR;
    if (n0 < cnt) {
        const int r0 = threadIdx.x / CH, c0 = threadIdx.x % CH * V;
        int64_t row[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) row[i] = n0 + r0 + i * RS < cnt ? a.rows[n0 + r0 + i * RS] : -1;
        wide_t<T> xv[NX], wv[NW];
        auto load = [&](int k0) {
            const int c = k0 + c0, left = a.dim - c;
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const bool in = row[i] >= 0 && left > 0;
                xv[i] = (T)0.f;
                if (in) xv[i] = load_row<false>(static_cast<const T*>(a.x) + row[i] * a.xs + c, left,
                                                (a.n - 1 - row[i]) * a.xs + left);
            }
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const int v = r0 + i * RS;
                const bool in = v < a.vocab && left > 0;
                wv[i] = (T)0.f;
                if (in) wv[i] = load_row<false>(static_cast<const T*>(a.w) + v * a.ws + c, left,
                                                (a.vocab - 1 - v) * a.ws + left);
            }
        };
        f32x16 acc[VT];
#pragma unroll
        for (int t = 0; t < VT; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[t][e] = 0.f;
        load(0);
        for (int k0 = 0; k0 < a.dim; k0 += KC) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NX; ++i)
                *reinterpret_cast<wide_t<T>*>(s_x + (r0 + i * RS) * PITCH + c0) =
                    clip<false, T>(xv[i], a.dim - k0 - c0);
#pragma unroll
            for (int i = 0; i < NW; ++i)
                *reinterpret_cast<wide_t<T>*>(s_w + (r0 + i * RS) * PITCH + c0) =
                    clip<false, T>(wv[i], a.dim - k0 - c0);
            __syncthreads();
            if (k0 + KC < a.dim) load(k0 + KC);
#pragma unroll
            for (int s = 0; s < KC / 64; ++s) {  // a wave's quarter of the columns, 16 at a time
                const int c = w * (KC / 4) + 16 * s + 8 * (l / 32);
#pragma unroll
                for (int t = 0; t < VT; ++t)
                    acc[t] = few_product(s_w + (32 * t + l % 32) * PITCH + c, s_x + (l % 32) * PITCH + c, acc[t]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < VT; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                s_z[w][l % 32][32 * t + 8 * (e / 4) + 4 * (l / 32) + e % 4] = acc[t][e];
    }
    __syncthreads();
    // eight threads per row, each every eighth label
    const int r = threadIdx.x / 8, sub = threadIdx.x % 8, n = n0 + r;
    if (n < cnt) {
        float z[VP / 8];
#pragma unroll
        for (int k = 0; k < VP / 8; ++k) {
            float s = s_z[0][r][sub + 8 * k];
#pragma unroll
            for (int q = 1; q < FT / 64; ++q) s += s_z[q][r][sub + 8 * k];
            z[k] = sub + 8 * k < a.vocab ? s : -INFINITY;
        }
        const int row = a.rows[n];
        const int lab = row_index(a.labels, a.wide_labels, row, a.vocab);
        if (FORWARD) {
            float top = -INFINITY, at = 0.f;
#pragma unroll
            for (int k = 0; k < VP / 8; ++k) {
                top = fmaxf(top, z[k]);
                at = sub + 8 * k == lab ? z[k] : at;
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
            at = __shfl(at, (l & ~7) | (lab & 7));
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < VP / 8; ++k) {
                // an entry equal to the maximum counts 1, also where that is +inf; none does where it is -inf
                const float e = z[k] == top ? 1.f : exp_diff(z[k], top);
                sum += top > -INFINITY ? e : z[k] != z[k] ? z[k] : 0.f;
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
            if (sub == 0) {
                const float ln = log2f(sum) * LN2;
                const float ls = top == INFINITY ? top - at : (top - at) + ln;
                a.lse[row] = top + ln;
                a.loss[row] = ls;
                s_loss[r] = (double)ls;
            }
        } else {
            const float lse = a.lse[row];
            float up = a.dloss ? a.dloss[row] : 0.f;
            if (a.dmean) up += a.dmean[0] / (float)cnt;
#pragma unroll
            for (int k = 0; k < VP / 8; ++k) {
                const int v = sub + 8 * k;
                if (v < a.ldg) a.g[(int64_t)n * a.ldg + v] =
                    v < a.vocab ? (exp_diff(z[k], lse) - (v == lab ? 1.f : 0.f)) * up : 0.f;
            }
        }
    } else if (FORWARD && sub == 0) {
        s_loss[r] = 0.0;
    }
    if (!FORWARD) return;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int k = 0; k < FR; ++k) s += s_loss[k];
        __hip_atomic_store(&a.block_sum[blockIdx.x], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (s_last) loss_mean<FT>(a.block_sum, (int)gridDim.x, cnt, a.mean, a.count_out);
}

// C columns of a row as they are in memory (0 beyond `left`).
template <int C, class T>
struct Cols {
    T v[C];
    __device__ __forceinline__ void load(const T* p, int left) {
        typedef T vec __attribute__((ext_vector_type(C), aligned(sizeof(T))));
        if (left >= C) {
            if constexpr (C == 1) {
                v[0] = *p;
            } else {
                const vec t = *reinterpret_cast<const vec*>(p);
#pragma unroll
                for (int i = 0; i < C; ++i) v[i] = t[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = i < left ? p[i] : (T)0.f;
        }
    }
};

template <int C, class T>
__device__ __forceinline__ void store_cols(T* p, int left, const float (&v)[C]) {
    typedef T vec __attribute__((ext_vector_type(C), aligned(sizeof(T))));
    if (left >= C) {
        if constexpr (C == 1) {
            *p = (T)v[0];
        } else {
            vec t;
#pragma unroll
            for (int i = 0; i < C; ++i) t[i] = (T)v[i];
            *reinterpret_cast<vec*>(p) = t;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i < left) p[i] = (T)v[i];
    }
}

// dx and the chunks' sums of dw. VB: labels rounded up; C: columns of a thread;
// tr threads share a row, the block's other threads take other rows.
template <class T, int VB, int C>
__global__ __launch_bounds__(FT) void k_few_grads(FewArgs a, int tr) {
    __shared__ float s_g[FG][VB];
    __shared__ int s_place[FG];
    __shared__ float s_red[VB * C * (FT / 2)];  // columns x labels, where several rows are taken at once
    const int groups = FT / tr, grp = threadIdx.x / tr, t = threadIdx.x % tr;
    const int c = (blockIdx.y * tr + t) * C, left = a.dim - c;
    float w[VB][C], acc[VB][C];
#pragma unroll
    for (int v = 0; v < VB; ++v) {
#pragma unroll
        for (int k = 0; k < C; ++k) w[v][k] = acc[v][k] = 0.f;
        if (a.dx && v < a.vocab && left > 0) {
            Cols<C, T> t;
            t.load(static_cast<const T*>(a.w) + v * a.ws + c, left);
#pragma unroll
            for (int k = 0; k < C; ++k) w[v][k] = (float)t.v[k];
        }
    }
    const int64_t first = blockIdx.x * a.chunk, end = first + a.chunk < a.n ? first + a.chunk : a.n;
    for (int64_t r0 = first; r0 < end; r0 += FG) {
        __syncthreads();
        for (int i = threadIdx.x; i < FG; i += FT) s_place[i] = r0 + i < end ? a.place[r0 + i] : -1;
        __syncthreads();
        for (int i = threadIdx.x; i < FG * VB; i += FT) {
            const int p = s_place[i / VB];
            s_g[i / VB][i % VB] = p >= 0 && i % VB < a.ldg ? a.g[(int64_t)p * a.ldg + i % VB] : 0.f;
        }
        __syncthreads();
        constexpr int U = 4;
        for (int i0 = grp; i0 < FG; i0 += U * groups) {
            Cols<C, T> x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * groups;
#pragma unroll
                for (int k = 0; k < C; ++k) x[u].v[k] = (T)0.f;
                // a row without a label is not read
                if (a.dw && i < FG && s_place[i] >= 0 && left > 0)
                    x[u].load(static_cast<const T*>(a.x) + (r0 + i) * a.xs + c, left);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * groups;
                if (i >= FG || r0 + i >= end) break;
                float d[C];
#pragma unroll
                for (int k = 0; k < C; ++k) d[k] = 0.f;
                if (s_place[i] >= 0)
#pragma unroll
                    for (int v = 0; v < VB; ++v) {
                        const float g = s_g[i][v];
#pragma unroll
                        for (int k = 0; k < C; ++k) {
                            d[k] = fmaf(g, w[v][k], d[k]);
                            acc[v][k] = fmaf(g, (float)x[u].v[k], acc[v][k]);
                        }
                    }
                if (a.dx && left > 0) store_cols<C>(static_cast<T*>(a.dx) + (r0 + i) * a.dxs + c, left, d);
            }
        }
    }
    if (!a.dw) return;
    if (groups > 1) {  // the row groups' sums: within a wave, then the waves in turn
#pragma unroll
        for (int v = 0; v < VB; ++v)
#pragma unroll
            for (int k = 0; k < C; ++k)
                for (int off = tr; off < 64; off <<= 1) acc[v][k] += __shfl_xor(acc[v][k], off);
        const int turns = FT / (tr < 64 ? 64 : tr), mine = threadIdx.x / (tr < 64 ? 64 : tr);
        const bool lead = tr >= 64 || (int)(threadIdx.x & 63) < tr;
        for (int turn = 0; turn < turns; ++turn) {
            if (mine == turn && lead)
#pragma unroll
                for (int v = 0; v < VB; ++v)
#pragma unroll
                    for (int k = 0; k < C; ++k) {
                        float* q = &s_red[(v * C + k) * tr + t];
                        if (turn) acc[v][k] += *q;
                        *q = acc[v][k];
                    }
            __syncthreads();
        }
        if (mine != turns - 1 || !lead) return;  // the last turn holds the whole sum
    }
#pragma unroll
    for (int v = 0; v < VB; ++v)
        if (v < a.vocab)
#pragma unroll
            for (int k = 0; k < C; ++k)
                if (k < left) a.dw[((int64_t)blockIdx.x * a.vocab + v) * a.kp + c + k] = acc[v][k];
}

}  // namespace

}  // namespace gs
