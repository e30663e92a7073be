// The vocabulary loss where one side is short, for labelloss.hip: few labels
// (closed label sets) or few rows (a picked region against a vocabulary).
//
// With up to SHORT rows on one side the products are too flat for tiles: the
// call is bound by reading the long side (x, or w) and writing its gradient. So
// nothing is packed: a block takes 32 rows of the long side and walks along
// their columns with the whole short side beside them, its four waves each with
// a quarter of the columns (float32 products in float32, bfloat16 in
// bfloat16); their sums meet in LDS as the logits of 32 rows. With few labels
// that is a row's whole softmax; with few rows it is a slab of every row's.
// The gradients take a column of the short side, and of the sum of its
// gradient, per thread in registers and walk over the long side's rows: 2 x
// (short rows) operations for each element read once and for each element
// written once, in float32 and without rounding dz. The short side's gradient
// is summed per chunk of rows; a second launch adds the chunks in order.
//
// With gradients, float32: 46272 x 896 x 3 labels 864 us by the tiled products,
// 254 us here; 22 rows x 1003 x 5184 labels 230 us by the tiled products,
// 77 us here.
#pragma once

#include "elem.hpp"

namespace gs {

namespace {

constexpr int SHORT = 64;    // rows of the short side at most
constexpr int FT = 256;      // threads
constexpr int FR = 32;       // rows of the long side in a block
constexpr int FG = 32;       // rows staged at a time by the gradient

struct FlatArgs {
    int64_t n;
    int dim, vocab;
    const void *x, *w;
    int64_t xs, ws;
    LabelRows labels;        // its arrays: written before (few labels), or by the first kernel (few rows)
    int32_t* count_out;
    float* mean;
    double* block_sum;
    float2* part;            // few rows: [block][SHORT] (maximum, sum) pairs
    float* target;           // few rows: the logit at the label
    const float *lse, *dmean, *dloss;
    float* g;                // dz: [long row][ldg]
    int ldg;
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

// Logits of 32 rows of the long side and up to 32 VT of the short one into s_z
// (one sum per wave). long_row(i), short_row(i): the rows' numbers, -1 for
// none; l_rows, s_rows: rows of the matrices. 128 columns at a time go through
// LDS, read along the rows (a lane per row would touch a line per lane), the
// next ones on their way in registers meanwhile.
template <class T, int VT>
struct FlatTile {
    static constexpr int VP = 32 * VT, V = WIDE<T>;
    static constexpr int KC = 128, PITCH = KC + V, CH = KC / V;  // columns, their row in LDS, accesses of a row
    static constexpr int RS = FT / CH;                           // rows that the block's threads read at once
    static constexpr int NX = FR / RS, NW = VP / RS;
    static constexpr int TILES = (FR + VP) * PITCH * (int)sizeof(T), SUMS = FT / 64 * FR * (VP + 1) * 4;
    static constexpr int BYTES = TILES > SUMS ? TILES : SUMS;
    typedef float Sums[FR][VP + 1];

    template <class LR, class SR>
    static __device__ __forceinline__ void run(char* mem, const T* lp, int64_t ls, int64_t l_rows, LR long_row,
                                               const T* sp, int64_t ss, int64_t s_rows, SR short_row, int dim) {
        T* s_x = reinterpret_cast<T*>(mem);
        T* s_w = s_x + FR * PITCH;
        Sums* s_z = reinterpret_cast<Sums*>(mem);
        const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
        const int r0 = threadIdx.x / CH, c0 = threadIdx.x % CH * V;
        int64_t lr[NX], sr[NW];
#pragma unroll
        for (int i = 0; i < NX; ++i) lr[i] = long_row(r0 + i * RS);
#pragma unroll
        for (int i = 0; i < NW; ++i) sr[i] = short_row(r0 + i * RS);
        wide_t<T> xv[NX], wv[NW];
        auto load = [&](int k0) {
            const int c = k0 + c0, left = dim - c;
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                xv[i] = (T)0.f;
                if (lr[i] >= 0 && left > 0)
                    xv[i] = load_row<false>(lp + lr[i] * ls + c, left, (l_rows - 1 - lr[i]) * ls + left);
            }
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                wv[i] = (T)0.f;
                if (sr[i] >= 0 && left > 0)
                    wv[i] = load_row<false>(sp + sr[i] * ss + c, left, (s_rows - 1 - sr[i]) * ss + left);
            }
        };
        f32x16 acc[VT];
#pragma unroll
        for (int t = 0; t < VT; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[t][e] = 0.f;
        load(0);
        for (int k0 = 0; k0 < dim; k0 += KC) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NX; ++i)
                *reinterpret_cast<wide_t<T>*>(s_x + (r0 + i * RS) * PITCH + c0) = clip<false, T>(xv[i], dim - k0 - c0);
#pragma unroll
            for (int i = 0; i < NW; ++i)
                *reinterpret_cast<wide_t<T>*>(s_w + (r0 + i * RS) * PITCH + c0) = clip<false, T>(wv[i], dim - k0 - c0);
            __syncthreads();
            if (k0 + KC < dim) load(k0 + KC);
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
        __syncthreads();
    }

    static __device__ __forceinline__ float logit(const char* mem, int r, int v) {
        const Sums* s_z = reinterpret_cast<const Sums*>(mem);
        float s = s_z[0][r][v];
#pragma unroll
        for (int q = 1; q < FT / 64; ++q) s += s_z[q][r][v];
        return s;
    }
};

// Few labels: the losses of 32 labelled rows (FORWARD, and by the block that
// ends last the mean), or their dz.
template <class T, int VT, bool FORWARD>
__global__ __launch_bounds__(FT) void k_few_labels(FlatArgs a, BlockRange range) {
    using Tile = FlatTile<T, VT>;
    constexpr int VP = Tile::VP;
    __shared__ __align__(16) char s_mem[Tile::BYTES];
    __shared__ double s_loss[FR];
    __shared__ int s_last;
    const int l = threadIdx.x & 63;
    const int block = range.first + (int)blockIdx.x, cnt = *a.labels.count, n0 = block * FR;
    if (n0 < cnt)
        Tile::run(s_mem, static_cast<const T*>(a.x), a.xs, a.n,
                  [&](int i) { return n0 + i < cnt ? (int64_t)a.labels.rows[n0 + i] : (int64_t)-1; },
                  static_cast<const T*>(a.w), a.ws, a.vocab,
                  [&](int i) { return i < a.vocab ? (int64_t)i : (int64_t)-1; }, a.dim);
    // eight threads per row, each every eighth label
    const int r = threadIdx.x / 8, sub = threadIdx.x % 8, n = n0 + r;
    if (n < cnt) {
        float z[VP / 8];
#pragma unroll
        for (int k = 0; k < VP / 8; ++k)
            z[k] = sub + 8 * k < a.vocab ? Tile::logit(s_mem, r, sub + 8 * k) : -INFINITY;
        const int row = a.labels.rows[n];
        const int lab = row_index(a.labels.labels, a.labels.wide, row, a.vocab);
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
            for (int k = 0; k < VP / 8; ++k) sum += exp_share(z[k], top);
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
            if (sub == 0) {
                const float ln = log2f(sum) * LN2;
                const float ls = top == INFINITY ? top - at : (top - at) + ln;
                a.labels.lse[row] = top + ln;
                a.labels.loss[row] = ls;
                s_loss[r] = (double)ls;
            }
        } else {
            const float lse = a.lse[row], up = up_of(a.dmean, a.dloss, row, cnt);
#pragma unroll
            for (int k = 0; k < VP / 8; ++k) {
                const int v = sub + 8 * k;
                if (v < a.ldg)
                    a.g[(int64_t)n * a.ldg + v] =
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
        __hip_atomic_store(&a.block_sum[block], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last =
            __hip_atomic_fetch_add(a.labels.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == range.all - 1;
    }
    __syncthreads();
    if (s_last) loss_mean<FT>(a.block_sum, range.all, cnt, a.mean, a.count_out);
}

// Few rows (n <= SHORT): per block the (maximum, sum) pairs of every row over
// the block's labels (FORWARD; joined as the slabs of the tiled product are), or
// their dz. Each block finds the labelled rows for itself, block 0 writes their arrays.
template <class T, int VT, bool FORWARD>
__global__ __launch_bounds__(FT) void k_few_rows(FlatArgs a) {
    using Tile = FlatTile<T, VT>;
    constexpr int VP = Tile::VP, TPS = FT / VP, PER = FR / TPS;  // threads of a row, labels of each in a tile
    __shared__ __align__(16) char s_mem[Tile::BYTES];
    __shared__ int s_row[SHORT], s_lab[SHORT];
    const int lane = threadIdx.x & 63;
    const int lab = lane < a.n ? row_index(a.labels.labels, a.labels.wide, lane, a.vocab) : -1;
    const uint64_t have = __ballot(lab >= 0);
    const int cnt = __popcll(have), to = __popcll(have & (((uint64_t)1 << lane) - 1));
    if (threadIdx.x < SHORT) {
        if (lab >= 0) {
            s_row[to] = lane;
            s_lab[to] = lab;
        }
        if (blockIdx.x == 0 && lane < a.n) {
            a.labels.place[lane] = lab >= 0 ? to : -1;
            if (lab >= 0) a.labels.rows[to] = lane;
            if (lab < 0 && a.labels.loss) a.labels.loss[lane] = 0.f;
            if (lab < 0 && a.labels.lse) a.labels.lse[lane] = 0.f;
        }
        if (blockIdx.x == 0 && lane == 0) {
            *a.labels.count = cnt;
            *a.labels.done = 0;
        }
    }
    __syncthreads();
    const int s = threadIdx.x / TPS, sub = threadIdx.x % TPS;
    const int row = s < cnt ? s_row[s] : 0, mine = s < cnt ? s_lab[s] : -1;
    float top = -INFINITY, sum = 0.f, lse = 0.f, up = 0.f;
    if (!FORWARD && s < cnt) {
        lse = a.lse[row];
        up = up_of(a.dmean, a.dloss, row, cnt);
    }
    for (int64_t v0 = (int64_t)blockIdx.x * FR; v0 < a.vocab; v0 += (int64_t)gridDim.x * FR) {
        __syncthreads();  // the last tile's logits are read
        Tile::run(s_mem, static_cast<const T*>(a.w), a.ws, a.vocab,
                  [&](int i) { return v0 + i < a.vocab ? v0 + i : (int64_t)-1; }, static_cast<const T*>(a.x), a.xs,
                  a.n, [&](int i) { return i < cnt ? (int64_t)s_row[i] : (int64_t)-1; }, a.dim);
        float z[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int64_t v = v0 + sub + k * TPS;
            z[k] = v < a.vocab ? Tile::logit(s_mem, sub + k * TPS, s) : -INFINITY;
            if (FORWARD) {
                if (v == mine && s < cnt) a.target[s] = z[k];
            } else if (s < a.ldg && v < a.vocab) {
                a.g[v * a.ldg + s] = s < cnt ? (exp_diff(z[k], lse) - (v == mine ? 1.f : 0.f)) * up : 0.f;
            }
        }
        if (FORWARD) {
            float t = top;
#pragma unroll
            for (int k = 0; k < PER; ++k) t = fmaxf(t, z[k]);
            float2 j = make_float2(t, 0.f);
#pragma unroll
            for (int k = 0; k < PER; ++k) j.y += exp_share(z[k], t);
            j = lse_join(make_float2(top, sum), j);
            top = j.x;
            sum = j.y;
        }
    }
    if (!FORWARD) return;
    float2 j = make_float2(top, sum);
#pragma unroll
    for (int off = TPS / 2; off > 0; off >>= 1)
        j = lse_join(j, make_float2(__shfl_xor(j.x, off), __shfl_xor(j.y, off)));
    if (sub == 0 && s < cnt) a.part[(int64_t)blockIdx.x * SHORT + s] = j;
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

struct FlatGrads {
    int64_t rows;            // of the long side
    int dim, kp;
    const int32_t* place;    // few labels: a long row's row of g, -1 for none; null: its own
    const float* g;
    int ldg;
    const void *lp, *sp;     // long and short side
    int64_t ls, ss;
    const int32_t *list, *count;  // few rows: the short side's rows and their number
    int short_rows;               // few labels: their number
    void* dlong;                  // nullable
    int64_t dls;
    float* dshort;                // nullable: [chunk][out_rows][kp]
    int out_rows;
    int64_t chunk;                // long rows of a chunk
};

// The long side's gradient and the chunks' sums of the short side's. VB: short
// rows rounded up; C: columns of a thread; tr threads share a row, the block's
// other threads take other rows.
template <class T, int VB, int C>
__global__ __launch_bounds__(FT) void k_flat_grads(FlatGrads a, int tr) {
    __shared__ float s_g[FG][VB];
    __shared__ int s_place[FG];
    // sums of the waves (or their pairs), where several long rows are taken at once
    __shared__ float s_red[VB * C * FT];
    const int groups = FT / tr, grp = threadIdx.x / tr, t = threadIdx.x % tr;
    const int c = (blockIdx.y * tr + t) * C, left = a.dim - c;
    const int ns = a.count ? *a.count : a.short_rows;
    const int lane = threadIdx.x & 63;
    const int listed = a.list && lane < ns ? a.list[lane] : lane;  // the lane's short row: read once, not per row below
    float w[VB][C], acc[VB][C];
#pragma unroll
    for (int v = 0; v < VB; ++v) {
        const int row = __builtin_amdgcn_readlane(listed, v);
#pragma unroll
        for (int k = 0; k < C; ++k) w[v][k] = acc[v][k] = 0.f;
        if (a.dlong && v < ns && left > 0) {
            Cols<C, T> q;
            q.load(static_cast<const T*>(a.sp) + row * a.ss + c, left);
#pragma unroll
            for (int k = 0; k < C; ++k) w[v][k] = (float)q.v[k];
        }
    }
    const int64_t first = blockIdx.x * a.chunk, end = first + a.chunk < a.rows ? first + a.chunk : a.rows;
    for (int64_t r0 = first; r0 < end; r0 += FG) {
        __syncthreads();
        for (int i = threadIdx.x; i < FG; i += FT)
            s_place[i] = r0 + i >= end ? -1 : a.place ? a.place[r0 + i] : (int)(r0 + i);
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
                if (a.dshort && i < FG && s_place[i] >= 0 && left > 0)
                    x[u].load(static_cast<const T*>(a.lp) + (r0 + i) * a.ls + c, left);
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
                if (a.dlong && left > 0) store_cols<C>(static_cast<T*>(a.dlong) + (r0 + i) * a.dls + c, left, d);
            }
        }
    }
    if (!a.dshort) return;
    if (groups > 1) {  // the row groups' sums: within a wave, then the waves in turn
#pragma unroll
        for (int v = 0; v < VB; ++v)
#pragma unroll
            for (int k = 0; k < C; ++k)
                for (int off = tr; off < 64; off <<= 1) acc[v][k] += __shfl_xor(acc[v][k], off);
        const int parts = FT / (tr < 64 ? 64 : tr), mine = threadIdx.x / (tr < 64 ? 64 : tr), size = VB * C * tr;
        if (tr >= 64 || (int)(threadIdx.x & 63) < tr)
#pragma unroll
            for (int v = 0; v < VB; ++v)
#pragma unroll
                for (int k = 0; k < C; ++k) s_red[mine * size + (v * C + k) * tr + t] = acc[v][k];
        __syncthreads();
        for (int i = threadIdx.x; i < ns * C * tr; i += FT) {
            float sum = s_red[i];
            for (int q = 1; q < parts; ++q) sum += s_red[q * size + i];
            const int v = i / (C * tr), k = i / tr % C, col = (blockIdx.y * tr + i % tr) * C + k;
            if (col < a.dim) a.dshort[((int64_t)blockIdx.x * a.out_rows + v) * a.kp + col] = sum;
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < VB; ++v)
        if (v < ns)
#pragma unroll
            for (int k = 0; k < C; ++k)
                if (k < left) a.dshort[((int64_t)blockIdx.x * a.out_rows + v) * a.kp + c + k] = acc[v][k];
}

// The same for more than 16 short rows, float32, on the matrix units (float32
// products, 32 x 32 x 2): a wave holds 32 columns, and for 32 long rows at a
// time multiplies their dz with the short side's columns and with their own.
// Operands lie in LDS with pitches that put a wave's 64 words in different
// banks (an odd multiple of 32 words; 33 for dz, which is read both ways).
// 46272 x 896 x 64: 292 us with the sums in the vector units, 146 us here (332 MB
// read and written, 2.3 TB/s; the products alone would take 80 us).
template <int VT>
__global__ __launch_bounds__(FT) void k_flat_products(FlatGrads a) {
    constexpr int VP = 32 * VT, CB = 128, PC = CB + 32;
    __shared__ __align__(16) float s_s[VP][PC];  // the short side's columns
    __shared__ __align__(16) float s_l[FR][PC];  // 32 long rows' columns
    __shared__ float s_g[VP][FR + 1];            // their dz, read along either side
    __shared__ int s_place[2][FR];
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, h = l / 32;
    const int ns = a.count ? *a.count : a.short_rows;
    const int c0 = blockIdx.y * CB;
    const int lr = threadIdx.x / 32, lc = threadIdx.x % 32 * 4, left = a.dim - c0 - lc;  // a thread's part of a tile
    for (int v = lr; v < VP; v += 8) {
        wide_t<float> t = 0.f;
        if (a.dlong && v < ns && left > 0) {
            const int64_t row = a.list ? a.list[v] : v;
            t = clip<false, float>(load_row<false>(static_cast<const float*>(a.sp) + row * a.ss + c0 + lc, left, left),
                                   left);
        }
        *reinterpret_cast<wide_t<float>*>(&s_s[v][lc]) = t;
    }
    const int64_t first = blockIdx.x * a.chunk, end = first + a.chunk < a.rows ? first + a.chunk : a.rows;
    f32x16 sums[VT];
#pragma unroll
    for (int t = 0; t < VT; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) sums[t][e] = 0.f;
    wide_t<float> next_l[4];
    float next_g[VP / 8];
    auto place_of = [&](int64_t r) { return r >= end ? -1 : a.place ? a.place[r] : (int)r; };
    auto load = [&](int64_t r0, const int* place) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            next_l[i] = 0.f;
            if (a.dshort && place[lr + 8 * i] >= 0 && left > 0)  // a row without a label is not read
                next_l[i] = load_row<false>(static_cast<const float*>(a.lp) + (r0 + lr + 8 * i) * a.ls + c0 + lc, left,
                                            (a.rows - 1 - r0 - lr - 8 * i) * a.ls + left);
        }
#pragma unroll
        for (int i = 0; i < VP / 8; ++i) {
            const int k = threadIdx.x + FT * i, p = place[k / VP];
            next_g[i] = p >= 0 && k % VP < a.ldg ? a.g[(int64_t)p * a.ldg + k % VP] : 0.f;
        }
    };
    if (threadIdx.x < FR) s_place[0][threadIdx.x] = place_of(first + threadIdx.x);
    __syncthreads();
    load(first, s_place[0]);
    int now = 0;
    for (int64_t r0 = first; r0 < end; r0 += FR, now ^= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<wide_t<float>*>(&s_l[lr + 8 * i][lc]) = clip<false, float>(next_l[i], left);
#pragma unroll
        for (int i = 0; i < VP / 8; ++i) {
            const int k = threadIdx.x + FT * i;
            s_g[k % VP][k / VP] = next_g[i];
        }
        if (threadIdx.x < FR) s_place[now ^ 1][threadIdx.x] = place_of(r0 + FR + threadIdx.x);
        __syncthreads();
        if (r0 + FR < end) load(r0 + FR, s_place[now ^ 1]);
        const int col = w * 32 + l % 32;
        if (a.dlong) {
            f32x16 d;
#pragma unroll
            for (int e = 0; e < 16; ++e) d[e] = 0.f;
#pragma unroll 8
            for (int v = 0; v < VP; v += 2)
                d = __builtin_amdgcn_mfma_f32_32x32x2f32(s_s[v + h][col], s_g[v + h][l % 32], d, 0, 0, 0);
            const int64_t r = r0 + l % 32;
            if (r < end) {
                const bool have = s_place[now][l % 32] >= 0;
                float* q = static_cast<float*>(a.dlong) + r * a.dls;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const int c = c0 + w * 32 + 2 * e + 4 * h;
                    float o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[k] = have ? d[e + k] : 0.f;
                    if (c < a.dim) store_row<false>(q + c, a.dim - c, o);
                }
            }
        }
        if (a.dshort)
#pragma unroll 8
            for (int r = 0; r < FR; r += 2)
#pragma unroll
                for (int t = 0; t < VT; ++t)
                    sums[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(s_l[r + h][col], s_g[32 * t + l % 32][r + h],
                                                                  sums[t], 0, 0, 0);
        __syncthreads();
    }
    if (!a.dshort) return;
#pragma unroll
    for (int t = 0; t < VT; ++t) {
        const int v = 32 * t + l % 32;
        if (v >= ns) continue;
        float* q = a.dshort + ((int64_t)blockIdx.x * a.out_rows + v) * a.kp;
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const int c = c0 + w * 32 + 2 * e + 4 * h;
            const float o[4] = {sums[t][e], sums[t][e + 1], sums[t][e + 2], sums[t][e + 3]};
            if (c < a.dim) store_row<false>(q + c, a.dim - c, o);
        }
    }
}

}  // namespace

}  // namespace gs
