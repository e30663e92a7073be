// Softmax cross entropy of feature rows against a vocabulary of label rows,
// and its gradients, without a matrix of logits.
//
//   z_iv = x_i . w_v,  lse_i = log sum_v exp z_iv,  loss_i = lse_i - z_i,label(i)
//   dz_iv = up_i (exp(z_iv - lse_i) - [v = label(i)])
//   dx_i = sum_v dz_iv w_v,  dw_v = sum_i dz_iv x_i
//
// All of it is matrix products (2 n V D operations each) on the bfloat16 matrix
// units, with the softmax in the products' epilogues:
//   forward   each tile of z leaves, per row, its maximum and the sum of
//             exp(z - maximum) over a slab of the vocabulary; a second launch
//             joins the slabs.
//   backward  piece by piece of the vocabulary: z is formed again (one product
//             more than keeping it, against 4 bytes per logit written and read
//             back), its epilogue writes dz of the piece to the workspace, and
//             two products read it: dx += dz w and dw = dz^T x.
// Rows without a label are left out before the products: a list of the
// labelled rows is made first, x is packed through it, and the number of tiles
// follows the count on the device, so unlabelled rows (whatever they hold)
// cost nothing and reach no sum.
//
// Types. bfloat16 rows are multiplied as they are, with float32 sums; dz is
// rounded to bfloat16 (half a step, 2^-9 of each value, independent between
// entries, so it stays below the rounding of dx and dw to the same type).
// float32 rows are split into three bfloat16 parts (8 + 8 + 8 bits: the value
// to 2^-24) and six products of parts are summed, smallest first; what is left
// out is below 2^-24 of the product of magnitudes, a float32 product's own
// rounding. The matrix units take bfloat16 sixteen times as fast as float32,
// so six products are cheaper than one.
#include "elem.hpp"
#include "launch.hpp"

namespace gs {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define LDS_PTR(p) ((__attribute__((address_space(3))) void*)(p))

constexpr int BT = 128;         // tile edge of every product, rows and columns
constexpr int BK = 64;          // depth of one staged step
constexpr int GT = 256;         // threads: 2 x 2 waves of 64 x 64
constexpr int SLAB = 64;        // vocabulary rows one wave sums: one (maximum, sum) pair per row
constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;

enum Mode { LSE, DZ, DX, DW };

struct Product {
    const bf16 *a, *b;            // operands: rows of tiles, or (transposed) rows along the depth
    int64_t lda, ldb, pa, pb;     // row strides and distance between the parts of a split operand
    int m, n, k;                  // n, k: host bounds where the device count does not give them
    int splits;                   // of the depth
    const int32_t* count;         // labelled rows
    // epilogues
    const int32_t* rows;          // labelled row -> row of the caller's arrays
    const void* labels;
    int wide_labels;
    int v0, vocab, np, slab0;
    float2* part;                 // LSE: [slab][np]
    float* target;                // LSE: z at the label
    const float *lse, *dmean, *dloss;
    bf16* dz;                     // DZ: [parts][np][lddz]
    int64_t lddz, pdz;
    float* acc;                   // DX, DW with splits: [split][rows][ldacc]
    int64_t ldacc, pacc;
    int add;
    void* out;                    // DW without splits
    int64_t ldout;
    int out_dim;
};

__device__ __forceinline__ float up_of(const Product& p, int row, int cnt) {
    float u = p.dloss ? p.dloss[row] : 0.f;
    if (p.dmean) u += p.dmean[0] / (float)cnt;
    return u;
}

// Stages a BT x BK operand tile into LDS: rows of 64 depth elements (128
// bytes, 16-byte chunks exchanged by the row's low bits so that the readers of
// one depth chunk spread over the banks) or, TR, depth rows of BT elements
// (64-byte segments exchanged by the depth row's low bits).
template <bool TR>
struct Stage {
    uint32_t off[4];  // byte offsets of the lane's chunks from the tile's first element

    __device__ __forceinline__ Stage(int64_t ld) {
        const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (TR) {
                const int r = (i * 4 + w) * 4 + l / 16;
                const int seg = ((l % 16) / 4) ^ (r & 3);
                off[i] = (uint32_t)((r * ld + seg * 32 + (l % 4) * 8) * 2);
            } else {
                const int r = (i * 4 + w) * 8 + l / 8;
                off[i] = (uint32_t)((r * ld + ((l % 8) ^ (r & 7)) * 8) * 2);
            }
        }
    }

    // p: first element of the tile; bytes: how far the operand's memory reaches from there (reads beyond give 0)
    __device__ __forceinline__ void load(const bf16* p, int64_t bytes, bf16* lds) const {
        const int w = threadIdx.x >> 6;
        const int lim = bytes > 0x7fffffff ? 0x7fffffff : bytes < 0 ? 0 : (int)bytes;
        auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<bf16*>(p), 0, lim, 0x00020000);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, LDS_PTR(lds + (i * 4 + w) * 512), 16, off[i], 0, 0, 0);
    }
};

// The 8 depth elements of a lane for one 32-row fragment: row `r0 + lane % 32`, depth 16 kk + 8 (lane / 32).
template <bool TR>
__device__ __forceinline__ bf16x8 fragment(const bf16* lds, int r0, int kk) {
    const int l = threadIdx.x & 63;
    if constexpr (TR) {
        const int j = l % 16, k = 16 * kk + 8 * (l / 32) + j / 4;
        const bf16* q = lds + k * BT + (((r0 / 32) ^ (j / 4)) * 32) + ((l / 16) & 1) * 16 + (j % 4) * 4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)q);
        const s16x4 hi =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(q + 4 * BT));
        bf16x8 v;
        __builtin_memcpy(&v, &lo, 8);
        __builtin_memcpy(reinterpret_cast<char*>(&v) + 8, &hi, 8);
        return v;
    } else {
        const int r = r0 + l % 32;
        return *reinterpret_cast<const bf16x8*>(lds + r * BK + ((2 * kk + l / 32) ^ (r & 7)) * 8);
    }
}

// exp(z - ref); the difference first, which is exact where the two are close. Results below 2^-126 are 0.
__device__ __forceinline__ float exp_diff(float z, float ref) { return __builtin_amdgcn_exp2f((z - ref) * LOG2E); }

// One product, C[m][n] = sum_k A[m][k] B[n][k], by 128 x 128 tiles; a lane
// holds, for one n, runs of four consecutive m. PARTS: 1, or 3 for split
// operands.
template <int MODE, int PARTS, class T>
__global__ __launch_bounds__(GT, 2) void k_product(Product p) {
    constexpr bool TA = MODE == DX || MODE == DW, TB = MODE == DW;
    __shared__ __align__(16) bf16 s_a[2][BT * BK];
    __shared__ __align__(16) bf16 s_b[2][BT * BK];
    const int cnt = *p.count;
    const int nn = MODE == DW ? p.n : cnt;
    const int mt = (p.m + BT - 1) / BT, nt = (nn + BT - 1) / BT;
    // consecutive blocks go to the eight dies in turn: each takes a contiguous
    // run of tiles, in groups of 8 columns, so that its cache serves both operands
    const int tiles = mt * nt, per_die = (tiles + 7) / 8;
    const int tile = (blockIdx.x & 7) * per_die + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per_die || tile >= tiles) return;
    const int grp = tile / (8 * mt), in_grp = tile - grp * 8 * mt;
    const int gw = min(8, nt - grp * 8);
    const int m0 = in_grp / gw * BT, n0 = (grp * 8 + in_grp % gw) * BT;

    const int depth = MODE == DW ? cnt : p.k;
    const int nk = (depth + BK - 1) / BK;
    const int share = (nk + p.splits - 1) / p.splits;
    const int k_first = min(nk, (int)blockIdx.y * share), k_end = min(nk, k_first + share);
    const int steps = (k_end - k_first) * (PARTS == 3 ? 6 : 1);

    const Stage<TA> sa(p.lda);
    const Stage<TB> sb(p.ldb);
    const int a_rows = TA ? (MODE == DW ? p.np : p.k) : p.m;  // rows of the operand's memory
    const int b_rows = p.np;
    auto issue = [&](int t, int buf) {
        int ia = 0, ib = 0, kt = t;
        if (PARTS == 3) {
            const int per = k_end - k_first, pr = t / per;
            kt = t - pr * per;
            ia = (0x001012 >> (4 * pr)) & 3;  // 2 1 0 1 0 0
            ib = (0x010210 >> (4 * pr)) & 3;  // 0 1 2 0 1 0
        }
        const int k0 = (k_first + kt) * BK;
        const bf16* a = p.a + ia * p.pa;
        const bf16* b = p.b + ib * p.pb;
        if (TA)
            sa.load(a + k0 * p.lda + m0, ((int64_t)(min(BK, a_rows - k0) - 1) * p.lda + p.m - m0) * 2, s_a[buf]);
        else
            sa.load(a + m0 * p.lda + k0, ((int64_t)(min(BT, a_rows - m0) - 1) * p.lda + BK) * 2, s_a[buf]);
        if (TB)
            sb.load(b + k0 * p.ldb + n0, ((int64_t)(min(BK, b_rows - k0) - 1) * p.ldb + p.ldb - n0) * 2, s_b[buf]);
        else
            sb.load(b + n0 * p.ldb + k0, ((int64_t)(min(BT, b_rows - n0) - 1) * p.ldb + BK) * 2, s_b[buf]);
    };

    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int wm = (w & 1) * 64, wn = (w >> 1) * 64;
    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

    if (steps > 0) issue(0, 0);
    for (int t = 0; t < steps; ++t) {
        const int buf = t & 1;
        __syncthreads();  // step t has arrived, and the other buffer's readers are done
        if (t + 1 < steps) issue(t + 1, buf ^ 1);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
            bf16x8 fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) fa[i] = fragment<TA>(s_a[buf], wm + 32 * i, kk);
#pragma unroll
            for (int j = 0; j < 2; ++j) fb[j] = fragment<TB>(s_b[buf], wn + 32 * j, kk);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
        }
    }

    // element e of acc[i][j]: m = mb + 32 i + 8 (e / 4) + e % 4, n = nb + 32 j
    const int mb = m0 + wm + 4 * (l / 32), nb = n0 + wn + l % 32;
    if constexpr (MODE == LSE || MODE == DZ) {
        const bool edge = m0 + BT > p.m;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int n = nb + 32 * j;
            const int row = n < cnt ? p.rows[n] : -1;
            const int lab = row >= 0 ? row_index(p.labels, p.wide_labels, row, p.vocab) - p.v0 : -1;
            const bool hit = __any(lab >= m0 + wm && lab < m0 + wm + SLAB);
            if constexpr (MODE == LSE) {
                if (edge)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (mb + 32 * i + 8 * (e / 4) + e % 4 >= p.m) acc[i][j][e] = -INFINITY;
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) top = fmaxf(top, acc[i][j][e]);
                top = fmaxf(top, __shfl_xor(top, 32));
                // an infinite maximum: entries equal to it count 1 (+inf) or 0 (-inf), others 0
                const bool fin = top > -INFINITY && top < INFINITY;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float z = acc[i][j][e];
                        sum += fin ? exp_diff(z, top) : z != z ? z : z == INFINITY ? 1.f : 0.f;
                    }
                sum += __shfl_xor(sum, 32);
                if (l < 32 && n < cnt)
                    p.part[(int64_t)(p.slab0 + (m0 + wm) / SLAB) * p.np + n] = make_float2(top, sum);
                if (hit)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (lab >= 0 && mb + 32 * i + 8 * (e / 4) + e % 4 == lab) p.target[n] = acc[i][j][e];
            } else {
                const float lse = row >= 0 ? p.lse[row] : 0.f;
                const float up = row >= 0 ? up_of(p, row, cnt) : 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const int m = mb + 32 * i + 2 * e;
                        bf16x4 o[PARTS];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float g = exp_diff(acc[i][j][e + q], lse);
                            if (hit && lab == m + q) g -= 1.f;
                            g *= up;
                            if (row < 0 || m + q >= p.m) g = 0.f;
                            o[0][q] = (bf16)g;
                            if (PARTS == 3) {
                                const float r1 = g - (float)o[0][q];
                                o[PARTS / 2][q] = (bf16)r1;
                                o[PARTS - 1][q] = (bf16)(r1 - (float)o[PARTS / 2][q]);
                            }
                        }
#pragma unroll
                        for (int c = 0; c < PARTS; ++c)
                            *reinterpret_cast<bf16x4*>(p.dz + c * p.pdz + n * p.lddz + m) = o[c];
                    }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int n = nb + 32 * j;
            if (n >= nn) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const int m = mb + 32 * i + 2 * e;
                    if (p.acc) {
                        if (m >= p.ldacc) continue;
                        float4* q = reinterpret_cast<float4*>(p.acc + blockIdx.y * p.pacc + n * p.ldacc + m);
                        float4 v = make_float4(acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]);
                        if (p.add) {
                            const float4 o = *q;
                            v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
                        }
                        *q = v;
                    } else {
                        T* q = static_cast<T*>(p.out) + n * p.ldout + m;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (m + c < p.out_dim) q[c] = (T)acc[i][j][e + c];
                    }
                }
        }
    }
}

// ---------------------------------------------------------------- labelled rows

constexpr int LT = 1024;          // threads
constexpr int LPT = 8;            // consecutive rows per thread
constexpr int LROWS = LT * LPT;   // rows per block

__device__ __forceinline__ int block_scan_excl(int v, int* s_w, int* total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int x = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(x, off);
        if (lane >= off) x += y;
    }
    if (lane == 63) s_w[w] = x;
    __syncthreads();
    int pre = 0, tot = 0;
    for (int k = 0; k < LT / 64; ++k) {
        pre += k < w ? s_w[k] : 0;
        tot += s_w[k];
    }
    __syncthreads();
    *total = tot;
    return pre + x - v;
}

__global__ __launch_bounds__(LT) void k_label_count(int64_t n, int vocab, const void* __restrict__ labels, bool wide,
                                                    int32_t* __restrict__ block_count) {
    __shared__ int s_w[LT / 64];
    const int64_t r0 = (int64_t)blockIdx.x * LROWS + threadIdx.x * LPT;
    int c = 0;
#pragma unroll
    for (int k = 0; k < LPT; ++k) c += r0 + k < n && row_index(labels, wide, r0 + k, vocab) >= 0;
    int tot;
    block_scan_excl(c, s_w, &tot);
    if (threadIdx.x == 0) block_count[blockIdx.x] = tot;
}

// rows[]: the labelled rows in order; place[r]: the position of row r in it, or
// -1; the count. loss and lse (nullable) are cleared for rows without a label.
__global__ __launch_bounds__(LT) void k_label_rows(int64_t n, int vocab, const void* __restrict__ labels, bool wide,
                                                   const int32_t* __restrict__ block_count,
                                                   int32_t* __restrict__ rows, int32_t* __restrict__ place,
                                                   int32_t* __restrict__ count, float* __restrict__ loss,
                                                   float* __restrict__ lse) {
    __shared__ int s_w[LT / 64];
    int base = 0;
    if (gridDim.x > 1) {
        int c = 0;
        for (int k = threadIdx.x; k < (int)blockIdx.x; k += LT) c += block_count[k];
        block_scan_excl(c, s_w, &base);
    }
    const int64_t r0 = (int64_t)blockIdx.x * LROWS + threadIdx.x * LPT;
    bool have[LPT];
    int c = 0;
#pragma unroll
    for (int k = 0; k < LPT; ++k) {
        have[k] = r0 + k < n && row_index(labels, wide, r0 + k, vocab) >= 0;
        c += have[k];
    }
    int tot;
    int at = base + block_scan_excl(c, s_w, &tot);
#pragma unroll
    for (int k = 0; k < LPT; ++k) {
        const int64_t r = r0 + k;
        if (r >= n) break;
        place[r] = have[k] ? at : -1;
        if (have[k]) {
            rows[at++] = (int32_t)r;
        } else {
            if (loss) loss[r] = 0.f;
            if (lse) lse[r] = 0.f;
        }
    }
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) *count = base + tot;
}

// Rows into bfloat16 parts of kp columns (a multiple of BK, zero beyond dim).
// With a list: the listed rows, and zero rows up to the next multiple of BT.
template <class T, int PARTS>
__global__ __launch_bounds__(256) void k_pack(int64_t rows, int dim, int kp, const T* __restrict__ x, int64_t xs,
                                              bool wide, const int32_t* __restrict__ list,
                                              const int32_t* __restrict__ count, bf16* __restrict__ out,
                                              int64_t part) {
    const int per = kp / 8;
    int64_t live = rows, padded = rows;
    if (list) {
        live = *count;
        padded = (live + BT - 1) / BT * BT;
    }
    const int64_t total = padded * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per;
        const int c = (int)(i - r * per) * 8;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
        if (r < live) {
            const T* q = x + (list ? (int64_t)list[r] : r) * xs + c;
            if (wide && c + 8 <= dim) {
                constexpr int V = WIDE<T>;
#pragma unroll
                for (int k = 0; k < 8; k += V) {
                    float t[V];
                    load_row<V>(q + k, t);
#pragma unroll
                    for (int j = 0; j < V; ++j) v[k + j] = t[j];
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + k < dim) v[k] = (float)q[k];
            }
        }
        bf16x8 o[PARTS];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            o[0][k] = (bf16)v[k];
            if (PARTS == 3) {
                // a value that would round up to infinity keeps its leading bits instead; an
                // infinite or NaN value stays in its first part alone
                const bool fin = fabsf(v[k]) < INFINITY;
                if (fin && !(fabsf((float)o[0][k]) < INFINITY))
                    o[0][k] = (bf16)__uint_as_float(__float_as_uint(v[k]) & 0xffff0000u);
                const float r1 = fin ? v[k] - (float)o[0][k] : 0.f;
                o[PARTS / 2][k] = (bf16)r1;
                o[PARTS - 1][k] = (bf16)(r1 - (float)o[PARTS / 2][k]);
            }
        }
#pragma unroll
        for (int q = 0; q < PARTS; ++q) *reinterpret_cast<bf16x8*>(out + q * part + r * kp + c) = o[q];
    }
}

// ---------------------------------------------------------------- joins

__device__ __forceinline__ float2 lse_join(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x);
    // an equal maximum scales by 1 (also where both are infinite); sums are 0 where the maximum is -inf
    const float fa = a.x == m ? 1.f : exp_diff(a.x, m), fb = b.x == m ? 1.f : exp_diff(b.x, m);
    return make_float2(m, a.y * fa + b.y * fb);
}

constexpr int JR = 64;  // rows per block of the join
constexpr int JT = 256;

// Joins the slabs' (maximum, sum) pairs of each labelled row (and `state`, the
// join of earlier pieces, with `more` pieces to come left there again), then
// the row's loss; block_sum: the block's losses added.
__global__ __launch_bounds__(JT) void k_lse_join(int slabs, int np, const float2* __restrict__ part,
                                                 const float* __restrict__ target, const int32_t* __restrict__ rows,
                                                 const int32_t* __restrict__ count, float2* __restrict__ state,
                                                 bool first, bool more, float* __restrict__ loss,
                                                 float* __restrict__ lse, double* __restrict__ block_sum) {
    __shared__ float2 s[JT / JR][JR];
    __shared__ double s_sum;
    const int j = threadIdx.x % JR, g = threadIdx.x / JR;
    const int n = blockIdx.x * JR + j, cnt = *count;
    float2 a = make_float2(-INFINITY, 0.f);
    if (n < cnt) {
        if (!first && g == 0) a = state[n];
#pragma unroll 4
        for (int k = g; k < slabs; k += JT / JR) a = lse_join(a, part[(int64_t)k * np + n]);
    }
    s[g][j] = a;
    __syncthreads();
    if (g == 0) {
        double mine = 0.0;
        if (n < cnt) {
            for (int k = 1; k < JT / JR; ++k) a = lse_join(a, s[k][j]);
            if (more) {
                state[n] = a;
            } else {
                const float v = a.x + log2f(a.y) * LN2;
                const float z = target[n];
                const int r = rows[n];
                // (maximum - z) first: exact where they are close
                const float ls = a.x == INFINITY ? a.x - z : (a.x - z) + log2f(a.y) * LN2;
                lse[r] = v;
                loss[r] = ls;
                mine = (double)ls;
            }
        }
        for (int off = 32; off > 0; off >>= 1) mine += __shfl_xor(mine, off);
        if (j == 0) s_sum = mine;
    }
    __syncthreads();
    if (threadIdx.x == 0) block_sum[blockIdx.x] = s_sum;
}

__global__ __launch_bounds__(LT) void k_loss_mean(const double* __restrict__ block_sum,
                                                  const int32_t* __restrict__ count, float* __restrict__ mean,
                                                  int32_t* __restrict__ count_out) {
    __shared__ double s[LT / 64];
    const int cnt = *count, blocks = (cnt + JR - 1) / JR;
    double a = 0.0;
    for (int k = threadIdx.x; k < blocks; k += LT) a += block_sum[k];
    for (int off = 32; off > 0; off >>= 1) a += __shfl_xor(a, off);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < LT / 64; ++k) a += s[k];
        *mean = cnt > 0 ? (float)(a / (double)cnt) : 0.f;
        *count_out = cnt;
    }
}

// out[r] = the splits' rows added in order, through place (-1: a zero row) if given.
template <class T>
__global__ __launch_bounds__(256) void k_join_splits(int64_t rows, int dim, int splits, const float* __restrict__ acc,
                                                     int64_t ldacc, int64_t pacc, const int32_t* __restrict__ place,
                                                     T* __restrict__ out, int64_t ldout) {
    const int lane = threadIdx.x & 63;
    for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < rows; r += (int64_t)gridDim.x * 4) {
        const int64_t src = place ? place[r] : r;
        for (int c = lane; c < dim; c += 64) {
            float a = 0.f;
            if (src >= 0)
                for (int s = 0; s < splits; ++s) a += acc[s * pacc + src * ldacc + c];
            out[r * ldout + c] = (T)a;
        }
    }
}

// ---------------------------------------------------------------- plan

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

struct LossPlan {
    int parts, kp;
    int64_t np;                    // rows of x padded to the tile
    int64_t piece_f, piece_b;      // vocabulary rows per piece (multiples of BT)
    int split_dx, split_dw;
    size_t rows, place, count, block_count, xp, wp, part, target, state, block_sum, dz, dxp, dwp, total;
};

// Blocks a launch needs to fill the chip; products with fewer tiles split their depth.
constexpr int FILL = 512;

int splits_for(int64_t tiles, int64_t nk) {
    int64_t s = tiles > 0 ? FILL / tiles : 1;
    if (s > nk / 4) s = nk / 4;  // at least four steps each
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

LossPlan loss_plan(int64_t n, int dim, int vocab, bool half, bool backward) {
    LossPlan L{};
    L.parts = half ? 1 : 3;
    L.kp = (int)up(dim, BK);
    L.np = up(n > 0 ? n : 1, BT);
    const int64_t vp = up(vocab, BT);
    auto piece = [&](int64_t budget) {  // vocabulary rows whose per-row cost fits the budget
        const int64_t v = budget / L.np / BT * BT;
        return v < BT ? BT : v > vp ? vp : v;
    };
    L.piece_f = piece((int64_t)1 << 31);  // 8 bytes per 64 vocabulary rows: 256 MB
    L.piece_b = piece(((int64_t)1 << 28) / L.parts);  // 2 bytes per part: 512 MB
    L.split_dx = splits_for(up(L.kp, BT) / BT * (L.np / BT), L.piece_b / BK);
    L.split_dw = splits_for(up(L.kp, BT) / BT * (L.piece_b / BT), L.np / BK);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (size_t)up((int64_t)bytes, 256);
        return at;
    };
    L.rows = take((size_t)L.np * 4);
    L.place = take((size_t)L.np * 4);
    L.count = take(4);
    L.block_count = take((size_t)(L.np / LROWS + 1) * 4);
    L.xp = take((size_t)L.parts * L.np * L.kp * 2);
    L.wp = take((size_t)L.parts * vocab * L.kp * 2);
    if (backward) {
        L.dz = take((size_t)L.parts * L.np * L.piece_b * 2);
        L.dxp = take((size_t)L.split_dx * L.np * L.kp * 4);
        L.dwp = L.split_dw > 1 ? take((size_t)L.split_dw * L.piece_b * L.kp * 4) : 0;
    }
    const size_t both = o;
    // the forward's arrays share the backward's space: no call uses both
    o = L.dz ? L.dz : both;
    L.part = take((size_t)(L.piece_f / SLAB) * L.np * 8);
    L.target = take((size_t)L.np * 4);
    L.state = take((size_t)L.np * 8);
    L.block_sum = take((size_t)(L.np / JR + 1) * 8);
    L.total = o > both ? o : both;
    return L;
}

struct Packed {
    const bf16* w;
    int64_t ldw, pw;
};

template <class T>
hipError_t label_rows(const LabelLossArgs& a, const LossPlan& L, char* ws, bool forward, Packed& pk, hipStream_t s) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 3;
    int32_t *rows = (int32_t*)(ws + L.rows), *place = (int32_t*)(ws + L.place), *count = (int32_t*)(ws + L.count),
            *bc = (int32_t*)(ws + L.block_count);
    const int64_t want = (a.n + LROWS - 1) / LROWS;
    const unsigned blocks = (unsigned)(want < 1 ? 1 : want);
    if (blocks > 1) k_label_count<<<blocks, LT, 0, s>>>(a.n, a.vocab, a.labels, a.wide_labels, bc);
    k_label_rows<<<blocks, LT, 0, s>>>(a.n, a.vocab, a.labels, a.wide_labels, bc, rows, place, count,
                                       forward ? a.loss : nullptr, forward ? a.lse : nullptr);
    auto grid = [&](int64_t r) {
        const int64_t b = (r * (L.kp / 8) + 255) / 256;
        return (unsigned)(b < 1 ? 1 : b > 8192 ? 8192 : b);
    };
    k_pack<T, PARTS><<<grid(L.np), 256, 0, s>>>(a.n, a.dim, L.kp, (const T*)a.x, a.x_stride,
                                               (uintptr_t)a.x % 16 == 0 && a.x_stride % WIDE<T> == 0, rows, count,
                                               (bf16*)(ws + L.xp), L.np * L.kp);
    const bool w_wide = (uintptr_t)a.w % 16 == 0 && a.w_stride % WIDE<T> == 0;
    if (PARTS == 1 && w_wide && a.dim == L.kp && a.w_stride <= 1 << 20) {  // the products read w where it is
        pk.w = (const bf16*)a.w;
        pk.ldw = a.w_stride;
    } else {
        k_pack<T, PARTS><<<grid(a.vocab), 256, 0, s>>>(a.vocab, a.dim, L.kp, (const T*)a.w, a.w_stride, w_wide, nullptr,
                                                      nullptr, (bf16*)(ws + L.wp), (int64_t)a.vocab * L.kp);
        pk.w = (const bf16*)(ws + L.wp);
        pk.ldw = L.kp;
    }
    pk.pw = (int64_t)a.vocab * L.kp;
    return hipGetLastError();
}

unsigned tile_grid(int64_t m, int64_t n) {
    const int64_t t = up(m, BT) / BT * (up(n, BT) / BT);
    return (unsigned)(t < 8 ? 8 : up(t, 8));
}

template <class T>
Product product_base(const LabelLossArgs& a, const LossPlan& L, char* ws) {
    Product p{};
    p.splits = 1;
    p.count = (const int32_t*)(ws + L.count);
    p.rows = (const int32_t*)(ws + L.rows);
    p.labels = a.labels;
    p.wide_labels = a.wide_labels;
    p.np = (int)L.np;
    p.vocab = a.vocab;
    p.lse = a.lse;
    p.dmean = a.dmean;
    p.dloss = a.dloss;
    return p;
}

template <class T>
hipError_t loss_fwd(const LabelLossArgs& a, char* ws, hipStream_t s) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 3;
    const LossPlan L = loss_plan(a.n, a.dim, a.vocab, PARTS == 1, false);
    Packed pk{};
    hipError_t e = label_rows<T>(a, L, ws, true, pk, s);
    if (e != hipSuccess) return e;
    float2 *part = (float2*)(ws + L.part), *state = (float2*)(ws + L.state);
    double* bs = (double*)(ws + L.block_sum);
    for (int64_t v0 = 0; v0 < a.vocab; v0 += L.piece_f) {
        Product p = product_base<T>(a, L, ws);
        const int64_t mv = a.vocab - v0 < L.piece_f ? a.vocab - v0 : L.piece_f;
        p.a = pk.w + v0 * pk.ldw;
        p.lda = pk.ldw;
        p.pa = pk.pw;
        p.b = (const bf16*)(ws + L.xp);
        p.ldb = L.kp;
        p.pb = L.np * L.kp;
        p.m = (int)mv;
        p.k = L.kp;
        p.v0 = (int)v0;
        p.part = part;
        p.target = (float*)(ws + L.target);
        k_product<LSE, PARTS, T><<<tile_grid(mv, a.n), GT, 0, s>>>(p);
        // every tile writes its two slabs, so the last may lie beyond the vocabulary (an empty one)
        k_lse_join<<<(unsigned)(L.np / JR), JT, 0, s>>>((int)(up(mv, BT) / SLAB), (int)L.np, part, p.target, p.rows,
                                                       p.count, state, v0 == 0, v0 + L.piece_f < a.vocab, a.loss,
                                                       a.lse, bs);
    }
    k_loss_mean<<<1, LT, 0, s>>>(bs, (const int32_t*)(ws + L.count), a.mean, a.count);
    return hipGetLastError();
}

template <class T>
hipError_t loss_bwd(const LabelLossArgs& a, char* ws, hipStream_t s) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 3;
    const LossPlan L = loss_plan(a.n, a.dim, a.vocab, PARTS == 1, true);
    Packed pk{};
    hipError_t e = label_rows<T>(a, L, ws, false, pk, s);
    if (e != hipSuccess) return e;
    const bf16* xp = (const bf16*)(ws + L.xp);
    bf16* dz = (bf16*)(ws + L.dz);
    float *dxp = (float*)(ws + L.dxp), *dwp = (float*)(ws + L.dwp);
    for (int64_t v0 = 0; v0 < a.vocab; v0 += L.piece_b) {
        const int64_t mv = a.vocab - v0 < L.piece_b ? a.vocab - v0 : L.piece_b;
        Product p = product_base<T>(a, L, ws);
        p.a = pk.w + v0 * pk.ldw;
        p.lda = pk.ldw;
        p.pa = pk.pw;
        p.b = xp;
        p.ldb = L.kp;
        p.pb = L.np * L.kp;
        p.m = (int)mv;
        p.k = L.kp;
        p.v0 = (int)v0;
        p.dz = dz;
        p.lddz = L.piece_b;
        p.pdz = L.np * L.piece_b;
        k_product<DZ, PARTS, T><<<tile_grid(mv, a.n), GT, 0, s>>>(p);
        if (a.dx) {
            Product q = product_base<T>(a, L, ws);
            q.a = p.a;
            q.lda = pk.ldw;
            q.pa = pk.pw;
            q.b = dz;
            q.ldb = L.piece_b;
            q.pb = p.pdz;
            q.m = L.kp;
            q.k = (int)mv;
            q.splits = L.split_dx;
            q.acc = dxp;
            q.ldacc = L.kp;
            q.pacc = L.np * L.kp;
            q.add = v0 > 0;
            k_product<DX, PARTS, T><<<dim3(tile_grid(L.kp, a.n), q.splits), GT, 0, s>>>(q);
        }
        if (a.dw) {
            Product q = product_base<T>(a, L, ws);
            q.a = xp;
            q.lda = L.kp;
            q.pa = L.np * L.kp;
            q.b = dz;
            q.ldb = L.piece_b;
            q.pb = p.pdz;
            q.m = L.kp;
            q.n = (int)mv;
            q.splits = L.split_dw;
            T* out = (T*)a.dw + v0 * a.dw_stride;
            if (L.split_dw > 1) {
                q.acc = dwp;
                q.ldacc = L.kp;
                q.pacc = L.piece_b * L.kp;
            } else {
                q.out = out;
                q.ldout = a.dw_stride;
                q.out_dim = a.dim;
            }
            k_product<DW, PARTS, T><<<dim3(tile_grid(L.kp, mv), q.splits), GT, 0, s>>>(q);
            if (L.split_dw > 1)
                k_join_splits<T><<<(unsigned)(mv < 16384 ? (mv + 3) / 4 : 4096), 256, 0, s>>>(
                    mv, a.dim, L.split_dw, dwp, L.kp, q.pacc, nullptr, out, a.dw_stride);
        }
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dx && a.n > 0)
        k_join_splits<T><<<(unsigned)(a.n < 16384 ? (a.n + 3) / 4 : 4096), 256, 0, s>>>(
            a.n, a.dim, L.split_dx, dxp, L.kp, L.np * L.kp, (const int32_t*)(ws + L.place), (T*)a.dx, a.dx_stride);
    return hipGetLastError();
}

}  // namespace

size_t label_loss_workspace(int64_t n, int dim, int vocab, bool half, bool backward) {
    const size_t f = loss_plan(n, dim, vocab, half, false).total;
    const size_t b = backward ? loss_plan(n, dim, vocab, half, true).total : 0;
    return f > b ? f : b;
}

hipError_t launch_label_loss_fwd(const LabelLossArgs& a, char* ws, hipStream_t stream) {
    return a.half ? loss_fwd<bf16>(a, ws, stream) : loss_fwd<float>(a, ws, stream);
}

hipError_t launch_label_loss_bwd(const LabelLossArgs& a, char* ws, hipStream_t stream) {
    return a.half ? loss_bwd<bf16>(a, ws, stream) : loss_bwd<float>(a, ws, stream);
}

}  // namespace gs
