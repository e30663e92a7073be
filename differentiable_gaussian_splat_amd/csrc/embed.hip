// Lookup of feature rows by index, and its gradient by sorted indices.
//
//   out_i = s T[ids_i], zero where ids_i names no row
//   dT_v  = s sum_{i: ids_i = v} dout_i
//
// The lookup is bound by the rows it reads and writes. The gradient sorts the
// positions by their index (the radix sort of the tile binning; up to 8192 by
// ranking each among all), so that a row's contributions stand side by side:
// blocks then sum runs of equal indices over a fixed number of sorted positions
// each, write the rows whose run lies inside the block, and leave the first and
// last run, where it goes on in a neighbouring block, as a partial sum. A last
// launch adds the partial sums of each such row in block order. A row that half
// of the positions name is thus spread over as many blocks as any other half,
// and the sums are the same bit for bit from run to run: no atomic takes part in
// them (the sort counts digits with integer ones, which come out the same).
// All sums are float32, rounded once. The vocabulary loss sums weighed rows by
// label in the same way (WeighedRows).
//
// A million rows of 64 float32 from a table of 16384, with the gradient: 186 us,
// of it the lookup 61 (256 MB written, 4.2 TB/s of the 4.8 that a copy reaches),
// the runs 78 (256 MB gathered row by row, 3.3 TB/s), the sort 36. 65536 rows of
// 512 bfloat16 with two fifths of them one word: 84 us, the sort 18 of it, five
// short launches bound by their latency.
#include "elem.hpp"
#include "launch.hpp"

namespace gs {

namespace {

constexpr int EB = 256;         // threads per block
constexpr int RUN_USUAL = 16;  // sorted positions a row group sums, all loaded at once; twice that ...
// ... from this many positions on: fewer partial sums to join (us, 16 and 32 positions: 1M x 64 float32 189 and 186,
// 400000 x 64 94.5 and 93.5, 250000 x 64 62.7 and 61, 100000 x 64 37.8 and 38.9)
constexpr int64_t RUN_LONG = 400000;
// Where there are few blocks, a group's sums one after the other take the time, so it has fewer, up to RUN_SHORT
// positions (3487 x 2 bf16 10.5 us against 16, 300 x 64 5.3 and a join of 2.7 against 6.8, 8192 x 64 float32 4.9
// against 5.7; 32768 x 500 would take 17 and a join of 11 against 16 and 4.6).
constexpr int RUN_FEW = 4;
constexpr int64_t RUN_SHORT = 8192;
constexpr int JOIN_T = 1024;
// Positions up to which one launch makes the gradient (a multiple of 64): 33 x 32 from 500 rows 3.5 us, 30 us by
// the sort; a row that all positions name is summed by one lane group, 8 at a time, hence not for more.
constexpr int FEW = 256;

// Positions up to which each is ranked among all (n^2 comparisons) in the launch that clears the table, instead of
// three to five launches more for the sort: 1000 x 64 bf16 4.8 us against 13.2 by the sort and its clear, 8192 x 64
// from 5000 rows 19 against 18 and three launches fewer, 16384 x 64 67 against 10 to 25.
constexpr int RANK_MOST = 8192;
constexpr int RANK_P = 16;  // positions ranked per block

enum EmbedPass { LOOKUP, FEW_SUMS, RUN_SUMS };

// Threads of a block that sums runs with lpr lanes per row: 32 lane groups (64 of one lane, 4 of a wave).
constexpr int run_threads(int lpr) { return lpr <= 2 ? 64 : lpr == 4 ? 128 : EB; }

// LPR lanes per output row, 16 bytes each per step over the row.
template <class T, int LPR, bool FULL>
__global__ __launch_bounds__(EB) void k_embed(int64_t n, int dim, int vocab, const T* __restrict__ table, int64_t ts,
                                              const void* __restrict__ ids, bool wide, float scale,
                                              T* __restrict__ out, int64_t os) {
    constexpr int U = 4;  // rows in flight per lane group
    constexpr int G = EB / LPR, VEC = WIDE<T>;
    const int l = threadIdx.x % LPR;
    const int64_t r0 = (int64_t)blockIdx.x * G * U + threadIdx.x / LPR;
    int row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + u * G;
        row[u] = r < n ? row_index(ids, wide, r, vocab) : -1;
    }
    for (int c = l * VEC; c < dim; c += LPR * VEC) {
        wide_t<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            raw[u] = (T)0.f;
            if (row[u] >= 0)
                raw[u] = load_row<FULL>(table + row[u] * ts + c, dim - c, (vocab - 1 - row[u]) * ts + dim - c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * G;
            float v[VEC];
            widen<true, T>(raw[u], dim - c, v);  // what is behind the row is not stored
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] = row[u] >= 0 ? v[k] * scale : 0.f;
            if (r < n) store_row<FULL>(out + r * os + c, dim - c, v);
        }
    }
}

// Block `block` of `blocks` that clear the table.
template <class T>
__device__ void zero_share(int block, int blocks, int rows, int dim, int lanes, T* __restrict__ p, int64_t stride) {
    const float z[WIDE<T>] = {};
    const int l = threadIdx.x % lanes, per = EB / lanes;
    for (int64_t r = (int64_t)block * per + threadIdx.x / lanes; r < rows; r += (int64_t)blocks * per)
        for (int c = l * WIDE<T>; c < dim; c += lanes * WIDE<T>) store_row<false>(p + r * stride + c, dim - c, z);
}

// Also clears the sort's digit totals.
template <class T>
__global__ __launch_bounds__(EB) void k_zero_rows(int rows, int dim, int lanes, T* __restrict__ p, int64_t stride,
                                                  uint32_t* __restrict__ totals, int n_totals) {
    for (int k = blockIdx.x * EB + threadIdx.x; k < n_totals; k += gridDim.x * EB) totals[k] = 0u;
    zero_share(blockIdx.x, gridDim.x, rows, dim, lanes, p, stride);
}

// The first blocks rank RANK_P positions each and write them, sorted by index
// and then by position as the sort has them; the others clear the table. A
// position's rank is the count of smaller indices, and of equal ones before it:
// 16 threads a position, each over every sixteenth four indices.
template <class T>
__global__ __launch_bounds__(EB) void k_rank_rows(int n, const void* __restrict__ ids, bool wide,
                                                  uint32_t* __restrict__ keys, uint32_t* __restrict__ pos,
                                                  int rank_blocks, int rows, int dim, int lanes, T* __restrict__ p,
                                                  int64_t stride) {
    if ((int)blockIdx.x >= rank_blocks) {
        zero_share((int)blockIdx.x - rank_blocks, (int)gridDim.x - rank_blocks, rows, dim, lanes, p, stride);
        return;
    }
    constexpr int S = EB / RANK_P;
    static_assert(RANK_MOST % (4 * S) == 0 && S * RANK_P == EB && 64 % RANK_P == 0, "whole steps");
    __shared__ uint4 s_key[RANK_MOST / 4];
    __shared__ int s_count[EB / 64][RANK_P];
    uint32_t* s = reinterpret_cast<uint32_t*>(s_key);
    const int steps = (n + 4 * S - 1) / (4 * S);
#pragma unroll 4
    for (int j = threadIdx.x; j < steps * 4 * S; j += EB) {
        const int v = j < n ? row_index(ids, wide, j, rows) : 0;
        s[j] = j >= n ? ~0u : (uint32_t)(v < 0 ? rows - 1 : v);  // past the positions: larger than any index
    }
    __syncthreads();
    const int at = threadIdx.x % RANK_P, i = blockIdx.x * RANK_P + at;
    const uint32_t key = s[i < n ? i : 0];
    int count = 0;
    for (int q = threadIdx.x / RANK_P; q < steps * S; q += S) {
        const uint4 k = s_key[q];
        const uint32_t below = key + (q < i / 4 ? 1u : 0u);
        count += (k.x < below) + (k.y < below) + (k.z < below) + (k.w < below);
    }
#pragma unroll
    for (int off = RANK_P; off < 64; off <<= 1) count += __shfl_xor(count, off);
    if ((threadIdx.x & 63) < RANK_P) s_count[threadIdx.x / 64][at] = count;
    __syncthreads();
    if (threadIdx.x < RANK_P && i < n) {
        count = 0;
#pragma unroll
        for (int w = 0; w < EB / 64; ++w) count += s_count[w][at];
        for (int j = i & ~3; j < i; ++j) count += s[j] == key;  // equal ones of its own four
        keys[count] = key;
        pos[count] = (uint32_t)i | (row_index(ids, wide, i, rows) < 0 ? INDEX_NONE : 0u);
    }
}

// The gradient of few positions in one launch: a wave takes 64 / LPR rows of
// the table in turn, and looks through the indices (in LDS) for each.
template <class T, int LPR, bool FULL>
__global__ __launch_bounds__(EB) void k_embed_few(int n, int dim, int vocab, const void* __restrict__ ids, bool wide,
                                                  float scale, const T* __restrict__ dout, int64_t ds,
                                                  T* __restrict__ dtable, int64_t ts) {
    constexpr int VEC = WIDE<T>, U = 8;
    __shared__ int s_id[FEW];
    for (int i = threadIdx.x; i < FEW; i += EB) s_id[i] = i < n ? row_index(ids, wide, i, vocab) : -1;
    __syncthreads();
    const int lane = threadIdx.x & 63, sub = lane / LPR;
    const int wave = (int)(blockIdx.x * (EB / 64)) + (int)(threadIdx.x >> 6), waves = (int)gridDim.x * (EB / 64);
    for (int64_t v0 = (int64_t)wave * (64 / LPR); v0 < vocab; v0 += (int64_t)waves * (64 / LPR)) {
        const int row = (int)v0 + sub;  // of this lane group
        const int c = (blockIdx.y * LPR + lane % LPR) * VEC;
        {
            float acc[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
            for (int i0 = 0; i0 < n; i0 += 64) {
                uint64_t mine = 0;
                const int id = s_id[i0 + lane];
                if (!__any(id >= (int)v0 && id < (int)v0 + 64 / LPR)) continue;
#pragma unroll
                for (int q = 0; q < 64 / LPR; ++q) {
                    const uint64_t m = __ballot(id == (int)v0 + q);
                    mine = q == sub ? m : mine;
                }
                while (mine) {
                    wide_t<T> raw[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        raw[u] = (T)0.f;
                        if (mine) {
                            const int i = i0 + __ffsll((unsigned long long)mine) - 1;
                            mine &= mine - 1;
                            if (c < dim)
                                raw[u] = load_row<FULL>(dout + (int64_t)i * ds + c, dim - c,
                                                        (n - 1 - i) * ds + dim - c);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float t[VEC];
                        widen<true, T>(raw[u], dim - c, t);
#pragma unroll
                        for (int k = 0; k < VEC; ++k) acc[k] += t[k];
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) acc[k] *= scale;
            if (row < vocab && c < dim) store_row<FULL>(dtable + (int64_t)row * ts + c, dim - c, acc);
        }
    }
}

// The first `left` of four columns.
template <class T>
__device__ __forceinline__ void store_four(T* p, int left, float4 v) {
    typedef T vec __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    if (left >= 4) {
        vec t;
        t[0] = (T)v.x, t[1] = (T)v.y, t[2] = (T)v.z, t[3] = (T)v.w;
        *reinterpret_cast<vec*>(p) = t;
    } else {
        p[0] = (T)v.x;
        if (left > 1) p[1] = (T)v.y;
        if (left > 2) p[2] = (T)v.z;
    }
}

// Sums of equal-key runs. Block b (of column chunk blockIdx.y) takes the sorted
// positions [b BT, (b + 1) BT), group g of LPR lanes RUN_TOKENS of them. part
// holds two rows of dim per block: the block's first run where it began in an
// earlier block, and its last run where it goes on in the next (and began in
// this one). tail_key[b]: that last run's key, or vocab; end_block[key]: the
// block in which a run that came from an earlier block ends. WEIGHED: the sums
// of w instead; a run's row of them is numbered by one of its positions.
template <class T, int LPR, bool FULL, int RUN_TOKENS, bool WEIGHED>
__global__ __launch_bounds__(run_threads(LPR)) void k_embed_runs(
    int n, int dim, int vocab, const uint32_t* __restrict__ keys, const uint32_t* __restrict__ pos,
    const T* __restrict__ dout, int64_t ds, float scale, T* __restrict__ dtable, int64_t ts,
    float* __restrict__ part, uint32_t* __restrict__ tail_key, uint32_t* __restrict__ end_block, WeighedRows w) {
    constexpr int NT = run_threads(LPR);
    constexpr int G = NT / LPR;
    constexpr int BT = G * RUN_TOKENS;
    constexpr int VEC = WIDE<T>, CW = LPR * VEC;
    constexpr int U = RUN_TOKENS < RUN_USUAL ? RUN_TOKENS : RUN_USUAL;
    __shared__ uint32_t s_tok[BT], s_pos[BT];
    __shared__ float s_weight[WEIGHED ? BT : 1];
    __shared__ uint32_t s_key[2 * G + 4];  // per group: its first run's key and its last run's, if one, the same
    __shared__ alignas(16) float s_sum[2 * G][CW];
    const uint32_t none = (uint32_t)vocab;
    const int g = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int c0 = blockIdx.y * CW, c = c0 + l * VEC;
    const int b0 = blockIdx.x * BT, b1 = min(n, b0 + BT);
    if (WEIGHED && (keys[b1 - 1] < w.first || keys[b0] >= w.last)) {
        if (threadIdx.x == 0 && blockIdx.y == 0) tail_key[blockIdx.x] = none;
        return;
    }
    auto taken = [&](uint32_t key) { return !WEIGHED || (key >= w.first && key < w.last); };
    for (int i = threadIdx.x; i < BT; i += NT) {
        const uint32_t key = b0 + i < b1 ? keys[b0 + i] : none;
        uint32_t at = b0 + i < b1 ? pos[b0 + i] : INDEX_NONE;
        if constexpr (WEIGHED) {
            at = !(at & INDEX_NONE) && taken(key) ? (uint32_t)w.place[at] : INDEX_NONE;
            s_weight[i] = at & INDEX_NONE ? 0.f : w.weight[at];
        }
        s_tok[i] = key;
        s_pos[i] = at;
    }
    const uint32_t before = b0 > 0 ? keys[b0 - 1] : none;
    const uint32_t after = b1 < n ? keys[b1] : none;
    __syncthreads();
    const int p0 = g * RUN_TOKENS;

    float acc[VEC];
    const uint32_t first = s_tok[p0];
    uint32_t cur = first;
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
    bool lead = true;  // still in the group's first run
#pragma unroll 1
    for (int p = p0; p < p0 + RUN_TOKENS; p += U) {
        if (s_tok[p] == none) break;  // past the positions
        uint32_t kk[U], at[U];
        wide_t<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            kk[u] = s_tok[p + u];
            at[u] = s_pos[p + u];  // past the positions: INDEX_NONE
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            raw[u] = (T)0.f;
            if (c < dim && !(at[u] & INDEX_NONE))
                raw[u] = load_row<FULL>(dout + at[u] * ds + c, dim - c, (n - 1 - (int)at[u]) * ds + dim - c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kk[u] != none && kk[u] != cur) {
                if (lead) {
#pragma unroll
                    for (int k = 0; k < VEC; ++k) s_sum[2 * g][l * VEC + k] = acc[k];
                    lead = false;
                } else if (c < dim && taken(cur)) {  // a run between two others of the group is whole
                    if constexpr (WEIGHED) {
                        const int64_t to = b0 + p + u - 1;  // its last position
                        if (c == 0) w.slot[cur] = (int32_t)to + 1;
#pragma unroll
                        for (int k = 0; k < VEC; k += 4)
                            store_four(w.sums + to * w.ld + c + k, 4,
                                       make_float4(acc[k], acc[k + 1], acc[k + 2], acc[k + 3]));
                    } else {
#pragma unroll
                        for (int k = 0; k < VEC; ++k) acc[k] *= scale;
                        store_row<FULL>(dtable + (int64_t)cur * ts + c, dim - c, acc);
                    }
                }
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
                cur = kk[u];
            }
            float v[VEC];
            widen<true, T>(raw[u], dim - c, v);  // sums of what is behind the row are not stored
#pragma unroll
            for (int k = 0; k < VEC; ++k) acc[k] = WEIGHED ? fmaf(s_weight[p + u], v[k], acc[k]) : acc[k] + v[k];
        }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        s_sum[2 * g + 1][l * VEC + k] = lead ? 0.f : acc[k];
        if (lead) s_sum[2 * g][l * VEC + k] = acc[k];
    }
    if (l == 0) {
        s_key[2 * g] = first;
        s_key[2 * g + 1] = cur;
    }
    if (threadIdx.x < 4) s_key[2 * G + threadIdx.x] = none;
    __syncthreads();

    // one thread per run and four columns: the sums of the groups that hold it, in order
    for (int i = threadIdx.x; i < 2 * G * (CW / 4); i += NT) {
        const int e = i / (CW / 4), j = i % (CW / 4) * 4;
        const uint32_t run = s_key[e];
        if (run == none || (e > 0 && s_key[e - 1] == run)) continue;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        int f = e;
        for (bool same = true; same; f += 4) {
            uint32_t key[4];
            float4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                key[u] = s_key[f + u];
                x[u] = *reinterpret_cast<const float4*>(&s_sum[min(f + u, 2 * G - 1)][j]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                same = same && key[u] == run;
                sum.x += same ? x[u].x : 0.f;
                sum.y += same ? x[u].y : 0.f;
                sum.z += same ? x[u].z : 0.f;
                sum.w += same ? x[u].w : 0.f;
            }
        }
        // the block's last run is its last position's
        const bool last = run == s_tok[b1 - 1 - b0], open = e == 0 && run == before && taken(run),
                   goes_on = last && run == after && taken(run);
        const int left = dim - (c0 + j);
        if (j == 0 && blockIdx.y == 0) {
            if (open && !goes_on) end_block[run] = blockIdx.x;
            if (last) tail_key[blockIdx.x] = goes_on && !open ? run : none;
        }
        if (left <= 0 || !taken(run)) continue;
        // of the run's positions: its group's first, or last
        const int64_t to = b0 + (e % 2 == 0 ? e / 2 * RUN_TOKENS : min(e / 2 * RUN_TOKENS + RUN_TOKENS, b1 - b0) - 1);
        if (WEIGHED && !open && !goes_on && c0 + j == 0) w.slot[run] = (int32_t)to + 1;
        if (open || goes_on)
            store_four(part + ((size_t)blockIdx.x * 2 + (open ? 0 : 1)) * dim + c0 + j, left, sum);
        else if constexpr (WEIGHED)
            store_four(w.sums + to * w.ld + c0 + j, left, sum);
        else
            store_four(dtable + (int64_t)run * ts + c0 + j, left,
                       make_float4(sum.x * scale, sum.y * scale, sum.z * scale, sum.w * scale));
    }
}

// Rows whose run crosses blocks: the last run of block b, then the first runs
// of the blocks after it up to the one where it ends, a contiguous share per
// row group, the groups joined in order.
template <class T, int LPR, bool FULL, bool WEIGHED>
__global__ __launch_bounds__(JOIN_T) void k_embed_join(int first, int dim, int vocab,
                                                       const uint32_t* __restrict__ tail_key,
                                                       const uint32_t* __restrict__ end_block,
                                                       const float* __restrict__ part, float scale,
                                                       T* __restrict__ dtable, int64_t ts, WeighedRows w) {
    constexpr int VEC = WIDE<T>, CW = LPR * VEC;
    constexpr int G = JOIN_T / LPR < 64 ? JOIN_T / LPR : 64;  // groups that take part
    __shared__ float s_sum[G][CW];
    const int b = first + (int)blockIdx.x;
    const uint32_t key = tail_key[b];
    if (key == (uint32_t)vocab) return;
    const int g = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int c = blockIdx.y * CW + l * VEC;
    const int cnt = (int)end_block[key] - b + 1;
    const int per = (cnt + G - 1) / G;
    const int j0 = g * per, j1 = g < G ? min(cnt, j0 + per) : 0;
    float acc[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
    if (c < dim) {
#pragma unroll 4
        for (int j = j0; j < j1; ++j) {
            const float* q = part + ((size_t)(b + j) * 2 + (j == 0 ? 1 : 0)) * dim + c;
#pragma unroll
            for (int k = 0; k < VEC; k += 4) {
                const wide_t<float> t = load_row<FULL>(q + k, dim - c - k, dim - c - k);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[k + i] += t[i];
            }
        }
    }
    if (g < G)
#pragma unroll
        for (int k = 0; k < VEC; ++k) s_sum[g][l * VEC + k] = acc[k];
    __syncthreads();
    for (int h = G / 2; h > 0; h >>= 1) {
        if (g < h)
#pragma unroll
            for (int k = 0; k < VEC; ++k) s_sum[g][l * VEC + k] += s_sum[g + h][l * VEC + k];
        __syncthreads();
    }
    if (g == 0 && c < dim) {
        if constexpr (WEIGHED) {
            const int64_t to = (int64_t)(b + 1) * w.per_block - 1;  // the run's last position in block b
            if (c == 0) w.slot[key] = (int32_t)to + 1;
#pragma unroll
            for (int k = 0; k < VEC; ++k) w.sums[to * w.ld + c + k] = s_sum[0][l * VEC + k];
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) acc[k] = s_sum[0][l * VEC + k] * scale;
            store_row<FULL>(dtable + (int64_t)key * ts + c, dim - c, acc);
        }
    }
}

struct EmbedArgs {
    int64_t n;
    int dim, vocab;
    bool wide;
    const void *ids, *src;  // src: the table (forward) or dout (backward)
    void* dst;              // out, or dtable
    int64_t ss, ds;
    float scale;
    const uint32_t *keys, *pos;
    float* part;
    uint32_t *tail_key, *end_block;
    WeighedRows weighed;
};

template <class T, int LPR, bool FULL, int RUN_TOKENS, bool WEIGHED = false>
hipError_t embed_sums(const EmbedArgs& a, hipStream_t s) {
    constexpr int BT = run_threads(LPR) / LPR * RUN_TOKENS;
    const int nb = (int)((a.n + BT - 1) / BT);
    const dim3 grid(nb, (a.dim + LPR * WIDE<T> - 1) / (LPR * WIDE<T>));
    WeighedRows w = a.weighed;
    w.per_block = BT;
    k_embed_runs<T, LPR, FULL, RUN_TOKENS, WEIGHED><<<grid, run_threads(LPR), 0, s>>>(
        (int)a.n, a.dim, a.vocab, a.keys, a.pos, (const T*)a.src, a.ss, a.scale, (T*)a.dst, a.ds, a.part, a.tail_key,
        a.end_block, w);
    for (int64_t b0 = 0; nb > 1 && b0 < nb; b0 += MOST_BLOCKS)
        k_embed_join<T, LPR, FULL, WEIGHED><<<dim3((unsigned)(nb - b0 < MOST_BLOCKS ? nb - b0 : MOST_BLOCKS), grid.y),
                                              JOIN_T, 0, s>>>((int)b0, a.dim, a.vocab, a.tail_key, a.end_block, a.part,
                                                              a.scale, (T*)a.dst, a.ds, w);
    return hipGetLastError();
}

template <class T, int LPR, bool FULL, bool WEIGHED = false>
hipError_t embed_runs(const EmbedArgs& a, hipStream_t s) {
    return a.n <= RUN_SHORT  ? embed_sums<T, LPR, FULL, RUN_FEW, WEIGHED>(a, s)
           : a.n < RUN_LONG ? embed_sums<T, LPR, FULL, RUN_USUAL, WEIGHED>(a, s)
                            : embed_sums<T, LPR, FULL, 2 * RUN_USUAL, WEIGHED>(a, s);
}

template <class T, int LPR, bool FULL>
hipError_t embed_rows(const EmbedArgs& a, EmbedPass pass, hipStream_t s) {
    if (pass == LOOKUP) {
        constexpr int64_t PER = EB / LPR * 4, MOST = PER * MOST_BLOCKS;  // rows of a block and of a launch
        for (int64_t r = 0; r < a.n; r += MOST) {
            const int64_t rows = a.n - r < MOST ? a.n - r : MOST;
            k_embed<T, LPR, FULL><<<(unsigned)((rows + PER - 1) / PER), EB, 0, s>>>(
                rows, a.dim, a.vocab, (const T*)a.src, a.ss, (const char*)a.ids + r * (a.wide ? 8 : 4), a.wide, a.scale,
                (T*)a.dst + r * a.ds, a.ds);
        }
        return hipGetLastError();
    }
    if (pass == FEW_SUMS) {
        const int64_t want = (a.vocab + EB / LPR - 1) / (EB / LPR);
        const dim3 grid((unsigned)(want < 2048 ? want : 2048), (a.dim + LPR * WIDE<T> - 1) / (LPR * WIDE<T>));
        k_embed_few<T, LPR, FULL><<<grid, EB, 0, s>>>(
            (int)a.n, a.dim, a.vocab, a.ids, a.wide, a.scale, (const T*)a.src, a.ss, (T*)a.dst, a.ds);
        return hipGetLastError();
    }
    return embed_runs<T, LPR, FULL>(a, s);
}

// The fewest lanes that hold a row with one 16-byte access each, up to a wave.
template <class T, bool FULL>
hipError_t embed_pick(const EmbedArgs& a, EmbedPass pass, hipStream_t s) {
    const int v = (a.dim + WIDE<T> - 1) / WIDE<T>;
    if (v <= 1) return embed_rows<T, 1, FULL>(a, pass, s);
    if (v <= 2) return embed_rows<T, 2, FULL>(a, pass, s);
    if (v <= 4) return embed_rows<T, 4, FULL>(a, pass, s);
    if (v <= 8) return embed_rows<T, 8, FULL>(a, pass, s);
    if (v <= 16) return embed_rows<T, 16, FULL>(a, pass, s);
    if (v <= 32) return embed_rows<T, 32, FULL>(a, pass, s);
    return embed_rows<T, 64, FULL>(a, pass, s);
}

template <class T>
hipError_t embed_run(const EmbedArgs& a, EmbedPass pass, hipStream_t s) {
    return a.dim % WIDE<T> == 0 ? embed_pick<T, true>(a, pass, s) : embed_pick<T, false>(a, pass, s);
}

// Clears the table and, of few positions, leaves them sorted in keys and pos; of more, readies the sort's totals.
template <class T>
hipError_t zero_rows(const EmbedArgs& a, uint32_t* keys, uint32_t* pos, char* totals, hipStream_t s) {
    int lanes = 1;
    while (lanes < 64 && lanes * WIDE<T> < a.dim) lanes *= 2;
    const int64_t want = ((int64_t)a.vocab * lanes + EB - 1) / EB;
    const int blocks = (int)(want < 4096 ? want : 4096);
    if (a.n <= RANK_MOST) {
        const int rank_blocks = (int)((a.n + RANK_P - 1) / RANK_P);
        k_rank_rows<T><<<rank_blocks + blocks, EB, 0, s>>>((int)a.n, a.ids, a.wide, keys, pos, rank_blocks, a.vocab,
                                                          a.dim, lanes, (T*)a.dst, a.ds);
    } else {
        k_zero_rows<T><<<blocks, EB, 0, s>>>(a.vocab, a.dim, lanes, (T*)a.dst, a.ds, (uint32_t*)totals,
                                            RADIX_TOTAL_WORDS);
    }
    return hipGetLastError();
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// The fewest positions per block (64 lanes per row) bound the block count.
int64_t max_blocks(int64_t n) {
    const int64_t per = EB / 64 * (n <= RUN_SHORT ? RUN_FEW : RUN_USUAL);
    return (n + per - 1) / per;
}

}  // namespace

EmbedLayout embed_bwd_layout(int64_t n, int dim, int vocab) {
    EmbedLayout L{};
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += up256(bytes);
        return at;
    };
    for (int k = 0; k < 2; ++k) {
        L.keys[k] = take((size_t)n * 4);
        L.pos[k] = take((size_t)n * 4);
    }
    L.sort = take(radix_sort_scratch(n));
    L.part = take((size_t)max_blocks(n) * 2 * dim * 4);
    L.tail_key = take((size_t)max_blocks(n) * 4);
    L.end_block = take((size_t)vocab * 4);
    L.total = o;
    return L;
}

hipError_t launch_embed_fwd(int64_t n, int dim, int vocab, bool half, const void* table, int64_t table_stride,
                            const void* ids, bool wide_ids, float scale, void* out, int64_t out_stride,
                            hipStream_t stream) {
    EmbedArgs a{};
    a.n = n;
    a.dim = dim;
    a.vocab = vocab;
    a.wide = wide_ids;
    a.ids = ids;
    a.src = table;
    a.ss = table_stride;
    a.dst = out;
    a.ds = out_stride;
    a.scale = scale;
    return half ? embed_run<bf16>(a, LOOKUP, stream) : embed_run<float>(a, LOOKUP, stream);
}

hipError_t launch_embed_bwd(int64_t n, int dim, int vocab, bool half, const void* ids, bool wide_ids, float scale,
                            const void* dout, int64_t dout_stride, void* dtable, int64_t dtable_stride, char* ws,
                            hipStream_t stream) {
    EmbedArgs a{};
    a.n = n;
    a.dim = dim;
    a.vocab = vocab;
    a.wide = wide_ids;
    a.ids = ids;
    a.src = dout;
    a.ss = dout_stride;
    a.dst = dtable;
    a.ds = dtable_stride;
    a.scale = scale;
    if (n <= FEW) return half ? embed_run<bf16>(a, FEW_SUMS, stream) : embed_run<float>(a, FEW_SUMS, stream);
    const EmbedLayout L = embed_bwd_layout(n, dim, vocab);
    uint32_t* keys[2] = {(uint32_t*)(ws + L.keys[0]), (uint32_t*)(ws + L.keys[1])};
    uint32_t* pos[2] = {(uint32_t*)(ws + L.pos[0]), (uint32_t*)(ws + L.pos[1])};
    hipError_t e = half ? zero_rows<bf16>(a, keys[0], pos[0], ws + L.sort, stream)
                        : zero_rows<float>(a, keys[0], pos[0], ws + L.sort, stream);
    int at = 0;
    if (e == hipSuccess && n > RANK_MOST)
        e = launch_index_sort((int)n, vocab, ids, wide_ids, keys, pos, ws + L.sort, &at, stream);
    if (e != hipSuccess) return e;
    a.keys = keys[at];
    a.pos = pos[at];
    a.part = (float*)(ws + L.part);
    a.tail_key = (uint32_t*)(ws + L.tail_key);
    a.end_block = (uint32_t*)(ws + L.end_block);
    return half ? embed_run<bf16>(a, RUN_SUMS, stream) : embed_run<float>(a, RUN_SUMS, stream);
}

hipError_t launch_rows_by_index(int64_t n, int rows, const void* ids, bool wide_ids, int ld, int32_t* slot, char* ws,
                                int* sorted_at, hipStream_t stream) {
    const EmbedLayout L = embed_bwd_layout(n, ld, rows);
    uint32_t* keys[2] = {(uint32_t*)(ws + L.keys[0]), (uint32_t*)(ws + L.keys[1])};
    uint32_t* pos[2] = {(uint32_t*)(ws + L.pos[0]), (uint32_t*)(ws + L.pos[1])};
    EmbedArgs a{};
    a.n = n;
    a.dim = 1;  // of the table that is cleared: slot
    a.vocab = rows;
    a.wide = wide_ids;
    a.ids = ids;
    a.dst = slot;
    a.ds = 1;
    *sorted_at = 0;
    const hipError_t e = zero_rows<float>(a, keys[0], pos[0], ws + L.sort, stream);
    if (e != hipSuccess || n <= RANK_MOST) return e;
    return launch_index_sort((int)n, rows, ids, wide_ids, keys, pos, ws + L.sort, sorted_at, stream);
}

hipError_t launch_weighed_rows(int64_t n, int rows, int sorted_at, const WeighedRows& w, char* ws,
                               hipStream_t stream) {
    const EmbedLayout L = embed_bwd_layout(n, (int)w.ld, rows);
    EmbedArgs a{};
    a.n = n;
    a.dim = (int)w.ld;
    a.vocab = rows;
    a.src = w.src;
    a.ss = w.ld;
    a.keys = (const uint32_t*)(ws + L.keys[sorted_at]);
    a.pos = (const uint32_t*)(ws + L.pos[sorted_at]);
    a.part = (float*)(ws + L.part);
    a.tail_key = (uint32_t*)(ws + L.tail_key);
    a.end_block = (uint32_t*)(ws + L.end_block);
    a.weighed = w;
    if (w.ld <= 32) return embed_runs<bf16, 4, true, true>(a, stream);
    if (w.ld <= 64) return embed_runs<bf16, 8, true, true>(a, stream);
    if (w.ld <= 128) return embed_runs<bf16, 16, true, true>(a, stream);
    if (w.ld <= 256) return embed_runs<bf16, 32, true, true>(a, stream);
    return embed_runs<bf16, 64, true, true>(a, stream);
}

}  // namespace gs
