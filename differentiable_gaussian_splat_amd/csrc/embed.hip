// Lookup of feature rows by index, and its gradient by sorted indices.
//
//   out_i = s T[ids_i], zero where ids_i names no row
//   dT_v  = s sum_{i: ids_i = v} dout_i
//
// The lookup is bound by the rows it reads and writes. The gradient sorts the
// positions by their index (the radix sort of the tile binning), so that a
// row's contributions stand side by side: blocks then sum runs of equal
// indices over a fixed number of sorted positions each, write the rows whose
// run lies inside the block, and leave the first and last run, where it goes
// on in a neighbouring block, as a partial sum. A last launch adds the partial
// sums of each such row in block order. A row that half of the positions name
// is thus spread over as many blocks as any other half, there are no atomics,
// and the sums are the same bit for bit from run to run. All sums are float32,
// rounded once.
#include "elem.hpp"
#include "launch.hpp"

namespace gs {

namespace {

constexpr int EB = 256;         // threads per block
constexpr int RUN_TOKENS = 32;  // sorted positions a row group sums
constexpr int JOIN_T = 1024;

// LPR lanes per output row, each VEC elements per step over the row.
template <class T, int VEC, int LPR>
__global__ __launch_bounds__(EB) void k_embed(int64_t n, int dim, int vocab, const T* __restrict__ table, int64_t ts,
                                              const void* __restrict__ ids, bool wide, float scale,
                                              T* __restrict__ out, int64_t os) {
    constexpr int U = 4;  // rows in flight per lane group
    constexpr int G = EB / LPR;
    const int l = threadIdx.x % LPR;
    const int64_t r0 = (int64_t)blockIdx.x * G * U + threadIdx.x / LPR;
    int row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + u * G;
        row[u] = r < n ? row_index(ids, wide, r, vocab) : -1;
    }
    for (int c = l * VEC; c < dim; c += LPR * VEC) {
        float v[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[u][k] = 0.f;
            if (row[u] >= 0) {
                load_row<VEC>(table + row[u] * ts + c, v[u]);
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[u][k] *= scale;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * G;
            if (r < n) store_row<VEC>(out + r * os + c, v[u]);
        }
    }
}

// Sort keys (the index, or vocab where it names no row) and positions; the sort's digit totals cleared.
__global__ __launch_bounds__(EB) void k_embed_keys(int n, int vocab, const void* __restrict__ ids, bool wide,
                                                   uint32_t* __restrict__ keys, uint32_t* __restrict__ pos,
                                                   uint32_t* __restrict__ totals, int n_totals) {
    const int i = blockIdx.x * EB + threadIdx.x;
    for (int k = i; k < n_totals; k += gridDim.x * EB) totals[k] = 0u;
    if (i < n) {
        const int r = row_index(ids, wide, i, vocab);
        keys[i] = r < 0 ? (uint32_t)vocab : (uint32_t)r;
        pos[i] = (uint32_t)i;
    }
}

template <class T, int VEC>
__global__ __launch_bounds__(EB) void k_zero_rows(int64_t rows, int dim, T* __restrict__ p, int64_t stride) {
    const int per = dim / VEC;
    const int64_t total = rows * per;
    const float z[VEC] = {};
    for (int64_t i = (int64_t)blockIdx.x * EB + threadIdx.x; i < total; i += (int64_t)gridDim.x * EB) {
        const int64_t r = i / per;
        store_row<VEC>(p + r * stride + (i - r * per) * VEC, z);
    }
}

// Sums of equal-key runs. Block b (of column chunk blockIdx.y) takes the sorted
// positions [b BT, (b + 1) BT), group g of LPR lanes RUN_TOKENS of them. part
// holds two rows of dim per block: the block's first run where it began in an
// earlier block, and its last run where it goes on in the next (and began in
// this one). tail_key[b]: that last run's key, or vocab; end_block[key]: the
// block in which a run that came from an earlier block ends.
template <class T, int VEC, int LPR>
__global__ __launch_bounds__(EB) void k_embed_runs(int n, int dim, int vocab, const uint32_t* __restrict__ keys,
                                                   const uint32_t* __restrict__ pos, const T* __restrict__ dout,
                                                   int64_t ds, float scale, T* __restrict__ dtable, int64_t ts,
                                                   float* __restrict__ part, uint32_t* __restrict__ tail_key,
                                                   uint32_t* __restrict__ end_block) {
    constexpr int G = EB / LPR;
    constexpr int BT = G * RUN_TOKENS;
    constexpr int CW = LPR * VEC;
    constexpr int U = 8;
    __shared__ uint32_t s_key[2 * G];  // per group: its first run's key and, if another, its last run's
    __shared__ float s_sum[2 * G][CW];
    const uint32_t none = (uint32_t)vocab;
    const int g = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int c0 = blockIdx.y * CW, c = c0 + l * VEC;
    const bool in = c < dim;
    const int b0 = blockIdx.x * BT, b1 = min(n, b0 + BT);
    const int p0 = b0 + g * RUN_TOKENS, p1 = min(b1, p0 + RUN_TOKENS);

    float acc[VEC];
    uint32_t cur = none, first = none;
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
    bool lead = true;  // still in the group's first run
    for (int p = p0; p < p1; p += U) {
        uint32_t kk[U];
        float v[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u) kk[u] = p + u < p1 ? keys[p + u] : none;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[u][k] = 0.f;
            if (kk[u] != none && in) load_row<VEC>(dout + (int64_t)pos[p + u] * ds + c, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kk[u] == none) break;  // sorted last: nothing follows
            if (p + u == p0) first = cur = kk[u];
            if (kk[u] != cur) {
                if (lead) {
#pragma unroll
                    for (int k = 0; k < VEC; ++k) s_sum[2 * g][l * VEC + k] = acc[k];
                    lead = false;
                } else if (in) {  // a run between two others of the group is whole
#pragma unroll
                    for (int k = 0; k < VEC; ++k) acc[k] *= scale;
                    store_row<VEC>(dtable + (int64_t)cur * ts + c, acc);
                }
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
                cur = kk[u];
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) acc[k] += v[u][k];
        }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) s_sum[2 * g + (lead ? 0 : 1)][l * VEC + k] = acc[k];
    if (l == 0) {
        s_key[2 * g] = first;
        s_key[2 * g + 1] = lead ? none : cur;
    }
    __syncthreads();

    // the groups' first and last runs in order, one thread per column
    const uint32_t before = b0 > 0 ? keys[b0 - 1] : none;
    const uint32_t after = b1 < n ? keys[b1] : none;
    for (int j = threadIdx.x; j < CW; j += EB) {
        const bool col = c0 + j < dim;
        uint32_t run = none;
        float sum = 0.f;
        bool open = false;      // the run began in an earlier block
        bool has_tail = false;  // the block's last run goes on and began here
        auto close = [&](bool goes_on) {
            if (run == none) return;
            if (open) {
                if (col) part[(size_t)blockIdx.x * 2 * dim + c0 + j] = sum;
                if (!goes_on && j == 0 && blockIdx.y == 0) end_block[run] = blockIdx.x;
            } else if (goes_on) {
                if (col) part[((size_t)blockIdx.x * 2 + 1) * dim + c0 + j] = sum;
                has_tail = true;
            } else if (col) {
                dtable[(int64_t)run * ts + c0 + j] = (T)(sum * scale);
            }
        };
        bool any = false;
        for (int e = 0; e < 2 * G; ++e) {
            const uint32_t key = s_key[e];
            if (key == none) continue;
            if (key != run) {
                close(false);
                open = !any && key == before;
                any = true;
                run = key;
                sum = 0.f;
            }
            sum += s_sum[e][j];
        }
        close(run == after);
        if (j == 0 && blockIdx.y == 0) tail_key[blockIdx.x] = has_tail ? run : none;
    }
}

// Rows whose run crosses blocks: the last run of block b, then the first runs
// of the blocks after it up to the one where it ends, a contiguous share per
// row group, the groups joined in order.
template <class T, int VEC, int LPR>
__global__ __launch_bounds__(JOIN_T) void k_embed_join(int dim, int vocab, const uint32_t* __restrict__ tail_key,
                                                       const uint32_t* __restrict__ end_block,
                                                       const float* __restrict__ part, float scale,
                                                       T* __restrict__ dtable, int64_t ts) {
    constexpr int G = JOIN_T / LPR;
    constexpr int CW = LPR * VEC;
    __shared__ float s_sum[G][CW];
    const uint32_t key = tail_key[blockIdx.x];
    if (key == (uint32_t)vocab) return;
    const int g = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int c = blockIdx.y * CW + l * VEC;
    const int b = blockIdx.x, cnt = (int)end_block[key] - b + 1;
    const int per = (cnt + G - 1) / G;
    const int j0 = g * per, j1 = min(cnt, j0 + per);
    float acc[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
    if (c < dim) {
#pragma unroll 4
        for (int j = j0; j < j1; ++j) {
            const float* q = part + ((size_t)(b + j) * 2 + (j == 0 ? 1 : 0)) * dim + c;
#pragma unroll
            for (int k = 0; k < VEC; ++k) acc[k] += q[k];
        }
    }
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
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] = s_sum[0][l * VEC + k] * scale;
        store_row<VEC>(dtable + (int64_t)key * ts + c, acc);
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
};

template <class T, int VEC, int LPR>
hipError_t embed_rows(const EmbedArgs& a, bool backward, hipStream_t s) {
    constexpr int G = EB / LPR;
    if (!backward) {
        const int64_t blocks = (a.n + G * 4 - 1) / (G * 4);
        k_embed<T, VEC, LPR><<<(unsigned)blocks, EB, 0, s>>>(a.n, a.dim, a.vocab, (const T*)a.src, a.ss, a.ids, a.wide,
                                                            a.scale, (T*)a.dst, a.ds);
        return hipGetLastError();
    }
    constexpr int BT = G * RUN_TOKENS;
    const int nb = (int)((a.n + BT - 1) / BT);
    const dim3 grid(nb, (a.dim + LPR * VEC - 1) / (LPR * VEC));
    k_embed_runs<T, VEC, LPR><<<grid, EB, 0, s>>>((int)a.n, a.dim, a.vocab, a.keys, a.pos, (const T*)a.src, a.ss,
                                                 a.scale, (T*)a.dst, a.ds, a.part, a.tail_key, a.end_block);
    if (nb > 1)
        k_embed_join<T, VEC, LPR><<<grid, JOIN_T, 0, s>>>(a.dim, a.vocab, a.tail_key, a.end_block, a.part, a.scale,
                                                         (T*)a.dst, a.ds);
    return hipGetLastError();
}

template <class T, int VEC>
hipError_t embed_pick(const EmbedArgs& a, bool backward, hipStream_t s) {
    const int v = (a.dim + VEC - 1) / VEC;
    if (v <= 8) return embed_rows<T, VEC, 8>(a, backward, s);
    if (v <= 16) return embed_rows<T, VEC, 16>(a, backward, s);
    if (v <= 32) return embed_rows<T, VEC, 32>(a, backward, s);
    return embed_rows<T, VEC, 64>(a, backward, s);
}

template <class T>
hipError_t embed_run(const EmbedArgs& a, bool backward, hipStream_t s) {
    if (wide_rows<T>(a.src, a.ss, a.dim) && wide_rows<T>(a.dst, a.ds, a.dim))
        return embed_pick<T, WIDE<T>>(a, backward, s);
    return embed_pick<T, 1>(a, backward, s);
}

template <class T>
hipError_t zero_rows(int64_t rows, int dim, void* p, int64_t stride, hipStream_t s) {
    const bool w = wide_rows<T>(p, stride, dim);
    const int64_t total = rows * (w ? dim / WIDE<T> : dim);
    const int64_t want = (total + EB - 1) / EB;
    const unsigned blocks = (unsigned)(want < 4096 ? want : 4096);
    if (w)
        k_zero_rows<T, WIDE<T>><<<blocks, EB, 0, s>>>(rows, dim, (T*)p, stride);
    else
        k_zero_rows<T, 1><<<blocks, EB, 0, s>>>(rows, dim, (T*)p, stride);
    return hipGetLastError();
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// The shortest run of positions per block (64 lanes per row) bounds the block count.
int64_t max_blocks(int64_t n) { return (n + EB / 64 * RUN_TOKENS - 1) / (EB / 64 * RUN_TOKENS); }

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
    return half ? embed_run<bf16>(a, false, stream) : embed_run<float>(a, false, stream);
}

hipError_t launch_embed_bwd(int64_t n, int dim, int vocab, bool half, const void* ids, bool wide_ids, float scale,
                            const void* dout, int64_t dout_stride, void* dtable, int64_t dtable_stride, char* ws,
                            hipStream_t stream) {
    hipError_t e = half ? zero_rows<bf16>(vocab, dim, dtable, dtable_stride, stream)
                        : zero_rows<float>(vocab, dim, dtable, dtable_stride, stream);
    if (e != hipSuccess || n == 0) return e;
    const EmbedLayout L = embed_bwd_layout(n, dim, vocab);
    uint32_t* keys[2] = {(uint32_t*)(ws + L.keys[0]), (uint32_t*)(ws + L.keys[1])};
    uint32_t* pos[2] = {(uint32_t*)(ws + L.pos[0]), (uint32_t*)(ws + L.pos[1])};
    k_embed_keys<<<(unsigned)((n + EB - 1) / EB), EB, 0, stream>>>((int)n, vocab, ids, wide_ids, keys[0], pos[0],
                                                                  (uint32_t*)(ws + L.sort), RADIX_TOTAL_WORDS);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    int at = 0;
    e = launch_radix_sort((int)n, vocab, keys, pos, ws + L.sort, &at, stream);
    if (e != hipSuccess) return e;
    EmbedArgs a{};
    a.n = n;
    a.dim = dim;
    a.vocab = vocab;
    a.src = dout;
    a.ss = dout_stride;
    a.dst = dtable;
    a.ds = dtable_stride;
    a.scale = scale;
    a.keys = keys[at];
    a.pos = pos[at];
    a.part = (float*)(ws + L.part);
    a.tail_key = (uint32_t*)(ws + L.tail_key);
    a.end_block = (uint32_t*)(ws + L.end_block);
    return half ? embed_run<bf16>(a, true, stream) : embed_run<float>(a, true, stream);
}

}  // namespace gs
