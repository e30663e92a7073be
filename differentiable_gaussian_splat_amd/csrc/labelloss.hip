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
// follows the count on the device, so unlabelled rows (whatever they hold) are
// not multiplied and reach no sum. Tile sizes, splits and workspace are chosen on
// the host for all rows, so that few labelled ones leave parts of the chip idle.
//
// Types. bfloat16 rows are multiplied as they are, with float32 sums. Between
// the products dz is two bfloat16 parts (to 2^-16 of each entry) where the
// products are small. Where they are large it is one (each entry off by half a
// step, 2^-8 of itself, at most: a second would take twice the bytes and twice the
// products), but for the label's entry, most of a row's gradient: that one stays
// float32 and joins dx and dw apart, in dw as sums over the rows of each label in
// a fixed order (8192 x 1024 x 65536: 53 us of 4.4 ms).
// float32 rows are split into three bfloat16 parts (8 + 8 + 8 bits, all of the
// value) and six products of parts are summed, smallest first; the three left
// out are below 2 x 2^-24 + 2^-32 of the product of magnitudes, near a float32
// product's own rounding. The matrix units take bfloat16 sixteen times as fast as float32,
// so six products are cheaper than one. Where one side is short the kernels of
// flatloss.hpp take over.
#include "elem.hpp"
#include "launch.hpp"

namespace gs {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int BN = 128;         // columns of every product's tile (rows of x, or of the vocabulary)
constexpr int GT = 256;         // threads: four waves, two blocks to a compute unit
// A staged step: 32 deep and three of them in LDS (one read, two on their way),
// or, with the three parts of split operands side by side, 16 deep and two:
// the six products of a step make up for the shorter way ahead. dz in two parts: 32 deep and two.
constexpr int step_depth(int parts) { return parts == 3 ? 16 : 32; }
constexpr int step_buffers(int parts_b) { return parts_b > 1 ? 2 : 3; }
constexpr int KPAD = 16;        // columns of packed operands are padded to it in float32, to twice it in bfloat16
constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;

enum Mode { LSE, DZ, DX, DW };

struct Product {
    const bf16 *a, *b;            // operands: rows of tiles, or (transposed) rows along the depth
    int64_t lda, ldb, pa, pb;     // row strides and distance between the parts of a split operand
    int m, n, k;                  // n, k: host bounds where the device count does not give them
    int splits;                   // of the depth
    int grid;                     // blocks per split
    const int32_t* count;         // labelled rows
    // epilogues
    const int32_t* rows;          // labelled row -> row of the caller's arrays
    const void* labels;
    int wide_labels;
    int v0, vocab, np;
    float2* part;                 // LSE: [slab][np]
    float* target;                // LSE: z at the label
    const float *lse, *dmean, *dloss;
    bf16* dz;                     // DZ: [parts][np][lddz]
    float* own;                   // DZ, one part of dz: per row, the label's entry (0 in dz)
    int64_t lddz, pdz;
    float* acc;                   // DX, DW with splits: [split][rows][ldacc]
    int64_t ldacc, pacc;
    int add;
    void* out;                    // DW without splits
    int64_t ldout;
    int out_dim, out_wide;
    const int32_t* slot;          // DW, one part of dz, no splits: per column of dz, its row of own_sums + 1, or 0
    const float* own_sums;        // the labels' entries times x, by label: [row][ldacc]
};

// The upstream gradient of a labelled row's loss.
__device__ __forceinline__ float up_of(const float* dmean, const float* dloss, int row, int cnt) {
    float u = dloss ? dloss[row] : 0.f;
    if (dmean) u += dmean[0] / (float)cnt;
    return u;
}

// How a row's chunks are exchanged.
template <int BK>
__device__ __forceinline__ int chunk_turn(int r) {
    return BK == 32 ? (r >> 2) & 3 : (r >> 3) & 1;
}

// Stages a T x BK operand tile into LDS: rows of BK depth elements (16-byte
// chunks exchanged by the row, so that the sixteen lanes that read together
// find one depth's chunks spread over all banks) or, TR, depth rows of T elements
// (64-byte segments exchanged by the depth row, for the transposing reads).
template <int T, bool TR, int BK>
struct Stage {
    static constexpr int NI = T * BK / 2048;  // 16-byte loads per lane
    uint32_t off[NI];                  // byte offsets of the lane's chunks from the tile's first element

    __device__ __forceinline__ Stage(int64_t ld) {
        const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (TR) {
                const int r = (i * 4 + w) * (512 / T) + l / (T / 8);
                const int seg = ((l % (T / 8)) / 4) ^ (r & (T / 32 - 1) & 3);
                off[i] = (uint32_t)((r * ld + seg * 32 + (l % 4) * 8) * 2);
            } else {
                constexpr int C = BK / 8;  // chunks of a row
                const int r = (i * 4 + w) * (64 / C) + l / C;
                off[i] = (uint32_t)((r * ld + ((l % C) ^ chunk_turn<BK>(r)) * 8) * 2);
            }
        }
    }

    // p: first element of the tile; bytes: how far the operand's memory reaches from there (reads beyond give 0);
    // lds: byte address of the tile in LDS. The load writes no register, so that nothing of it is the compiler's to
    // keep: step_barrier waits for its arrival. (As a builtin, every LDS read behind it would wait for it first.)
    // The wait states are those that a vector write of the descriptor and the write of m0 need before it.
    __device__ __forceinline__ void load(const bf16* p, int64_t bytes, uint32_t lds) const {
        const uint32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const uint64_t at = (uint64_t)p;
        u32x4 r;
        r[0] = __builtin_amdgcn_readfirstlane((uint32_t)at);
        r[1] = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)) & 0xffffu;
        r[2] = __builtin_amdgcn_readfirstlane((uint32_t)(bytes > 0x7fffffff ? 0x7fffffff : bytes < 0 ? 0 : bytes));
        r[3] = 0x00020000u;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(
                             lds + (i * 4 + w) * 1024),
                         "v"(off[i]), "s"(r)
                         : "memory", "m0");
    }
};

// The 8 depth elements of a lane for one 32-row fragment: row r0 + lane % 32, depth 16 kk + 8 (lane / 32).
template <int T, bool TR, int BK>
__device__ __forceinline__ bf16x8 fragment(const bf16* lds, int r0, int kk) {
    const int l = threadIdx.x & 63;
    if constexpr (TR) {
        const int j = l % 16, k = 16 * kk + 8 * (l / 32) + j / 4;
        const bf16* q = lds + k * T + (((r0 / 32) ^ ((j / 4) & (T / 32 - 1))) * 32) + ((l / 16) & 1) * 16 + (j % 4) * 4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)q);
        const s16x4 hi =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(q + 4 * T));
        bf16x8 v;
        __builtin_memcpy(&v, &lo, 8);
        __builtin_memcpy(reinterpret_cast<char*>(&v) + 8, &hi, 8);
        return v;
    } else {
        const int r = r0 + l % 32;
        return *reinterpret_cast<const bf16x8*>(lds + r * BK + ((2 * kk + l / 32) ^ chunk_turn<BK>(r)) * 8);
    }
}

// Waits until all but the last `left` of this wave's loads have arrived and its LDS reads are done, then for the block.
template <int LEFT>
__device__ __forceinline__ void step_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// 2^x; results below 2^-126 are 0
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// exp(z - ref); the difference first, which is exact where the two are close. One multiply-add with a scaled reference
// would be off by the rounding of that, which grows with the logit and not with its term (8192 x 256 x 50021 forward
// 255 us, so 258; 5003 x 129 x 8191 float32 with gradients 330 and 332). The backward's reference, lse, is one float32:
// p is off by half a step of it, and p of a label whose logit exceeds the others' by more than lse can hold is 1.
__device__ __forceinline__ float exp_diff(float z, float ref) { return exp2_fast((z - ref) * LOG2E); }

// Rows staged for TM row blocks per wave (a power of two, for the staging's lanes).
constexpr int staged_rows(int tm, int parts) { return tm == 1 && parts == 1 ? 64 : tm <= 2 ? 128 : 256; }
constexpr int tile_elements(int tm, int parts, int parts_b) {
    return step_buffers(parts_b) * (parts * staged_rows(tm, parts) + parts_b * BN) * step_depth(parts);
}
// The parts of operand b: dz's where it is one.
constexpr int parts_of_b(int mode, int parts, int dzp) { return mode == DX || mode == DW ? dzp : parts; }

// The logits of split operands that are no number because one of their values is infinite, or too large for a part's
// product: the value stands in its first part alone, and its products with the other operand's later parts (0, or of
// the other sign) are wrong. Where the six products give no number, the product of the first parts alone is the
// logit: infinite (the other products would not change that), or no number in earnest. Read straight from the packed
// operands: rows of a from p.a + m, of b from p.b + n.
template <int TM, int TN>
__device__ __forceinline__ void first_parts(const Product& p, int m, int n, f32x16 (&acc)[TM][TN]) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 16; ++e) bad = bad || acc[i][j][e] != acc[i][j][e];
            if (!__any(bad)) continue;
            const bf16* a = p.a + min(m + 32 * i + l % 32, p.m - 1) * p.lda + 8 * (l / 32);
            const bf16* b = p.b + (n + 32 * j + l % 32) * p.ldb + 8 * (l / 32);
            f32x16 z;
#pragma unroll
            for (int e = 0; e < 16; ++e) z[e] = 0.f;
#pragma unroll 1
            for (int k = 0; k < p.k; k += 16)
                z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8*>(a + k),
                                                           *reinterpret_cast<const bf16x8*>(b + k), z, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = acc[i][j][e] != acc[i][j][e] ? z[e] : acc[i][j][e];
        }
}

// One product, C[m][n] = sum_k A[m][k] B[n][k], by 64 TM x 128 tiles; a lane
// holds, for one n, runs of four consecutive m. PARTS: 1, or 3 for split
// operands; DZP: dz's parts.
//
// The loop keeps several steps in LDS: while one is multiplied the next are
// loaded straight to LDS, and one barrier a step both publishes the arrived
// step and frees the one before it. Loads past the last step are made with an
// empty extent (they bring zeros), which keeps the count of loads in flight
// the same in every step.
//
// 8192 x 1024 x 65536 bfloat16: LSE 1.16 ms (0.95 PFLOP/s), DZ 1.29 (0.85),
// DX and DW together 2.08 (1.06); a large library product reaches 1.25 to 1.49,
// the matrix units alone on random data 1.84 (2.4 on zeros). The units are busy
// 52 % of the time in LSE, 43 in DZ and 57 in the pair, at 1.8 GHz: the epilogues
// run beside no product, and what holds the rest was not found. LDS is read
// without bank conflicts and 20 % of the time. 256 x 256 tiles (by eight
// waves, or by four of 128 x 128), reads of the next fragments ahead of the
// barrier, and raised priority of the products all measured within 3 %.
template <int MODE, int PARTS, int DZP, int TM, class T>
__device__ __forceinline__ void product(const Product& p, int block, bf16* s_tiles) {
    constexpr bool TA = MODE == DX || MODE == DW, TB = MODE == DW;
    constexpr int TN = 2, WM = 32 * TM, WN = 32 * TN;  // 2 x 2 waves of WM rows and WN columns
    constexpr int PB = parts_of_b(MODE, PARTS, DZP);
    constexpr int BM = 2 * WM, SM = staged_rows(TM, PARTS), BK = step_depth(PARTS), BUFS = step_buffers(PB);
    constexpr int STEP = (PARTS * SM + PB * BN) * BK;  // elements of a staged step: the a tile's parts, then the b tile's
    const int cnt = *p.count;
    const int nn = MODE == DW ? p.n : cnt;
    const int mt = (p.m + BM - 1) / BM, nt = (nn + BN - 1) / BN;
    // consecutive blocks go to the eight dies in turn: each takes a contiguous
    // run of tiles, in groups of 8 columns, so that its cache serves both operands
    const int tiles = mt * nt, per_die = (tiles + 7) / 8;
    const int split = block / p.grid, b0 = block - split * p.grid;  // p.grid: blocks of one split, a multiple of 8
    const int tile = (b0 & 7) * per_die + (b0 >> 3);
    if ((b0 >> 3) >= per_die || tile >= tiles) return;
    const int grp = tile / (8 * mt), in_grp = tile - grp * 8 * mt;
    const int gw = min(8, nt - grp * 8);
    const int m0 = in_grp / gw * BM, n0 = (grp * 8 + in_grp % gw) * BN;

    const int depth = MODE == DW ? cnt : p.k;
    const int nk = (depth + BK - 1) / BK;
    const int share = (nk + p.splits - 1) / p.splits;
    const int k_first = min(nk, split * share), k_end = min(nk, k_first + share);
    const int steps = k_end - k_first;

    const Stage<SM, TA, BK> sa(p.lda);
    const Stage<BN, TB, BK> sb(p.ldb);
    const int a_rows = TA ? (MODE == DW ? p.np : p.k) : p.m;  // rows of the operand's memory
    const int b_rows = p.np;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)s_tiles;
    int kt = 0;  // the next step to load
    auto issue = [&](int buf) {
        const bool live = kt < steps;
        const int64_t k0 = live ? (k_first + kt) * BK : 0;
        const bf16* a = p.a + (TA ? k0 * p.lda + m0 : m0 * p.lda + k0);
        const bf16* b = p.b + (TB ? k0 * p.ldb + n0 : n0 * p.ldb + k0);
        const int64_t ea = TA ? (min((int64_t)BK, a_rows - k0) - 1) * p.lda + p.m - m0
                              : (int64_t)(min(SM, a_rows - m0) - 1) * p.lda + BK;
        const int64_t eb = TB ? (min((int64_t)BK, b_rows - k0) - 1) * p.ldb + p.ldb - n0
                              : (int64_t)(min(BN, b_rows - n0) - 1) * p.ldb + BK;
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
            sa.load(a + q * p.pa, live ? ea * 2 : 0, lds0 + (buf * STEP + q * SM * BK) * 2);
#pragma unroll
        for (int q = 0; q < PB; ++q)
            sb.load(b + q * p.pb, live ? eb * 2 : 0, lds0 + (buf * STEP + PARTS * SM * BK + q * BN * BK) * 2);
        ++kt;
    };

    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int wm = (w % 2) * WM, wn = (w / 2) * WN;
    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

    constexpr int LOADS = PARTS * Stage<SM, TA, BK>::NI + PB * Stage<BN, TB, BK>::NI;  // of one step
    for (int t = 0; t < BUFS - 1; ++t) issue(t);
    int buf = 0;
    for (int t = 0; t < steps; ++t) {
        step_barrier<(BUFS - 2) * LOADS>();
        issue(buf == 0 ? BUFS - 1 : buf - 1);
        const bf16 *la = s_tiles + buf * STEP, *lb = la + PARTS * SM * BK;
        buf = buf == BUFS - 1 ? 0 : buf + 1;
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
            bf16x8 fa[PARTS][TM], fb[PB][TN];
#pragma unroll
            for (int q = PB - 1; q >= 0; --q) {  // PB >= PARTS
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    if (q < PARTS) fa[q][i] = fragment<SM, TA, BK>(la + q * SM * BK, wm + 32 * i, kk);
#pragma unroll
                for (int j = 0; j < TN; ++j) fb[q][j] = fragment<BN, TB, BK>(lb + q * BN * BK, wn + 32 * j, kk);
            }
            // the products of parts whose sizes add up to 2^-16 of the operands' and more, smallest first
#pragma unroll
            for (int sum = PB - 1; sum >= 0; --sum)
#pragma unroll
                for (int q = sum < PARTS ? sum : PARTS - 1; q >= 0; --q)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[q][i], fb[sum - q][j], acc[i][j], 0,
                                                                               0, 0);
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the loads past the last step

    // element e of acc[i][j]: m = mb + 32 i + 8 (e / 4) + e % 4, n = nb + 32 j
    const int mb = m0 + wm + 4 * (l / 32), nb = n0 + wn + l % 32;
    if constexpr (MODE == LSE || MODE == DZ) {
        if constexpr (PARTS == 3) first_parts(p, m0 + wm, n0 + wn, acc);
        const bool edge = m0 + BM > p.m;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int n = nb + 32 * j;
            int room = p.m - mb;  // elements at or beyond it are past the vocabulary
            asm volatile("" : "+v"(room));  // compared anew for each j: kept comparisons would not fit the registers
            const int row = n < cnt ? p.rows[n] : -1;
            const int lab = row >= 0 ? row_index(p.labels, p.wide_labels, row, p.vocab) - p.v0 : -1;
            const int at = lab - mb;  // of the label's element among this lane's: 32 i + 8 (e / 4) + e % 4
            const bool hit = __any(lab >= m0 + wm && lab < m0 + wm + WM);
            if constexpr (MODE == LSE) {
                if (edge)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (32 * i + 8 * (e / 4) + e % 4 >= room) acc[i][j][e] = -INFINITY;
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 2) top = fmaxf(fmaxf(top, acc[i][j][e]), acc[i][j][e + 1]);
                top = fmaxf(top, __shfl_xor(top, 32));
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        s0 += exp_diff(acc[i][j][e], top);
                        s1 += exp_diff(acc[i][j][e + 1], top);
                    }
                float sum = s0 + s1;
                if (!__all(fabsf(top) < INFINITY)) {
                    // an infinite maximum: entries equal to +inf count 1, other numbers 0
                    float c = 0.f;
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float z = acc[i][j][e];
                            c += z != z ? z : z == INFINITY ? 1.f : 0.f;
                        }
                    if (!(fabsf(top) < INFINITY)) sum = c;
                }
                sum += __shfl_xor(sum, 32);
                if (l < 32 && n < cnt)
                    p.part[(int64_t)((m0 + wm) / WM) * p.np + n] = make_float2(top, sum);
                if (hit)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (at == 32 * i + 8 * (e / 4) + e % 4 && lab >= 0) p.target[n] = acc[i][j][e];
            } else {
                const float lse = row >= 0 ? p.lse[row] : 0.f;
                const float up = row >= 0 ? up_of(p.dmean, p.dloss, row, cnt) : 0.f;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] = exp_diff(acc[i][j][e], lse);
                if (hit) {
                    float own = 0.f;
                    bool here = false;
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const bool is = at == 32 * i + 8 * (e / 4) + e % 4;
                            acc[i][j][e] -= is ? 1.f : 0.f;
                            if (DZP == 1) {
                                own = is ? acc[i][j][e] : own;
                                acc[i][j][e] = is ? 0.f : acc[i][j][e];
                            }
                            here = here || is;
                        }
                    if (DZP == 1 && here && lab >= 0) p.own[n] = own * up;
                }
                // dz is zero for rows past the labelled ones (read up to whole steps by dw's product; z there is no
                // number where a label's row is infinite) and past the vocabulary
                if (__any(row < 0))
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[i][j][e] = row < 0 ? 0.f : acc[i][j][e];
                if (edge)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (32 * i + 8 * (e / 4) + e % 4 >= room) acc[i][j][e] = 0.f;
                // a lane and the one 32 further hold runs of four columns in turn: they
                // exchange runs, so that each stores eight columns at a time
                const int h = l / 32;
                bf16* q = p.dz + n * p.lddz + (m0 + wm + 8 * h);
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 8) {
                        float g[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) g[c] = acc[i][j][e + c] * up;
#pragma unroll
                        for (int c = 0; c < DZP; ++c) {
                            union {
                                bf16x4 v[2];
                                uint32_t u[4];
                            } o;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const bf16 b = (bf16)g[k];
                                o.v[k / 4][k % 4] = b;
                                if (c + 1 < DZP) g[k] -= (float)b;
                            }
                            auto x0 = __builtin_amdgcn_permlane32_swap(o.u[0], o.u[2], false, false);
                            auto x1 = __builtin_amdgcn_permlane32_swap(o.u[1], o.u[3], false, false);
                            *reinterpret_cast<uint4*>(q + c * p.pdz + 32 * i + 2 * e) =
                                make_uint4(x0[0], x1[0], x0[1], x1[1]);
                        }
                    }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int n = nb + 32 * j;
            if (n >= nn) continue;
            int room = (p.acc ? (int)p.ldacc : p.out_dim) - mb;
            asm volatile("" : "+v"(room));
            if (p.acc) {
                float* q = p.acc + split * p.pacc + n * p.ldacc + mb;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        if (32 * i + 2 * e >= room) continue;
                        float4* d = reinterpret_cast<float4*>(q + 32 * i + 2 * e);
                        float4 v = make_float4(acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]);
                        if (p.add) {
                            const float4 o = *d;
                            v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
                        }
                        *d = v;
                    }
            } else {
                T* q = static_cast<T*>(p.out) + n * p.ldout + mb;
                if constexpr (MODE == DW && DZP == 1) {
                    const int slot = p.slot[n];
                    if (slot) {
                        const float* own = p.own_sums + (int64_t)(slot - 1) * p.ldacc + mb;
#pragma unroll
                        for (int i = 0; i < TM; ++i)
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                if (32 * i + 2 * e >= room) continue;
                                const float4 v = *reinterpret_cast<const float4*>(own + 32 * i + 2 * e);
                                acc[i][j][e] += v.x;
                                acc[i][j][e + 1] += v.y;
                                acc[i][j][e + 2] += v.z;
                                acc[i][j][e + 3] += v.w;
                            }
                    }
                }
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const int c0 = 32 * i + 2 * e;
                        if (p.out_wide && c0 + 4 <= room) {
                            if constexpr (sizeof(T) == 2) {
                                bf16x4 v;
#pragma unroll
                                for (int c = 0; c < 4; ++c) v[c] = (bf16)acc[i][j][e + c];
                                *reinterpret_cast<bf16x4*>(q + c0) = v;
                            } else {
                                *reinterpret_cast<float4*>(q + c0) =
                                    make_float4(acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]);
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (c0 + c < room) q[c0 + c] = (T)acc[i][j][e + c];
                        }
                    }
            }
        }
    }
}

template <int MODE, int PARTS, int DZP, int TM, class T>
__global__ __launch_bounds__(GT, 2) void k_product(Product p) {
    __shared__ __align__(16) bf16 s_tiles[tile_elements(TM, PARTS, parts_of_b(MODE, PARTS, DZP))];
    product<MODE, PARTS, DZP, TM, T>(p, blockIdx.x, s_tiles);
}

// dx and dw, which read the same dz, in one launch: together they fill the chip better, and small ones wait once.
template <int PARTS, int DZP, int TM, class T>
__global__ __launch_bounds__(GT, 2) void k_product_pair(Product dx, Product dw) {
    __shared__ __align__(16) bf16 s_tiles[tile_elements(TM, PARTS, DZP)];
    const int first = dx.grid * dx.splits;
    if ((int)blockIdx.x < first)
        product<DX, PARTS, DZP, TM, T>(dx, blockIdx.x, s_tiles);
    else
        product<DW, PARTS, DZP, TM, T>(dw, blockIdx.x - first, s_tiles);
}

// ---------------------------------------------------------------- labelled rows

constexpr int LPT = 4;                // rows per thread
constexpr int LT = 1024, LROWS = LT * LPT;  // threads and rows of a block that lists labelled rows
constexpr int PT = 256, PROWS = PT * LPT;   // threads of a packing block, rows of which it can make the list itself
constexpr int64_t LOOK_BACK = 8192;  // rows up to which a block counts the labels before its own rows itself

// The arrays that the labels give: rows[], the labelled rows in order; place[r],
// the position of row r in it, or -1; their number; loss and lse (nullable),
// cleared for the other rows; done, the joining blocks' counter, cleared.
struct LabelRows {
    int64_t n;
    int vocab;
    int wide;
    const void* labels;
    int32_t *rows, *place, *count, *done;
    float *loss, *lse;
};

// block_count[b] = labelled rows of block b.
__global__ __launch_bounds__(LT) void k_label_count(LabelRows a, int32_t* __restrict__ block_count) {
    __shared__ int s_w[LT / 64];
    const int64_t r0 = (int64_t)blockIdx.x * LROWS + threadIdx.x;
    int c = 0;
#pragma unroll
    for (int k = 0; k < LPT; ++k)
        c += __popcll(__ballot(r0 + k * LT < a.n && row_index(a.labels, a.wide, r0 + k * LT, a.vocab) >= 0));
    if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = c;
    __syncthreads();
    if (threadIdx.x == 0) {
        c = 0;
        for (int k = 0; k < LT / 64; ++k) c += s_w[k];
        block_count[blockIdx.x] = c;
    }
}

// The labels of block `b`'s rows (a wave takes 64 LPT consecutive ones); `before`:
// a count per thread that adds up to the labelled rows before the block. s_list
// (nullable): the rows also go there. Returns the labelled rows up to the block's end.
template <int NT>
__device__ __forceinline__ int label_rows(const LabelRows& a, int b, int before, bool write, int* s_w, int* s_list) {
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t r0 = (int64_t)b * NT * LPT + w * (64 * LPT) + lane;
    uint64_t have[LPT];
    int own = 0;
#pragma unroll
    for (int k = 0; k < LPT; ++k) {
        have[k] = __ballot(r0 + 64 * k < a.n && row_index(a.labels, a.wide, r0 + 64 * k, a.vocab) >= 0);
        own += __popcll(have[k]);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) before += __shfl_xor(before, off);
    if (lane == 0) {
        s_w[w] = before;
        s_w[NT / 64 + w] = own;
    }
    __syncthreads();
    int at = 0, end = 0;
#pragma unroll
    for (int k = 0; k < NT / 64; ++k) {
        at += s_w[k] + (k < w ? s_w[NT / 64 + k] : 0);
        end += s_w[k] + s_w[NT / 64 + k];
    }
#pragma unroll
    for (int k = 0; k < LPT; ++k) {
        const int64_t r = r0 + 64 * k;
        const bool mine = (have[k] >> lane) & 1;
        const int to = at + __popcll(have[k] & (((uint64_t)1 << lane) - 1));
        at += __popcll(have[k]);
        if (mine && s_list) s_list[to] = (int)r;
        if (!write || r >= a.n) continue;
        a.place[r] = mine ? to : -1;
        if (mine) a.rows[to] = (int32_t)r;
        if (!mine && a.loss) a.loss[r] = 0.f;
        if (!mine && a.lse) a.lse[r] = 0.f;
    }
    return end;
}

// block_count (nullable): the blocks' labelled rows, counted before.
__global__ __launch_bounds__(LT) void k_label_rows(LabelRows a, const int32_t* __restrict__ block_count) {
    __shared__ int s_w[2 * LT / 64];
    int c = 0;
    if (block_count) {
        for (int k = threadIdx.x; k < (int)blockIdx.x; k += LT) c += block_count[k];
    } else {  // whole blocks of rows before this one
        const int end = (int)blockIdx.x * LROWS;
        for (int r = threadIdx.x; r < end; r += 16 * LT)
#pragma unroll
            for (int k = 0; k < 16; ++k)
                c += r + k * LT < end && row_index(a.labels, a.wide, r + k * LT, a.vocab) >= 0;
    }
    const int last = label_rows<LT>(a, blockIdx.x, c, true, s_w, nullptr);
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) {
        *a.count = last;
        *a.done = 0;
    }
}

// Rows into bfloat16 parts of kp columns (whole steps, zero beyond dim):
// the first x_blocks blocks pack x's labelled rows, and zero rows up to the
// next multiple of BN, the others every row of w. SMALL: x has at most PROWS
// rows, and each block makes the list of labelled rows for itself first (block
// 0 also writes its arrays), which saves a launch.
struct PackArgs {
    int dim, kp, per_block;  // per_block: rows of a block
    int x_blocks;
    const void *x, *w;
    int64_t xs, ws, w_rows;
    bf16 *xp, *wp;
    int64_t x_part, w_part;  // distance of the parts
};

template <class T, int PARTS, bool SMALL>
__global__ __launch_bounds__(PT) void k_pack(LabelRows a, PackArgs p) {
    __shared__ int s_w[2 * PT / 64];
    __shared__ int s_list[SMALL ? PROWS : 1];
    const bool x = (int)blockIdx.x < p.x_blocks;
    const int64_t r0 = (int64_t)(blockIdx.x - (x ? 0 : p.x_blocks)) * p.per_block;
    int64_t live = p.w_rows, padded = p.w_rows;
    if (x) {
        if (SMALL) {
            live = label_rows<PT>(a, 0, 0, blockIdx.x == 0, s_w, s_list);
            __syncthreads();
            if (blockIdx.x == 0 && threadIdx.x == 0) {
                *a.count = (int)live;
                *a.done = 0;
            }
        } else {
            live = *a.count;
        }
        padded = (live + BN - 1) / BN * BN;
    }
    const int64_t left = padded - r0;
    if (left <= 0) return;
    const uint32_t per = p.kp / 8, total = (uint32_t)(left < p.per_block ? left : p.per_block) * per;
    const T* src = static_cast<const T*>(x ? p.x : p.w);
    const int64_t stride = x ? p.xs : p.ws, part = x ? p.x_part : p.w_part;
    bf16* dst = x ? p.xp : p.wp;
    for (uint32_t i = threadIdx.x; i < total; i += PT) {
        const uint32_t rr = i / per;
        const int64_t r = r0 + rr;
        const int c = (int)(i - rr * per) * 8;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
        if (r < live) {
            const int64_t row = !x ? r : SMALL ? s_list[r] : a.rows[r];
            constexpr int V = WIDE<T>;
            const int64_t room = ((x ? a.n : p.w_rows) - 1 - row) * stride + p.dim - c;
            wide_t<T> raw[8 / V];
#pragma unroll
            for (int k = 0; k < 8 / V; ++k)
                raw[k] = load_row<false>(src + row * stride + c + k * V, p.dim - c - k * V, room - k * V);
#pragma unroll
            for (int k = 0; k < 8 / V; ++k) {
                float t[V];
                widen<false, T>(raw[k], p.dim - c - k * V, t);
#pragma unroll
                for (int j = 0; j < V; ++j) v[k * V + j] = t[j];
            }
        }
        bf16x8 o[PARTS];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            o[0][k] = (bf16)v[k];
            if (PARTS == 3) {
                // a value that would round up to infinity keeps its leading bits instead; an
                // infinite or NaN value stays in its first part alone (first_parts sees to its products)
                const bool fin = fabsf(v[k]) < INFINITY;
                if (fin && !(fabsf((float)o[0][k]) < INFINITY))
                    o[0][k] = (bf16)__uint_as_float(__float_as_uint(v[k]) & 0xffff0000u);
                const float r1 = fin ? v[k] - (float)o[0][k] : 0.f;
                o[PARTS / 2][k] = (bf16)r1;
                o[PARTS - 1][k] = (bf16)(r1 - (float)o[PARTS / 2][k]);
            }
        }
#pragma unroll
        for (int q = 0; q < PARTS; ++q) *reinterpret_cast<bf16x8*>(dst + q * part + r * p.kp + c) = o[q];
    }
}

// ---------------------------------------------------------------- joins

__device__ __forceinline__ float2 lse_join(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x);
    // an equal maximum scales by 1 (also where both are infinite); sums are 0 where the maximum is -inf
    const float fa = a.x == m ? 1.f : exp_diff(a.x, m), fb = b.x == m ? 1.f : exp_diff(b.x, m);
    return make_float2(m, a.y * fa + b.y * fb);
}

// exp(z - top) where top is a maximum that may be infinite: an entry equal to it counts 1 (+inf) or 0 (-inf).
__device__ __forceinline__ float exp_share(float z, float top) {
    if (!(top > -INFINITY)) return z != z ? z : 0.f;
    return z == top ? 1.f : exp_diff(z, top);
}

// The blocks of one launch among all that a kernel takes for its rows.
struct BlockRange {
    int first, all;
};

// Calls launch(blocks, range) for the launches that `all` blocks take.
template <class F>
void launch_ranges(int64_t all, F launch) {
    for (int64_t first = 0; first < all; first += MOST_BLOCKS)
        launch((unsigned)(all - first < MOST_BLOCKS ? all - first : MOST_BLOCKS), BlockRange{(int)first, (int)all});
}

constexpr int JR = 64;  // rows per block of the join
constexpr int JT = 1024;

// The mean loss from the blocks' sums, added in block order, by one block of NT threads.
template <int NT>
__device__ __forceinline__ void loss_mean(const double* block_sum, int blocks, int cnt, float* mean,
                                          int32_t* count_out) {
    __shared__ double s_sum[NT / 64];
    double sum = 0.0;
    for (int k = threadIdx.x; k < blocks; k += NT)
        sum += __hip_atomic_load(&block_sum[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < NT / 64; ++k) sum += s_sum[k];
        *mean = cnt > 0 ? (float)(sum / (double)cnt) : 0.f;
        *count_out = cnt;
    }
}

// Joins the slabs' (maximum, sum) pairs of each labelled row (and `state`, the
// join of earlier pieces; with `more` pieces to come the result is left there
// again), then the row's loss. Of all launches' blocks the one that ends last adds
// the blocks' losses in block order: the mean.
__global__ __launch_bounds__(JT) void k_lse_join(BlockRange range, int slabs, int np, const float2* __restrict__ part,
                                                 const float* __restrict__ target, const int32_t* __restrict__ rows,
                                                 const int32_t* __restrict__ count, float2* __restrict__ state,
                                                 bool first, bool more, float* __restrict__ loss,
                                                 float* __restrict__ lse, double* __restrict__ block_sum,
                                                 int32_t* __restrict__ done, float* __restrict__ mean,
                                                 int32_t* __restrict__ count_out) {
    constexpr int G = JT / JR;
    __shared__ float2 s[G][JR];
    __shared__ int s_last;
    const int j = threadIdx.x % JR, g = threadIdx.x / JR;
    const int block = range.first + (int)blockIdx.x, n = block * JR + j, cnt = *count;
    float2 a = make_float2(-INFINITY, 0.f);
    if (n < cnt) {
        if (!first && g == 0) a = state[n];
#pragma unroll 8
        for (int k = g; k < slabs; k += G) a = lse_join(a, part[(int64_t)k * np + n]);
    }
    s[g][j] = a;
    __syncthreads();
    if (g == 0) {
        double mine = 0.0;
        if (n < cnt) {
            for (int k = 1; k < G; ++k) a = lse_join(a, s[k][j]);
            if (more) {
                state[n] = a;
            } else {
                const float z = target[n], ln = log2f(a.y) * LN2;
                const int r = rows[n];
                // (maximum - z) first: exact where they are close
                const float ls = a.x == INFINITY ? a.x - z : (a.x - z) + ln;
                lse[r] = a.x + ln;
                loss[r] = ls;
                mine = (double)ls;
            }
        }
        if (!more) {
            for (int off = 32; off > 0; off >>= 1) mine += __shfl_xor(mine, off);
            if (j == 0) {
                __hip_atomic_store(&block_sum[block], mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                s_last = __hip_atomic_fetch_add(done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                         range.all - 1;
            }
        }
    }
    if (more) return;
    __syncthreads();
    if (s_last) loss_mean<JT>(block_sum, range.all, cnt, mean, count_out);
}

// out[r] = the splits' rows of acc added in order, through place (-1: a zero row) if given.
// own (nullable): per row of acc, a multiple of the row of w that the label names, added on top.
// slot (nullable): per row of out, a row of own_sums + 1 that is added on top, or 0.
struct SplitJoin {
    int64_t rows;
    int splits;
    const float* acc;
    int64_t pacc;
    const int32_t* place;
    void* out;
    int64_t ldout;
    int blocks;
    const float* own;
    const void *labels, *w;
    int wide, vocab;
    int64_t ws;
    const int32_t* slot;
    const float* own_sums;
};

// Two joins in one launch: the first a.blocks blocks do a, the others b.
template <class T>
__global__ __launch_bounds__(256) void k_join_splits(SplitJoin a, SplitJoin b, int dim, int kp, int per_block) {
    const bool second = (int)blockIdx.x >= a.blocks;
    const SplitJoin& j = second ? b : a;
    const int64_t r0 = (int64_t)(blockIdx.x - (second ? a.blocks : 0)) * per_block;
    const int64_t left = j.rows - r0;
    const uint32_t per = (dim + 3) / 4, total = (uint32_t)(left < per_block ? left : per_block) * per;
    for (uint32_t i = threadIdx.x; i < total; i += 256) {
        const uint32_t rr = i / per;
        const int64_t r = r0 + rr;
        const int c = (int)(i - rr * per) * 4;
        const int64_t src = j.place ? j.place[r] : r;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (src >= 0) {
            const float* q = j.acc + src * kp + c;
#pragma unroll 8
            for (int s = 0; s < j.splits; ++s) {
                const float4 t = *reinterpret_cast<const float4*>(q + s * j.pacc);
                v = make_float4(v.x + t.x, v.y + t.y, v.z + t.z, v.w + t.w);
            }
        }
        T* o = static_cast<T*>(j.out) + r * j.ldout + c;
        float f[4] = {v.x, v.y, v.z, v.w};
        if (j.own && src >= 0) {
            const T* w = static_cast<const T*>(j.w) + row_index(j.labels, j.wide, r, j.vocab) * j.ws + c;
            const float own = j.own[src];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + k < dim) f[k] = fmaf(own, (float)w[k], f[k]);
        }
        const int slot = j.slot ? j.slot[r] : 0;
        if (slot) {
            const float4 t = *reinterpret_cast<const float4*>(j.own_sums + (int64_t)(slot - 1) * kp + c);
            f[0] += t.x;
            f[1] += t.y;
            f[2] += t.z;
            f[3] += t.w;
        }
        if (c + 4 <= dim) {
            typedef T vec __attribute__((ext_vector_type(4), aligned(sizeof(T))));
            vec t;
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = (T)f[k];
            *reinterpret_cast<vec*>(o) = t;
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (c + k < dim) o[k] = (T)f[k];
        }
    }
}

}  // namespace

}  // namespace gs

#include "flatloss.hpp"

namespace gs {

namespace {

// ---------------------------------------------------------------- plan

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Blocks a launch needs to fill the chip; products with fewer tiles split their depth.
constexpr int FILL = 512;
constexpr int FEW_TM = 1;

// What m rows cost in tiles of 64 tm: the rows multiplied, weighted by what a
// wave reads from LDS per multiplication (tm + 2 fragments for 2 tm of them).
int64_t tile_cost(int64_t m, int tm) { return up(m, 64 * tm) * (tm + 2) * 6 / tm; }

// Row blocks per wave over the vocabulary: the cheapest of those that make
// enough tiles, otherwise FEW_TM (short tiles: their epilogue is what there is to wait for).
int tm_vocab(int64_t v, int64_t np) {
    int best = FEW_TM;
    int64_t least = 0;
    for (int tm = 1; tm <= 4; ++tm) {
        if (up(v, 64 * tm) / (64 * tm) * (np / BN) < FILL / 2) continue;
        if (least == 0 || tile_cost(v, tm) <= least) {
            best = tm;
            least = tile_cost(v, tm);
        }
    }
    return best;
}

// Row blocks per wave over dim (whose products split their depth to make enough tiles): the cheapest.
int tm_dim(int64_t kp) {
    int best = 1;
    for (int tm = 2; tm <= 4; ++tm)
        if (tile_cost(kp, tm) < tile_cost(kp, best)) best = tm;
    return best;
}

// Splits of a depth of nk steps, `share` of them to a block.
int splits_for(int64_t nk, int64_t share) {
    const int64_t s = (nk + share / 2) / share;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

enum Side { NEITHER, LABELS, ROWS };

// Which side is short enough for the flat kernels. Their gradients' operations
// grow with the short side, the tiled products' cost with the next 128 of it.
// float32 products (six of bfloat16) lose up to SHORT: 46272 x 896 x 64 with
// gradients 0.38 ms flat, 0.59 tiled (x 65); 64 x 1024 x 65536 0.52 and 0.92.
// tiled bfloat16 ones win from 17 labels on (46272 x 896 x 20: 0.42 flat, 0.28
// tiled), and over few rows unless all of it is small (16 x 32 x 1000: 29 us
// flat, 31 tiled; 16 x 64 x 8000: 43 and 39; x 20000: 53 and 50).
Side short_side(int64_t n, int dim, int vocab, bool half) {
    const int most = half ? 16 : SHORT;
    if (vocab <= most) return LABELS;
    if (n > 0 && n <= most && (!half || (int64_t)vocab * dim <= 1 << 20)) return ROWS;
    return NEITHER;
}

struct LossPlan {
    int parts, dzp, kp;            // of the operands, of dz
    int64_t np;                    // rows of x padded to the tile
    int64_t piece_f, piece_b;      // vocabulary rows per piece (whole tiles)
    int tm_z, tm_d;                // row blocks per wave: over the vocabulary, over dim
    int split_dx, split_dw;
    Side shorter;                  // a short side: no packing, no tiles
    int flat_tr, flat_slabs, flat_chunks;
    size_t g;
    size_t rows, place, count, done, block_count, xp, wp, part, target, state, block_sum, dz, own, dxp, dwp, total;
    size_t by_label, slot, own_sums;  // one part of dz: the rows by label, and their sums
};

constexpr int ROW_BLOCKS = 512;  // blocks of the few rows' forward: slabs to join

// The short side's rows rounded up to the gradient kernel's sizes, and its columns per thread.
int few_bucket(int64_t vocab) { return vocab <= 4 ? 4 : vocab <= 8 ? 8 : vocab <= 16 ? 16 : vocab <= 32 ? 32 : 64; }
int few_columns(int64_t vocab) { return vocab <= 8 ? 4 : 2; }

// bfloat16 dz is in two parts (to 2^-16) where that costs less than keeping the labels' entries apart: up to so many
// multiplications in a product. With gradients, us, two parts and apart (and with plain bfloat16 dz): 300 x 64 x 101
// 36, 50 (37); 4000 x 64 x 2000 69, 88 (65); 46272 x 896 x 20 271, 332 (291); 65536 x 64 x 500 191, 195 (158); beyond,
// 65536 x 64 x 1000 258, 239 (200); 300 x 64 x 100000 191, 152 (139); 20000 x 256 x 3000 318, 286 (254); but
// 8192 x 512 x 1000 135, 154 (119).
constexpr int64_t TWO_PARTS = (int64_t)1 << 31;

LossPlan loss_plan(int64_t n, int dim, int vocab, bool half, bool backward) {
    LossPlan L{};
    L.parts = half ? 1 : 3;
    L.kp = (int)up(dim, half ? 2 * KPAD : KPAD);
    L.np = up(n > 0 ? n : 1, BN);
    L.dzp = !half ? 3 : (double)L.np * L.kp * vocab <= (double)TWO_PARTS ? 2 : 1;
    L.tm_z = tm_vocab(vocab, L.np);
    const int64_t unit = 64 * L.tm_z, vp = up(vocab, unit);
    auto piece = [&](int64_t budget) {  // vocabulary rows whose per-row cost fits the budget, in whole tiles
        const int64_t v = budget / L.np / unit * unit;
        return v < unit ? unit : v > vp ? vp : v;
    };
    L.piece_f = piece((int64_t)1 << 30);  // 8 bytes per 32 vocabulary rows at most: 256 MB (or one tile's)
    L.piece_b = piece(((int64_t)1 << 28) / L.dzp);  // 2 bytes per part: 512 MB, or one tile's where that is more
    L.tm_d = tm_dim(L.kp);
    const int64_t mt = up(L.kp, 64 * L.tm_d) / (64 * L.tm_d);
    // dx and dw run in one launch: their depths are split so that all blocks have about one share of it
    const int bk = step_depth(L.parts);
    const int64_t nk_x = (L.piece_b + bk - 1) / bk, nk_w = L.np / bk;
    const int64_t steps = mt * (L.np / BN) * nk_x + mt * (L.piece_b / BN) * nk_w;
    const int64_t least = half ? 8 : 4;  // steps a block should have (of six products each in float32)
    const int64_t share = steps / FILL > least ? steps / FILL : least;
    L.split_dx = splits_for(nk_x, share);
    L.split_dw = splits_for(nk_w, share);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (size_t)up((int64_t)bytes, 256);
        return at;
    };
    L.rows = take((size_t)L.np * 4);
    L.place = take((size_t)L.np * 4);
    L.count = take(4);
    L.done = take(4);
    L.block_count = take((size_t)(L.np / LROWS + 1) * 4);
    L.shorter = short_side(n, dim, vocab, half);
    if (L.shorter != NEITHER) {
        const int64_t few = L.shorter == LABELS ? vocab : n, rows = L.shorter == LABELS ? n : vocab;
        const int cols = few_columns(few);
        L.flat_tr = 1;
        while (L.flat_tr < FT && L.flat_tr * cols < dim) L.flat_tr *= 2;
        L.flat_slabs = few <= 16 ? (dim + L.flat_tr * cols - 1) / (L.flat_tr * cols) : (dim + 127) / 128;
        const int64_t most = 1024 / L.flat_slabs < 64 ? 64 : 1024 / L.flat_slabs > 256 ? 256 : 1024 / L.flat_slabs;
        const int64_t want = (rows + FG - 1) / FG;
        L.flat_chunks = (int)(want < 1 ? 1 : want < most ? want : most);
        L.block_sum = take((size_t)(L.np / FR + 1) * 8);
        if (L.shorter == ROWS) {
            L.part = take((size_t)ROW_BLOCKS * SHORT * 8);
            L.target = take((size_t)SHORT * 4);
        }
        if (backward) {
            L.g = take((size_t)(rows > 0 ? rows : 1) * few_bucket(few) * 4);
            L.dwp = take((size_t)L.flat_chunks * (few > 0 ? few : 1) * L.kp * 4);
        }
        L.total = o;
        return L;
    }
    L.xp = take((size_t)L.parts * L.np * L.kp * 2);
    L.wp = take((size_t)L.parts * vocab * L.kp * 2);
    if (backward) {
        L.dz = take((size_t)L.dzp * L.np * L.piece_b * 2);
        if (L.dzp == 1) {
            L.own = take((size_t)L.np * 4);
            L.by_label = take(embed_bwd_layout(n, L.kp, vocab).total);
            L.slot = take((size_t)vocab * 4);
            L.own_sums = take((size_t)L.np * L.kp * 4);
        }
        L.dxp = take((size_t)L.split_dx * L.np * L.kp * 4);
        L.dwp = L.split_dw > 1 ? take((size_t)L.split_dw * L.piece_b * L.kp * 4) : 0;
    } else {
        L.part = take((size_t)(L.piece_f / (32 * L.tm_z)) * L.np * 8);
        L.target = take((size_t)L.np * 4);
        L.state = take((size_t)L.np * 8);
        L.block_sum = take((size_t)(L.np / JR + 1) * 8);
    }
    L.total = o;
    return L;
}

struct Packed {
    const bf16* w;
    int64_t ldw, pw;
};

// Sets the product's blocks per split for m rows and n columns.
void set_grid(Product& p, int tm, int64_t m, int64_t n) {
    const int64_t t = up(m, 64 * tm) / (64 * tm) * (up(n, BN) / BN);
    p.grid = (int)(t < 8 ? 8 : up(t, 8));
}

template <int MODE, int PARTS, int DZP, class T>
void launch_product(int tm, const Product& p, hipStream_t s) {
    const unsigned grid = (unsigned)p.grid * p.splits;
    if (tm == 4)
        k_product<MODE, PARTS, DZP, 4, T><<<grid, GT, 0, s>>>(p);
    else if (tm == 3)
        k_product<MODE, PARTS, DZP, 3, T><<<grid, GT, 0, s>>>(p);
    else if (tm == 2)
        k_product<MODE, PARTS, DZP, 2, T><<<grid, GT, 0, s>>>(p);
    else
        k_product<MODE, PARTS, DZP, 1, T><<<grid, GT, 0, s>>>(p);
}

template <int PARTS, int DZP, class T>
void launch_pair(int tm, const Product& dx, const Product& dw, hipStream_t s) {
    const unsigned grid = (unsigned)dx.grid * dx.splits + (unsigned)dw.grid * dw.splits;
    if (tm == 4)
        k_product_pair<PARTS, DZP, 4, T><<<grid, GT, 0, s>>>(dx, dw);
    else if (tm == 3)
        k_product_pair<PARTS, DZP, 3, T><<<grid, GT, 0, s>>>(dx, dw);
    else if (tm == 2)
        k_product_pair<PARTS, DZP, 2, T><<<grid, GT, 0, s>>>(dx, dw);
    else
        k_product_pair<PARTS, DZP, 1, T><<<grid, GT, 0, s>>>(dx, dw);
}

LabelRows label_arrays(const LabelLossArgs& a, const LossPlan& L, char* ws, bool forward) {
    LabelRows r{};
    r.n = a.n;
    r.vocab = a.vocab;
    r.wide = a.wide_labels;
    r.labels = a.labels;
    r.rows = (int32_t*)(ws + L.rows);
    r.place = (int32_t*)(ws + L.place);
    r.count = (int32_t*)(ws + L.count);
    r.done = (int32_t*)(ws + L.done);
    r.loss = forward ? a.loss : nullptr;
    r.lse = forward ? a.lse : nullptr;
    return r;
}

void list_rows(const LabelRows& r, const LossPlan& L, char* ws, hipStream_t s) {
    int32_t* bc = r.n <= LOOK_BACK ? nullptr : (int32_t*)(ws + L.block_count);
    const unsigned lb = (unsigned)(r.n > 0 ? (r.n + LROWS - 1) / LROWS : 1);
    if (bc) k_label_count<<<lb, LT, 0, s>>>(r, bc);
    k_label_rows<<<lb, LT, 0, s>>>(r, bc);
}

template <class T>
hipError_t prepare(const LabelLossArgs& a, const LossPlan& L, char* ws, bool forward, Packed& pk, hipStream_t s) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 3;
    const LabelRows r = label_arrays(a, L, ws, forward);
    PackArgs p{};
    p.dim = a.dim;
    p.kp = L.kp;
    p.per_block = up(1024, L.kp / 8) / (L.kp / 8);  // about four 16-byte chunks a thread
    p.x = a.x;
    p.w = a.w;
    p.xs = a.x_stride;
    p.ws = a.w_stride;
    p.xp = (bf16*)(ws + L.xp);
    p.wp = (bf16*)(ws + L.wp);
    p.x_part = L.np * L.kp;
    p.w_part = (int64_t)a.vocab * L.kp;
    p.x_blocks = (int)((L.np + p.per_block - 1) / p.per_block);
    pk.pw = p.w_part;
    if (PARTS == 1 && (uintptr_t)a.w % 16 == 0 && a.w_stride % 8 == 0 && a.dim == L.kp && a.w_stride <= 1 << 20) {
        pk.w = (const bf16*)a.w;  // the products read w where it is
        pk.ldw = a.w_stride;
    } else {
        p.w_rows = a.vocab;
        pk.w = p.wp;
        pk.ldw = L.kp;
    }
    const unsigned blocks = p.x_blocks + (unsigned)((p.w_rows + p.per_block - 1) / p.per_block);
    if (a.n <= PROWS) {
        k_pack<T, PARTS, true><<<blocks, PT, 0, s>>>(r, p);
        return hipGetLastError();
    }
    list_rows(r, L, ws, s);
    k_pack<T, PARTS, false><<<blocks, PT, 0, s>>>(r, p);
    return hipGetLastError();
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

template <class T, int VT, bool FORWARD>
void flat_logits(const FlatArgs& f, Side side, int64_t tiles, hipStream_t s) {
    if (side == LABELS) {
        launch_ranges(tiles, [&](unsigned blocks, BlockRange range) {
            k_few_labels<T, VT, FORWARD><<<blocks, FT, 0, s>>>(f, range);
        });
    } else {  // whose blocks walk over the tiles
        const int64_t most = FORWARD ? ROW_BLOCKS : MOST_BLOCKS;
        k_few_rows<T, VT, FORWARD><<<(unsigned)(tiles < most ? tiles : most), FT, 0, s>>>(f);
    }
}

template <class T, bool FORWARD>
void flat_logits(const FlatArgs& f, Side side, int64_t few, int64_t tiles, hipStream_t s) {
    if constexpr (sizeof(T) == 4) {
        if (few > 32) return flat_logits<T, 2, FORWARD>(f, side, tiles, s);
    }
    flat_logits<T, 1, FORWARD>(f, side, tiles, s);
}

template <class T>
hipError_t flat_loss(const LabelLossArgs& a, const LossPlan& L, char* ws, bool forward, hipStream_t s) {
    const bool few_labels = L.shorter == LABELS;
    const int64_t few = few_labels ? a.vocab : a.n, rows = few_labels ? a.n : a.vocab;
    FlatArgs f{};
    f.n = a.n;
    f.dim = a.dim;
    f.vocab = a.vocab;
    f.x = a.x;
    f.w = a.w;
    f.xs = a.x_stride;
    f.ws = a.w_stride;
    f.labels = label_arrays(a, L, ws, forward);
    f.count_out = a.count;
    f.mean = a.mean;
    f.block_sum = (double*)(ws + L.block_sum);
    f.part = (float2*)(ws + L.part);
    f.target = (float*)(ws + L.target);
    f.lse = a.lse;
    f.dmean = a.dmean;
    f.dloss = a.dloss;
    f.g = (float*)(ws + L.g);
    f.ldg = few_bucket(few);
    if (few_labels) list_rows(f.labels, L, ws, s);
    const int64_t tiles = rows > 0 ? (rows + FR - 1) / FR : 1;
    if (forward) {
        flat_logits<T, true>(f, L.shorter, few, tiles, s);
        if (!few_labels)
            k_lse_join<<<1, JT, 0, s>>>({0, 1}, (int)(tiles < ROW_BLOCKS ? tiles : ROW_BLOCKS), SHORT, f.part, f.target,
                                        f.labels.rows, f.labels.count, nullptr, true, false, a.loss, a.lse, f.block_sum,
                                        f.labels.done, a.mean, a.count);
        return hipGetLastError();
    }
    flat_logits<T, false>(f, L.shorter, few, tiles, s);
    FlatGrads g{};
    g.rows = rows;
    g.dim = a.dim;
    g.kp = L.kp;
    g.g = f.g;
    g.ldg = f.ldg;
    g.chunk = up((rows + L.flat_chunks - 1) / L.flat_chunks, FR);
    void* dshort = few_labels ? a.dw : a.dx;
    g.dshort = dshort ? (float*)(ws + L.dwp) : nullptr;
    g.out_rows = (int)few;
    if (few_labels) {
        g.place = f.labels.place;
        g.lp = a.x;
        g.ls = a.x_stride;
        g.sp = a.w;
        g.ss = a.w_stride;
        g.short_rows = a.vocab;
        g.dlong = a.dx;
        g.dls = a.dx_stride;
    } else {
        g.lp = a.w;
        g.ls = a.w_stride;
        g.sp = a.x;
        g.ss = a.x_stride;
        g.list = f.labels.rows;
        g.count = f.labels.count;
        g.dlong = a.dw;
        g.dls = a.dw_stride;
    }
    const dim3 grid(L.flat_chunks, L.flat_slabs);
    if (g.ldg == 4)
        k_flat_grads<T, 4, 4><<<grid, FT, 0, s>>>(g, L.flat_tr);
    else if (g.ldg == 8)
        k_flat_grads<T, 8, 4><<<grid, FT, 0, s>>>(g, L.flat_tr);
    else if (g.ldg == 16)
        k_flat_grads<T, 16, 2><<<grid, FT, 0, s>>>(g, L.flat_tr);
    else if constexpr (sizeof(T) == 4) {
        if (g.ldg == 32)
            k_flat_products<1><<<grid, FT, 0, s>>>(g);
        else
            k_flat_products<2><<<grid, FT, 0, s>>>(g);
    }
    if (dshort) {
        SplitJoin j{}, none{};
        j.rows = few;
        j.splits = L.flat_chunks;
        j.acc = g.dshort;
        j.pacc = few * L.kp;
        j.place = few_labels ? nullptr : f.labels.place;
        j.out = dshort;
        j.ldout = few_labels ? a.dw_stride : a.dx_stride;
        j.blocks = (int)few;
        if (few > 0) k_join_splits<T><<<j.blocks, 256, 0, s>>>(j, none, a.dim, L.kp, 1);
    }
    return hipGetLastError();
}

template <class T>
hipError_t loss_fwd(const LabelLossArgs& a, char* ws, hipStream_t s) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 3;
    const LossPlan L = loss_plan(a.n, a.dim, a.vocab, PARTS == 1, false);
    if (L.shorter != NEITHER) return flat_loss<T>(a, L, ws, true, s);
    Packed pk{};
    hipError_t e = prepare<T>(a, L, ws, true, pk, s);
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
        set_grid(p, L.tm_z, mv, a.n);
        launch_product<LSE, PARTS, PARTS, T>(L.tm_z, p, s);
        // every tile writes its slabs, so the last may lie beyond the vocabulary (an empty one)
        const int slabs = (int)(up(mv, 64 * L.tm_z) / (32 * L.tm_z));
        launch_ranges(a.n > 0 ? (a.n + JR - 1) / JR : 1, [&](unsigned blocks, BlockRange range) {
            k_lse_join<<<blocks, JT, 0, s>>>(range, slabs, (int)L.np, part, p.target, p.rows, p.count, state, v0 == 0,
                                             v0 + L.piece_f < a.vocab, a.loss, a.lse, bs, (int32_t*)(ws + L.done),
                                             a.mean, a.count);
        });
    }
    return hipGetLastError();
}

template <class T, int DZP>
hipError_t loss_bwd(const LabelLossArgs& a, const LossPlan& L, char* ws, hipStream_t s) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 3;
    Packed pk{};
    hipError_t e = prepare<T>(a, L, ws, false, pk, s);
    if (e != hipSuccess) return e;
    const bool apart = DZP == 1 && a.dw;  // the labels' entries join dw apart (and dx)
    int32_t* slot = (int32_t*)(ws + L.slot);
    const bf16* xp = (const bf16*)(ws + L.xp);
    bf16* dz = (bf16*)(ws + L.dz);
    float *dxp = (float*)(ws + L.dxp), *dwp = (float*)(ws + L.dwp);
    WeighedRows own{};
    int sorted_at = 0;
    if (apart) {
        own.src = xp;
        own.place = (const int32_t*)(ws + L.place);
        own.weight = (const float*)(ws + L.own);
        own.ld = L.kp;
        own.sums = (float*)(ws + L.own_sums);
        own.slot = slot;
        e = launch_rows_by_index(a.n, a.vocab, a.labels, a.wide_labels, L.kp, slot, ws + L.by_label, &sorted_at, s);
        if (e != hipSuccess) return e;
    }
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
        p.own = (float*)(ws + L.own);
        set_grid(p, L.tm_z, mv, a.n);
        launch_product<DZ, PARTS, DZP, T>(L.tm_z, p, s);
        if (apart) {
            own.first = (uint32_t)v0;
            own.last = (uint32_t)(v0 + mv);
            e = launch_weighed_rows(a.n, a.vocab, sorted_at, own, ws + L.by_label, s);
            if (e != hipSuccess) return e;
        }
        const bool last = v0 + L.piece_b >= a.vocab;
        Product qx = product_base<T>(a, L, ws), qw = qx;
        SplitJoin jx{}, jw{};
        if (a.dx) {
            qx.a = p.a;
            qx.lda = pk.ldw;
            qx.pa = pk.pw;
            qx.b = dz;
            qx.ldb = L.piece_b;
            qx.pb = p.pdz;
            qx.m = L.kp;
            qx.k = (int)mv;
            qx.splits = L.split_dx;
            qx.acc = dxp;
            qx.ldacc = L.kp;
            qx.pacc = L.np * L.kp;
            qx.add = v0 > 0;
            set_grid(qx, L.tm_d, L.kp, a.n);
            if (last) {
                jx.rows = a.n;
                jx.splits = L.split_dx;
                jx.acc = dxp;
                jx.pacc = qx.pacc;
                jx.place = (const int32_t*)(ws + L.place);
                jx.out = a.dx;
                jx.ldout = a.dx_stride;
                if (DZP == 1) {
                    jx.own = p.own;
                    jx.labels = a.labels;
                    jx.wide = a.wide_labels;
                    jx.vocab = a.vocab;
                    jx.w = a.w;
                    jx.ws = a.w_stride;
                }
            }
        }
        if (a.dw) {
            qw.a = xp;
            qw.lda = L.kp;
            qw.pa = L.np * L.kp;
            qw.b = dz;
            qw.ldb = L.piece_b;
            qw.pb = p.pdz;
            qw.m = L.kp;
            qw.n = (int)mv;
            qw.splits = L.split_dw;
            set_grid(qw, L.tm_d, L.kp, mv);
            T* out = (T*)a.dw + v0 * a.dw_stride;
            if (L.split_dw > 1) {
                qw.acc = dwp;
                qw.ldacc = L.kp;
                qw.pacc = L.piece_b * L.kp;
                jw.rows = mv;
                jw.splits = L.split_dw;
                jw.acc = dwp;
                jw.pacc = qw.pacc;
                jw.out = out;
                jw.ldout = a.dw_stride;
                if (apart) {
                    jw.slot = slot + v0;
                    jw.own_sums = own.sums;
                }
            } else {
                qw.out = out;
                qw.ldout = a.dw_stride;
                qw.out_dim = a.dim;
                qw.out_wide = (uintptr_t)a.dw % (4 * sizeof(T)) == 0 && a.dw_stride % 4 == 0;
                if (apart) {
                    qw.slot = slot + v0;
                    qw.own_sums = own.sums;
                    qw.ldacc = L.kp;
                }
            }
        }
        if (a.dx && a.dw)
            launch_pair<PARTS, DZP, T>(L.tm_d, qx, qw, s);
        else if (a.dx)
            launch_product<DX, PARTS, DZP, T>(L.tm_d, qx, s);
        else
            launch_product<DW, PARTS, DZP, T>(L.tm_d, qw, s);
        const int per = (a.dim + 3) / 4, per_block = (1024 + per - 1) / per;
        jx.blocks = (int)((jx.rows + per_block - 1) / per_block);
        jw.blocks = (int)((jw.rows + per_block - 1) / per_block);
        if (jx.blocks + jw.blocks > 0)
            k_join_splits<T><<<jx.blocks + jw.blocks, 256, 0, s>>>(jx, jw, a.dim, L.kp, per_block);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
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
    const LossPlan L = loss_plan(a.n, a.dim, a.vocab, a.half, true);
    if (L.shorter != NEITHER)
        return a.half ? flat_loss<bf16>(a, L, ws, false, stream) : flat_loss<float>(a, L, ws, false, stream);
    return !a.half      ? loss_bwd<float, 3>(a, L, ws, stream)
           : L.dzp == 2 ? loss_bwd<bf16, 2>(a, L, ws, stream)
                        : loss_bwd<bf16, 1>(a, L, ws, stream);
}

}  // namespace gs
