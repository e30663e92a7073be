// Clipping of gradients by their global norm.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   c = min(1, max_norm / (norm + 1e-6)),  out = c g
//
// Two launches over chunks of all tensors: the first leaves a sum of squares
// per block, the second has every block add those sums again (in one order, so
// that all agree bit for bit) and scale its chunks. Squares and their sums are
// float64: the square of a float32 is exact there, nothing overflows or
// underflows, and the conversion costs no time beside the loads.
// Bound by memory: read, read again and write. A block scales its chunks in the
// reverse of the order in which it read them, so that the last ones come from
// the caches. 59M float32 in five tensors 142 us (3 x 236 MB: 5.0 TB/s, a large copy
// has 4.8); chunks of 16 or 64 KB and up to 4096 blocks are within 3 % of it. 300
// bfloat16 tensors of 40M elements 57 us, 45 of it the two launches; two others put
// the tensors' table in memory, 160 of them to a launch's arguments. Small calls are
// one launch of one block: 1000 elements 4.6 us, by two launches 7.9.
#include "elem.hpp"
#include "launch.hpp"

namespace gs {

namespace {

constexpr int CB = 256;                // threads per block
constexpr int CHUNK_BYTES = 32768;     // of one tensor
constexpr int CLIP_BLOCKS = 1024;      // at most; a partial sum each
constexpr int TABLE = 160;             // tensors in a launch's arguments, which hold 4 KB

struct ClipTensor {
    const void* g;
    void* out;        // null: norm only
    uint32_t first;   // its first chunk
    uint32_t last;    // elements of its last chunk, and HALF for bfloat16
};
constexpr uint32_t HALF = 0x80000000u;

// The tensors by value (in the launch's arguments) if they fit, otherwise in memory.
struct ClipTable {
    ClipTensor t[TABLE];
};

template <class T>
constexpr int CHUNK = CHUNK_BYTES / (int)sizeof(T);

// The tensor that holds chunk c: how many begin at or before it, counted by the wave's lanes together (a search by
// halves waits for one load after another).
__device__ __forceinline__ int tensor_of(const ClipTensor* t, int count, uint32_t c) {
    int k = -1;
    for (int i = 0; i < count; i += 64) {
        const int at = i + (threadIdx.x & 63);
        k += __popcll(__ballot(at < count && t[at].first <= c));
    }
    return __builtin_amdgcn_readfirstlane(k);
}

__device__ __forceinline__ double block_sum(double v, double* s) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
    __syncthreads();  // earlier readers of s are done
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.;
#pragma unroll
    for (int k = 0; k < CB / 64; ++k) v += s[k];
    return v;
}

// A thread's accesses of a chunk of `left` elements, all under way together; those past its end are zeros.
template <class T>
constexpr int STEPS = CHUNK<T> / (CB * WIDE<T>);
template <bool FULL, class T>
__device__ __forceinline__ void load_chunk(const T* g, int left, wide_t<T> (&raw)[STEPS<T>]) {
#pragma unroll
    for (int i = 0; i < STEPS<T>; ++i) {
        const int at = (i * CB + (int)threadIdx.x) * WIDE<T>;
        raw[i] = (T)0.f;
        if (FULL || at + WIDE<T> <= left) raw[i] = *reinterpret_cast<const wide_any<T>*>(g + at);
    }
}

// This thread's element of those behind a chunk's last whole access, or -1.
template <class T>
__device__ __forceinline__ int behind(int left) {
    const int at = left / WIDE<T> * WIDE<T> + (int)threadIdx.x;
    return at < left ? at : -1;
}

template <bool FULL, class T>
__device__ __forceinline__ double chunk_squares(const T* g, int left) {
    double s0 = 0., s1 = 0.;
    wide_t<T> raw[STEPS<T>];
    load_chunk<FULL>(g, left, raw);
    if (!FULL) {
        const int at = behind<T>(left);
        const double a = at < 0 ? 0. : (double)(float)g[at];
        s0 = a * a;
    }
#pragma unroll
    for (int i = 0; i < STEPS<T>; ++i)
#pragma unroll
        for (int k = 0; k < WIDE<T>; k += 2) {
            const double a = (double)(float)raw[i][k], b = (double)(float)raw[i][k + 1];
            s0 = fma(a, a, s0);
            s1 = fma(b, b, s1);
        }
    return s0 + s1;
}

template <bool FULL, class T>
__device__ __forceinline__ void chunk_scale(const T* g, T* o, int left, float c) {
    wide_t<T> raw[STEPS<T>];
    load_chunk<FULL>(g, left, raw);
    if (!FULL) {
        const int at = behind<T>(left);
        if (at >= 0) o[at] = (T)((float)g[at] * c);
    }
#pragma unroll
    for (int i = 0; i < STEPS<T>; ++i) {
        const int at = (i * CB + (int)threadIdx.x) * WIDE<T>;
#pragma unroll
        for (int k = 0; k < WIDE<T>; ++k) raw[i][k] = (T)((float)raw[i][k] * c);
        if (FULL || at + WIDE<T> <= left) *reinterpret_cast<wide_any<T>*>(o + at) = raw[i];
    }
}

// chunk: of the tensor; last: whether it is the tensor's last.
template <class T>
__device__ __forceinline__ double squares(const ClipTensor& e, uint32_t chunk, bool last) {
    const T* g = (const T*)e.g + (int64_t)chunk * CHUNK<T>;
    const int left = last ? (int)(e.last & ~HALF) : CHUNK<T>;
    return left == CHUNK<T> ? chunk_squares<true>(g, 0) : chunk_squares<false>(g, left);
}

template <class T>
__device__ __forceinline__ void scale(const ClipTensor& e, uint32_t chunk, bool last, float c) {
    const int64_t at = (int64_t)chunk * CHUNK<T>;
    const int left = last ? (int)(e.last & ~HALF) : CHUNK<T>;
    const T* g = (const T*)e.g + at;
    T* o = (T*)e.out + at;
    if (left == CHUNK<T>)
        chunk_scale<true>(g, o, 0, c);
    else
        chunk_scale<false>(g, o, left, c);
}

// What the gradients are multiplied by: no number where the norm is none; 1 whatever the norm where max_norm is
// infinite, which asks for the norm alone.
__device__ __forceinline__ float factor(float max_norm, double norm) {
    const double f = (double)max_norm / (norm + 1e-6);
    return f >= 1. || max_norm == INFINITY ? 1.f : (float)f;
}

// A block's run of chunks: as many for each block, one more for the first ones.
__device__ __forceinline__ void block_chunks(uint32_t chunks, uint32_t& first, uint32_t& end) {
    const uint32_t b = blockIdx.x, each = chunks / gridDim.x, more = chunks % gridDim.x;
    first = b * each + min(b, more);
    end = first + each + (b < more ? 1 : 0);
}

// Where the tensor behind tensor k begins.
__device__ __forceinline__ uint32_t end_of(const ClipTensor* t, int count, int k, uint32_t chunks) {
    return k + 1 < count ? t[k + 1].first : chunks;
}

__device__ __forceinline__ void clip_norm(const ClipTensor* t, int count, uint32_t chunks, double* part) {
    __shared__ double s[CB / 64];
    uint32_t first, end;
    block_chunks(chunks, first, end);
    double sum = 0.;
    int k = first < end ? tensor_of(t, count, first) : 0;
    uint32_t next = end_of(t, count, k, chunks);
    for (uint32_t c = first; c < end; ++c) {
        if (c == next) next = end_of(t, count, ++k, chunks);  // no tensor is without chunks
        const ClipTensor e = t[k];
        const bool last = c + 1 == next;
        sum += e.last & HALF ? squares<bf16>(e, c - e.first, last) : squares<float>(e, c - e.first, last);
    }
    sum = block_sum(sum, s);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// parts: how many sums the first launch left. wanted: whether the tensors are, beside the norm.
__device__ __forceinline__ void clip_scale(const ClipTensor* t, int count, uint32_t chunks, const double* part,
                                           int parts, float max_norm, float* norm, bool wanted) {
    __shared__ double s[CB / 64];
    uint32_t first, end;
    block_chunks(chunks, first, end);
    int k = wanted && first < end ? tensor_of(t, count, end - 1) : 0;
    uint32_t next = end_of(t, count, k, chunks);
    double sum = 0.;
    for (int i = threadIdx.x; i < parts; i += CB) sum += part[i];
    const double whole = sqrt(block_sum(sum, s));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)whole;
    if (!wanted) return;
    const float c = factor(max_norm, whole);
    for (uint32_t j = end; j-- > first;) {
        if (j < t[k].first) next = t[k--].first;
        const ClipTensor e = t[k];
        if (c == 1.f && e.g == e.out) continue;  // in place, and nothing to change
        if (e.last & HALF)
            scale<bf16>(e, j - e.first, j + 1 == next, c);
        else
            scale<float>(e, j - e.first, j + 1 == next, c);
    }
}

__global__ __launch_bounds__(CB) void k_clip_norm(ClipTable t, int count, uint32_t chunks, double* part) {
    clip_norm(t.t, count, chunks, part);
}

__global__ __launch_bounds__(CB) void k_clip_norm_many(const ClipTensor* __restrict__ t, int count, uint32_t chunks,
                                                       double* part) {
    clip_norm(t, count, chunks, part);
}

__global__ __launch_bounds__(CB) void k_clip_scale(ClipTable t, int count, uint32_t chunks, const double* part,
                                                   int parts, float max_norm, float* norm, bool wanted) {
    clip_scale(t.t, count, chunks, part, parts, max_norm, norm, wanted);
}

__global__ __launch_bounds__(CB) void k_clip_scale_many(const ClipTensor* __restrict__ t, int count, uint32_t chunks,
                                                        const double* part, int parts, float max_norm, float* norm,
                                                        bool wanted) {
    clip_scale(t, count, chunks, part, parts, max_norm, norm, wanted);
}

// Small calls in one launch of one block: its waves hold all elements in registers between the sum and the scaling. A
// unit is a wave's 16-byte accesses; t[].first counts units.
constexpr int SMALL_WAVES = 16, SMALL_UNITS = 4;  // units to a wave
constexpr int UNIT_BYTES = 1024;

__global__ __launch_bounds__(64 * SMALL_WAVES) void k_clip_small(ClipTable t, int count, int units, float max_norm,
                                                                 float* norm, bool wanted) {
    __shared__ double s[SMALL_WAVES];
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint32_t first = lane < count ? t.t[lane].first : (uint32_t)units;
    uint32_t raw[SMALL_UNITS][4];
    double sum = 0.;
    // what(element, left from there on, tensor, bfloat16) of this lane in the wave's i-th unit
    auto each = [&](int i, auto what) {
        const uint32_t u = w + i * SMALL_WAVES;
        if (u >= (uint32_t)units) return;
        const int k = __builtin_amdgcn_readfirstlane(__popcll(__ballot(first <= u)) - 1);
        const ClipTensor& e = t.t[k];
        const bool half = e.last & HALF;
        const int whole = UNIT_BYTES / (half ? 2 : 4), in = lane * (half ? 8 : 4);
        const int here = u + 1 == end_of(t.t, count, k, units) ? (int)(e.last & ~HALF) : whole;
        what((int)(u - e.first) * whole + in, here - in, e, half);
    };
#pragma unroll
    for (int i = 0; i < SMALL_UNITS; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[i][j] = 0;
        each(i, [&](int at, int left, const ClipTensor& e, bool half) {
            typedef uint32_t four_any __attribute__((ext_vector_type(4), aligned(2)));
            const char* p = (const char*)e.g + (int64_t)at * (half ? 2 : 4);
            if (left >= (half ? 8 : 4)) {
                const four_any v = *reinterpret_cast<const four_any*>(p);
#pragma unroll
                for (int j = 0; j < 4; ++j) raw[i][j] = v[j];
            } else if (half) {
#pragma unroll
                for (int j = 0; j < 7; ++j)
                    if (j < left) raw[i][j / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[j] << (j % 2 * 16);
            } else {
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (j < left) raw[i][j] = reinterpret_cast<const uint32_t*>(p)[j];
            }
        });
    }
#pragma unroll
    for (int i = 0; i < SMALL_UNITS; ++i)
        each(i, [&](int, int, const ClipTensor&, bool half) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const double a = (double)__uint_as_float(half ? raw[i][j] << 16 : raw[i][j]);
                const double b = half ? (double)__uint_as_float(raw[i][j] & 0xffff0000u) : 0.;
                sum = fma(a, a, fma(b, b, sum));
            }
        });
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    if (lane == 0) s[w] = sum;
    __syncthreads();
    double all = 0.;
#pragma unroll
    for (int k = 0; k < SMALL_WAVES; ++k) all += s[k];
    const double whole = sqrt(all);
    if (threadIdx.x == 0) *norm = (float)whole;
    if (!wanted) return;
    const float c = factor(max_norm, whole);
#pragma unroll
    for (int i = 0; i < SMALL_UNITS; ++i)
        each(i, [&](int at, int left, const ClipTensor& e, bool half) {
            if (left <= 0 || (c == 1.f && e.g == e.out)) return;
            if (half) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = __uint_as_float(j % 2 ? raw[i][j / 2] & 0xffff0000u : raw[i][j / 2] << 16) * c;
                store_row<false>((bf16*)e.out + at, left, v);
            } else {
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(raw[i][j]) * c;
                store_row<false>((float*)e.out + at, left, v);
            }
        });
}

__global__ __launch_bounds__(TABLE) void k_clip_table(ClipTable t, int count, ClipTensor* __restrict__ to) {
    if ((int)threadIdx.x < count) to[threadIdx.x] = t.t[threadIdx.x];
}

}  // namespace

// The partial sums, then the tensors where a launch's arguments do not hold them.
size_t clip_workspace(int64_t tensors) {
    return CLIP_BLOCKS * sizeof(double) + (tensors > TABLE ? (size_t)tensors * sizeof(ClipTensor) : 0);
}

hipError_t launch_clip_grads(int tensors, const void* const* grads, void* const* outs, const int64_t* numels,
                             const int32_t* half, float max_norm, float* norm, char* ws, hipStream_t stream) {
    ClipTable t{};
    double* part = reinterpret_cast<double*>(ws);
    ClipTensor* table = reinterpret_cast<ClipTensor*>(ws + CLIP_BLOCKS * sizeof(double));
    // tensors without elements are left out, so the chunks' tensors follow one another
    int64_t chunks = 0, units = 0;
    int count = 0, held = 0, full = 0;
    for (int i = 0; i < tensors; ++i) {
        full += numels[i] > 0;
        units += (numels[i] * (half[i] ? 2 : 4) + UNIT_BYTES - 1) / UNIT_BYTES;
    }
    const bool many = full > TABLE, small = full <= 64 && units <= SMALL_WAVES * SMALL_UNITS;
    for (int i = 0; i < tensors; ++i) {
        if (numels[i] == 0) continue;
        const int64_t per = (small ? UNIT_BYTES : CHUNK_BYTES) / (half[i] ? 2 : 4), mine = (numels[i] + per - 1) / per;
        ClipTensor& e = t.t[held++];
        e.g = grads[i];
        e.out = outs ? outs[i] : nullptr;
        e.first = (uint32_t)chunks;
        e.last = (uint32_t)(numels[i] - (mine - 1) * per) | (half[i] ? HALF : 0u);
        chunks += mine;
        if (many && (held == TABLE || count + held == full)) {
            k_clip_table<<<1, TABLE, 0, stream>>>(t, held, table + count);
            if (hipError_t e2 = hipGetLastError()) return e2;
            count += held;
            held = 0;
        }
    }
    if (!many) count = held;
    if (small) {
        k_clip_small<<<1, 64 * SMALL_WAVES, 0, stream>>>(t, count, (int)units, max_norm, norm, outs != nullptr);
        return hipGetLastError();
    }
    const int blocks = (int)(chunks < CLIP_BLOCKS ? chunks : CLIP_BLOCKS);
    if (blocks > 0) {
        if (many)
            k_clip_norm_many<<<blocks, CB, 0, stream>>>(table, count, (uint32_t)chunks, part);
        else
            k_clip_norm<<<blocks, CB, 0, stream>>>(t, count, (uint32_t)chunks, part);
        if (hipError_t e = hipGetLastError()) return e;
    }
    const int scale_blocks = outs && blocks > 0 ? blocks : 1;
    if (many)
        k_clip_scale_many<<<scale_blocks, CB, 0, stream>>>(table, count, chunks, part, blocks, max_norm, norm, outs);
    else
        k_clip_scale<<<scale_blocks, CB, 0, stream>>>(t, count, chunks, part, blocks, max_norm, norm, outs);
    return hipGetLastError();
}

}  // namespace gs
