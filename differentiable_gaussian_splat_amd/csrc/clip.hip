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
// the caches.
#include "elem.hpp"
#include "launch.hpp"

namespace gs {

namespace {

constexpr int CB = 256;                // threads per block
constexpr int CHUNK_BYTES = 32768;     // of one tensor
constexpr int CLIP_BLOCKS = 1024;      // at most; a partial sum each
constexpr int TABLE = 96;              // tensors in a launch's arguments

struct ClipTensor {
    const void* g;
    void* out;        // null: norm only
    int64_t n;        // elements; bfloat16: ~elements
    int64_t first;    // its first chunk
};

// The tensors by value (in the launch's arguments) if they fit, otherwise in memory.
struct ClipTable {
    ClipTensor t[TABLE];
};

template <class T>
constexpr int CHUNK = CHUNK_BYTES / (int)sizeof(T);

// The tensor that holds chunk c.
__device__ __forceinline__ int tensor_of(const ClipTensor* t, int count, int64_t c) {
    int lo = 0, hi = count;  // t[lo].first <= c < t[hi].first
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t[mid].first <= c)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
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

template <class T>
__device__ __forceinline__ double chunk_squares(const T* g, int64_t left) {
    constexpr int V = WIDE<T>, STEPS = CHUNK<T> / (CB * V);
    double s0 = 0., s1 = 0.;
    if (left >= CHUNK<T>) {
        wide_t<T> raw[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            raw[i] = *reinterpret_cast<const wide_any<T>*>(g + (i * CB + threadIdx.x) * V);
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
            for (int k = 0; k < V; k += 2) {
                const double a = (double)(float)raw[i][k], b = (double)(float)raw[i][k + 1];
                s0 = fma(a, a, s0);
                s1 = fma(b, b, s1);
            }
    } else {
        for (int i = threadIdx.x * V; i < left; i += CB * V) {
            if (i + V <= left) {
                const wide_t<T> r = *reinterpret_cast<const wide_any<T>*>(g + i);
#pragma unroll
                for (int k = 0; k < V; ++k) s0 = fma((double)(float)r[k], (double)(float)r[k], s0);
            } else {
                for (int k = i; k < left; ++k) s1 = fma((double)(float)g[k], (double)(float)g[k], s1);
            }
        }
    }
    return s0 + s1;
}

template <class T>
__device__ __forceinline__ void chunk_scale(const T* g, T* o, int64_t left, float c) {
    constexpr int V = WIDE<T>, STEPS = CHUNK<T> / (CB * V);
    if (left >= CHUNK<T>) {
        wide_t<T> raw[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            raw[i] = *reinterpret_cast<const wide_any<T>*>(g + (i * CB + threadIdx.x) * V);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
#pragma unroll
            for (int k = 0; k < V; ++k) raw[i][k] = (T)((float)raw[i][k] * c);
            *reinterpret_cast<wide_any<T>*>(o + (i * CB + threadIdx.x) * V) = raw[i];
        }
    } else {
        for (int i = threadIdx.x * V; i < left; i += CB * V) {
            if (i + V <= left) {
                wide_t<T> r = *reinterpret_cast<const wide_any<T>*>(g + i);
#pragma unroll
                for (int k = 0; k < V; ++k) r[k] = (T)((float)r[k] * c);
                *reinterpret_cast<wide_any<T>*>(o + i) = r;
            } else {
                for (int k = i; k < left; ++k) o[k] = (T)((float)g[k] * c);
            }
        }
    }
}

// A block's run of chunks: as many for each block, one more for the first ones.
__device__ __forceinline__ void block_chunks(int64_t chunks, int64_t& first, int64_t& end) {
    const int64_t b = blockIdx.x, each = chunks / gridDim.x, more = chunks % gridDim.x;
    first = b * each + (b < more ? b : more);
    end = first + each + (b < more ? 1 : 0);
}

__device__ __forceinline__ void clip_norm(const ClipTensor* t, int count, int64_t chunks, double* part) {
    __shared__ double s[CB / 64];
    int64_t first, end;
    block_chunks(chunks, first, end);
    double sum = 0.;
    int k = first < end ? tensor_of(t, count, first) : 0;
    for (int64_t c = first; c < end; ++c) {
        while (k + 1 < count && t[k + 1].first <= c) ++k;
        const ClipTensor e = t[k];
        if (e.n < 0) {
            const int64_t at = (c - e.first) * CHUNK<bf16>;
            sum += chunk_squares((const bf16*)e.g + at, ~e.n - at);
        } else {
            const int64_t at = (c - e.first) * CHUNK<float>;
            sum += chunk_squares((const float*)e.g + at, e.n - at);
        }
    }
    sum = block_sum(sum, s);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// parts: how many sums the first launch left. scale: whether the tensors are wanted, beside the norm.
__device__ __forceinline__ void clip_scale(const ClipTensor* t, int count, int64_t chunks, const double* part,
                                           int parts, float max_norm, float* norm, bool scale) {
    __shared__ double s[CB / 64];
    double sum = 0.;
    for (int i = threadIdx.x; i < parts; i += CB) sum += part[i];
    const double whole = sqrt(block_sum(sum, s));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)whole;
    if (!scale) return;
    const double f = (double)max_norm / (whole + 1e-6);
    const float c = f >= 1. || max_norm == INFINITY ? 1.f : (float)f;  // no number where the norm is none
    int64_t first, end;
    block_chunks(chunks, first, end);
    int k = first < end ? tensor_of(t, count, end - 1) : 0;
    for (int64_t j = end - 1; j >= first; --j) {
        while (t[k].first > j) --k;
        const ClipTensor e = t[k];
        if (c == 1.f && e.g == e.out) continue;  // in place, and nothing to change
        if (e.n < 0) {
            const int64_t at = (j - e.first) * CHUNK<bf16>;
            chunk_scale((const bf16*)e.g + at, (bf16*)e.out + at, ~e.n - at, c);
        } else {
            const int64_t at = (j - e.first) * CHUNK<float>;
            chunk_scale((const float*)e.g + at, (float*)e.out + at, e.n - at, c);
        }
    }
}

__global__ __launch_bounds__(CB) void k_clip_norm(ClipTable t, int count, int64_t chunks, double* part) {
    clip_norm(t.t, count, chunks, part);
}

__global__ __launch_bounds__(CB) void k_clip_norm_many(const ClipTensor* __restrict__ t, int count, int64_t chunks,
                                                       double* part) {
    clip_norm(t, count, chunks, part);
}

__global__ __launch_bounds__(CB) void k_clip_scale(ClipTable t, int count, int64_t chunks, const double* part,
                                                   int parts, float max_norm, float* norm, bool scale) {
    clip_scale(t.t, count, chunks, part, parts, max_norm, norm, scale);
}

__global__ __launch_bounds__(CB) void k_clip_scale_many(const ClipTensor* __restrict__ t, int count, int64_t chunks,
                                                        const double* part, int parts, float max_norm, float* norm,
                                                        bool scale) {
    clip_scale(t, count, chunks, part, parts, max_norm, norm, scale);
}

__global__ __launch_bounds__(128) void k_clip_table(ClipTable t, int count, ClipTensor* __restrict__ to) {
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
    int64_t chunks = 0;
    int count = 0, held = 0;
    int full = 0;
    for (int i = 0; i < tensors; ++i) full += numels[i] > 0;
    const bool many = full > TABLE;
    for (int i = 0; i < tensors; ++i) {
        if (numels[i] == 0) continue;
        ClipTensor& e = t.t[held++];
        e.g = grads[i];
        e.out = outs ? outs[i] : nullptr;
        e.n = half[i] ? ~numels[i] : numels[i];
        e.first = chunks;
        const int64_t per = half[i] ? CHUNK<bf16> : CHUNK<float>;
        chunks += (numels[i] + per - 1) / per;
        if (many && (held == TABLE || count + held == full)) {
            k_clip_table<<<1, 128, 0, stream>>>(t, held, table + count);
            if (hipError_t e2 = hipGetLastError()) return e2;
            count += held;
            held = 0;
        }
    }
    if (!many) count = held;
    const int blocks = (int)(chunks < CLIP_BLOCKS ? chunks : CLIP_BLOCKS);
    if (blocks > 0) {
        if (many)
            k_clip_norm_many<<<blocks, CB, 0, stream>>>(table, count, chunks, part);
        else
            k_clip_norm<<<blocks, CB, 0, stream>>>(t, count, chunks, part);
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
