// The global norm of many gradient tensors and its clipping, for gfx950.
//
//   norm = sqrt(sum over all tensors of g^2),  out = g * min(1, max_norm / (norm + 1e-6))
//
// Memory-bound: the gradients are read twice (the coefficient depends on all of them) and the
// outputs written once.  The tensors are cut into chunks of kChunk elements, which the workgroups
// take in turn; the tensors' addresses travel in the kernel's arguments, so nothing is copied to the
// device first.  The first kernel leaves one sum of squares per workgroup, in fp64 (a square of an
// fp32 gradient need not fit fp32's range); in the second every workgroup adds those up in the same
// fixed order, which costs less than a launch between the two.  The second goes through the chunks
// backwards: what the first read last is what the caches still hold.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ops_device.h"
#include "ops_internal.h"

namespace tefp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                          // eight-element vectors per thread and chunk
constexpr int64_t kChunk = kThreads * kVecs * 8;  // elements

// The last tensor whose first chunk is at or before `chunk`.
__device__ __forceinline__ int tensor_of(const ClipBatch& b, int64_t chunk)
{
    int lo = 0, hi = b.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b.first[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Calls f(vector, element offset, valid elements) for the thread's vectors of the chunk, after all
// of them have been loaded.
template <class T, class F>
__device__ __forceinline__ void each_vector(const ClipTensor& t, int64_t first, F f)
{
    const auto* g = static_cast<const typename T::store_t*>(t.grad);
    Raw8<T> r[kVecs];
    const int64_t left = t.n - first;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int at = (i * kThreads + (int)threadIdx.x) * 8;
        r[i] = zero8<T>();
        if (at + 8 <= left) r[i] = load8(g + first + at);
        else if (at < left) r[i] = load_few(g + first + at, (int)(left - at));
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int at = (i * kThreads + (int)threadIdx.x) * 8;
        float v[8];
        unpack8(r[i], v);
        const int64_t n = left - at;
        f(v, first + at, n < 0 ? 0 : n > 8 ? 8 : (int)n);
    }
}

// Sum over the workgroup, in every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double red[kThreads / 64];
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) s += red[i];
    return s;
}

__global__ __launch_bounds__(kThreads) void grad_sumsq_kernel(const ClipBatch b, double* __restrict__ partial)
{
    double s = 0.0;
    auto add = [&](const float (&v)[8], int64_t, int) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s += (double)v[j] * (double)v[j];
    };
    for (int64_t c = blockIdx.x; c < b.chunks; c += gridDim.x) {
        const int i = tensor_of(b, c);
        const int64_t first = (c - b.first[i]) * kChunk;
        if (b.types[i] & 1) each_vector<Bf16>(b.t[i], first, add);
        else each_vector<F32>(b.t[i], first, add);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

template <class G, class O>
__device__ __forceinline__ void scale_chunk(const ClipTensor& t, int64_t first, float coef)
{
    auto* out = static_cast<typename O::store_t*>(t.out);
    each_vector<G>(t, first, [&](const float (&v)[8], int64_t at, int n) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = v[j] * coef;
        const Raw8<O> r = pack8(O{}, y);
        if (n == 8) store8(out + at, r);
        else if (n > 0) store_few(out + at, r, n);
    });
}

__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const ClipBatch b, const double* __restrict__ partial,
                                                              int64_t slots, float max_norm, float* __restrict__ norm_out)
{
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < slots; i += kThreads) s += partial[i];
    const float norm = (float)sqrt(block_sum(s));
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    float coef = max_norm / (norm + 1e-6f);
    coef = coef > 1.0f ? 1.0f : coef;   // (NaN stays)
    for (int64_t c = b.chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        const int i = tensor_of(b, c);
        const ClipTensor& t = b.t[i];
        if (!t.out || (t.out == t.grad && coef == 1.0f)) continue;   // nothing to write, or nothing changes
        const int64_t first = (c - b.first[i]) * kChunk;
        switch (b.types[i]) {
        case 0: scale_chunk<F32, F32>(t, first, coef); break;
        case 1: scale_chunk<Bf16, F32>(t, first, coef); break;
        case 2: scale_chunk<F32, Bf16>(t, first, coef); break;
        default: scale_chunk<Bf16, Bf16>(t, first, coef); break;
        }
    }
}

}  // namespace

int64_t clip_blocks(const ClipBatch& b) { return std::max<int64_t>(1, std::min<int64_t>(b.chunks, kClipBlocks)); }

int64_t clip_chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }

int64_t clip_workspace_bytes(int64_t tensors)
{
    return std::max<int64_t>(1, (tensors + kClipBatch - 1) / kClipBatch) * kClipBlocks * (int64_t)sizeof(double);
}

hipError_t launch_grad_sumsq(const ClipBatch& b, double* partial, hipStream_t stream)
{
    grad_sumsq_kernel<<<(unsigned)clip_blocks(b), kThreads, 0, stream>>>(b, partial);
    return hipGetLastError();
}

hipError_t launch_grad_scale(const ClipBatch& b, const double* partial, int64_t slots, float max_norm, float* norm,
                             hipStream_t stream)
{
    grad_scale_kernel<<<(unsigned)clip_blocks(b), kThreads, 0, stream>>>(b, partial, slots, max_norm, norm);
    return hipGetLastError();
}

}  // namespace tefp8
