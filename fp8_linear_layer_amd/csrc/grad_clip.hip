// The global norm of many gradient tensors and its clipping, for gfx950.
//
//   norm = sqrt(sum over all tensors of g^2),  out = g * min(1, max_norm / (norm + 1e-6))
//
// Memory-bound: the gradients are read twice (the coefficient depends on all of them) and the
// outputs written once.  The tensors are cut into chunks of kChunk elements, which the workgroups
// take in turn; the tensors' addresses travel in the kernel's arguments, so nothing is copied to the
// device first; one launch takes kClipBatch of them.  The first kernel leaves one sum of squares per
// workgroup, in fp64 (a square of an fp32 gradient need not fit fp32's range); later launches add to the
// sums of the earlier ones' workgroups, so that there are never more than kClipBlocks.  In the second kernel
// every workgroup adds those up in the same fixed order, which costs less than a launch between the two.  The
// second goes through the launches and their chunks backwards: what the first read last is what the caches still
// hold (with gradients many times their size the order makes no difference).
//
// Measured with 470 million fp32 gradients into bf16: 270 us (7.0 TB/s) and 508 us (5.5 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ops_device.h"
#include "ops_internal.h"

namespace tefp8 {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kChunk = 8192;   // elements
// A thread loads sixteen bytes at a time, so that a wave's load is one run of 1 KiB: four fp32 or eight bf16
// elements, eight or four such units per chunk.
template <class T> constexpr int kUnit = 16 / sizeof(typename T::store_t);
template <class T> constexpr int kUnits = (int)(kChunk / kThreads / kUnit<T>);

// Which tensor a chunk belongs to: the last whose first chunk is at or before it.  Every lane holds the first
// chunks of two tensors, so a look-up is two votes; a binary search through the arguments waits for
// memory at each of its steps.
struct Tensors {
    int32_t lo, hi;
    __device__ __forceinline__ explicit Tensors(const ClipBatch& b)
    {
        static_assert(kClipBatch <= 128, "two tensors per lane");
        const int lane = threadIdx.x & 63;
        lo = lane < b.n ? b.first[lane] : INT32_MAX;
        hi = 64 + lane < b.n ? b.first[64 + lane < kClipBatch ? 64 + lane : 0] : INT32_MAX;
    }
    __device__ __forceinline__ int of(int32_t chunk) const
    {
        const int i = __popcll(__ballot(lo <= chunk)) + __popcll(__ballot(hi <= chunk)) - 1;
        return __builtin_amdgcn_readfirstlane(i);
    }
};

// What is far larger than the last cache is read and written past it (kStream): 470 million fp32 gradients
// take 270 us instead of 335 in the first pass so.
template <bool kStream>
__device__ __forceinline__ u32x4_t load16(const u32x4_a2* p)
{
    if constexpr (kStream) return __builtin_nontemporal_load(p);
    else return *p;
}
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
template <bool kStream>
__device__ __forceinline__ void store16(u32x4_a2* p, const u32x4_t& v)
{
    if constexpr (kStream) __builtin_nontemporal_store(v, p);
    else *p = v;
}
template <bool kStream>
__device__ __forceinline__ void store8b(u32x2_a2* p, const u32x2_t& v)
{
    if constexpr (kStream) __builtin_nontemporal_store(v, p);
    else *p = v;
}

__device__ __forceinline__ void unpack(Bf16, const u32x4_t& r, float (&v)[8]) { unpack8(Raw8<Bf16>{r}, v); }
__device__ __forceinline__ void unpack(F32, const u32x4_t& r, float (&v)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = as_float(r[i]);
}

// Calls f(values, first element, how many of them) for the thread's units of the chunk, after all of
// them have been loaded; values past the tensor's end are zeros.
template <class T, bool kStream, class F>
__device__ __forceinline__ void each_unit(const ClipTensor& t, int64_t first, F f)
{
    constexpr int kN = kUnit<T>;
    const auto* g = static_cast<const typename T::store_t*>(t.grad) + first;
    const int64_t left = t.n - first;
    u32x4_t r[kUnits<T>];
    if (left >= kChunk) {
#pragma unroll
        for (int i = 0; i < kUnits<T>; ++i)
            r[i] = load16<kStream>(reinterpret_cast<const u32x4_a2*>(g + (i * kThreads + (int)threadIdx.x) * kN));
    } else {
#pragma unroll
        for (int i = 0; i < kUnits<T>; ++i) {
            const int at = (i * kThreads + (int)threadIdx.x) * kN;
            r[i] = u32x4_t{0, 0, 0, 0};
            if (at + kN <= left) r[i] = load16<false>(reinterpret_cast<const u32x4_a2*>(g + at));
            else if (at < left) r[i] = load_few(g + at, (int)(left - at)).a;
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits<T>; ++i) {
        const int at = (i * kThreads + (int)threadIdx.x) * kN;
        float v[kN];
        unpack(T{}, r[i], v);
        f(v, first + at, left >= kChunk ? kN : (int)(min(left, kChunk) - at));
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

// `have` sums are there from earlier launches.
template <bool kStream>
__global__ __launch_bounds__(kThreads) void grad_sumsq_kernel(const ClipBatch b, double* __restrict__ partial, int have)
{
    double s = 0.0;
    auto add = [&](const auto& v, int64_t, int) {
#pragma unroll
        for (float x : v) s += (double)x * (double)x;
    };
    const Tensors tensors(b);
    for (int32_t c = blockIdx.x; c < b.chunks; c += gridDim.x) {
        const int i = tensors.of(c);
        const int64_t first = (int64_t)(c - b.first[i]) * kChunk;
        if (b.types[i] & 1) each_unit<Bf16, kStream>(b.t[i], first, add);
        else each_unit<F32, kStream>(b.t[i], first, add);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) partial[blockIdx.x] = (int)blockIdx.x < have ? partial[blockIdx.x] + s : s;
}

template <class G, class O, bool kStream>
__device__ __forceinline__ void scale_chunk(const ClipTensor& t, int64_t first, float coef)
{
    constexpr int kN = kUnit<G>;
    auto* out = static_cast<typename O::store_t*>(t.out);
    each_unit<G, kStream>(t, first, [&](const float (&v)[kN], int64_t at, int n) {
        float y[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) y[j] = v[j] * coef;
        if (n >= kN) {
#pragma unroll
            for (int j = 0; j < kN; j += 4) {
                if constexpr (__is_same(O, F32))
                    store16<kStream>(reinterpret_cast<u32x4_a2*>(out + at + j),
                                     u32x4_t{as_bits(y[j]), as_bits(y[j + 1]), as_bits(y[j + 2]), as_bits(y[j + 3])});
                else if constexpr (kN == 4)
                    store8b<kStream>(reinterpret_cast<u32x2_a2*>(out + at), u32x2_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])});
                else if (j == 0)
                    store16<kStream>(reinterpret_cast<u32x4_a2*>(out + at), pack8(Bf16{}, y).a);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kN - 1; ++j) {
                if (j >= n) continue;
                if constexpr (__is_same(O, F32)) out[at + j] = y[j];
                else out[at + j] = (uint16_t)pack_bf16(y[j], 0.0f);
            }
        }
    });
}

template <bool kStream>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const ClipBatch b, const double* __restrict__ partial,
                                                              int64_t slots, float max_norm, float* __restrict__ norm_out)
{
    const Tensors tensors(b);
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < slots; i += kThreads) s += partial[i];
    const float norm = (float)sqrt(block_sum(s));
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    float coef = max_norm / (norm + 1e-6f);
    coef = coef > 1.0f ? 1.0f : coef;   // (NaN stays)
    for (int32_t c = b.chunks - 1 - (int32_t)blockIdx.x; c >= 0; c -= gridDim.x) {
        const int i = tensors.of(c);
        const ClipTensor& t = b.t[i];
        if (!t.out || (t.out == t.grad && coef == 1.0f)) continue;   // nothing to write, or nothing changes
        const int64_t first = (int64_t)(c - b.first[i]) * kChunk;
        switch (b.types[i]) {
        case 0: scale_chunk<F32, F32, kStream>(t, first, coef); break;
        case 1: scale_chunk<Bf16, F32, kStream>(t, first, coef); break;
        case 2: scale_chunk<F32, Bf16, kStream>(t, first, coef); break;
        default: scale_chunk<Bf16, Bf16, kStream>(t, first, coef); break;
        }
    }
}

}  // namespace

int64_t clip_blocks(const ClipBatch& b) { return std::max(1, std::min(b.chunks, kClipBlocks)); }

int64_t clip_chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }

int64_t clip_workspace_bytes() { return kClipBlocks * (int64_t)sizeof(double); }

hipError_t launch_grad_sumsq(const ClipBatch& b, double* partial, int64_t have, bool past, hipStream_t stream)
{
    const unsigned grid = (unsigned)clip_blocks(b);
    if (past) grad_sumsq_kernel<true><<<grid, kThreads, 0, stream>>>(b, partial, (int)have);
    else grad_sumsq_kernel<false><<<grid, kThreads, 0, stream>>>(b, partial, (int)have);
    return hipGetLastError();
}

hipError_t launch_grad_scale(const ClipBatch& b, const double* partial, int64_t slots, float max_norm, float* norm,
                             bool past, hipStream_t stream)
{
    const unsigned grid = (unsigned)clip_blocks(b);
    if (past) grad_scale_kernel<true><<<grid, kThreads, 0, stream>>>(b, partial, slots, max_norm, norm);
    else grad_scale_kernel<false><<<grid, kThreads, 0, stream>>>(b, partial, slots, max_norm, norm);
    return hipGetLastError();
}

}  // namespace tefp8
