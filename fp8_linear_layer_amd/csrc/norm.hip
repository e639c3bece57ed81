// Root-mean-square norm with the residual's addition, for gfx950.
//
//   v = x + residual, rounded to the residual's type and stored as h (v = x without a residual)
//   rstd = 1 / sqrt(mean over the row of v^2 + eps),  y = (v * rstd) * gamma
//
// y is stored in bf16 or fp32, or as its per-token fp8 cast (1x128 groups, the operand of the next
// GEMM) and / or the cast of its transpose (the weight gradient's operand).
//
// Memory-bound.  A row is read once into registers, a workgroup of 256 threads per row, eight
// consecutive columns (16 bytes of bf16) per thread and step; the row's sum of squares is reduced
// over the wave by lane exchanges and over the waves through LDS, and everything that follows
// works from the registers.  Sixteen consecutive lanes hold one 128-column group, so the fp8 cast
// needs a four-step lane exchange and no LDS.
//
// Rows whose length is no multiple of eight: the last chunk starts at cols - 8 and overlaps its
// neighbour; the columns that the neighbour has too are left out of the sums and written twice
// with the same value.  Every write of a row comes after all its reads (the reduction lies
// between), so h may be the residual's own buffer.
//
// The cast of the transpose has groups of 128 rows and needs the rstd of each of them, so it runs
// as a second kernel over 128 x 128 tiles of the stored h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fp8_codec.h"
#include "ops_device.h"
#include "ops_internal.h"

namespace tefp8 {
namespace {

constexpr int kThreads = 256;

struct NoResidual {};
enum class Out { Bf16, F32, Fp8 };

// Chunk of eight columns whose nominal first column is `col`.
struct Chunk {
    bool on;    // any column inside the row
    int c0;     // first column loaded
    int skip;   // leading columns that belong to the chunk before
};
__device__ __forceinline__ Chunk chunk_at(int col, int cols)
{
    const int c0 = max(min(col, cols - 8), 0);
    return {col < cols, c0, col - c0};
}
template <class T, class P>
__device__ __forceinline__ Raw8<T> load_chunk(const P* row, const Chunk& c, int cols)
{
    if (!c.on) return zero8<T>();
    if (cols < 8) return load_few(row, cols);
    return load8(row + c.c0);
}
template <class P, class R>
__device__ __forceinline__ void store_chunk(P* row, const Chunk& c, int cols, const R& r)
{
    if (!c.on) return;
    if (cols < 8) store_few(row, r, cols);
    else store8(row + c.c0, r);
}

// Sum over the kTPR threads of a row.  `red` has room for the waves of a row.
template <int kTPR>
__device__ __forceinline__ float row_sum(float v, float* red)
{
    v = sum_lanes<64>(v);
    if (kTPR == 64) return v;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kTPR / 64; ++i) s += red[i];
    return s;
}

template <int kFmt, bool kPow2>
__device__ __forceinline__ uint2 cast8(const float (&y)[8], float amax, float& scale)
{
    float mult, s[8];
    group_scale<kFmt, kPow2>(amax, scale, mult);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = y[j] * mult;
    return encode8<kFmt>(s);
}
__device__ __forceinline__ uint2 cast8(int fmt, int pow2, const float (&y)[8], float amax, float& scale)
{
    if (fmt == FMT_E4M3)
        return pow2 ? cast8<FMT_E4M3, true>(y, amax, scale) : cast8<FMT_E4M3, false>(y, amax, scale);
    return pow2 ? cast8<FMT_E5M2, true>(y, amax, scale) : cast8<FMT_E5M2, false>(y, amax, scale);
}

template <class X, class H, Out kOut, int kTPR, int kNV>
__global__ __launch_bounds__(kTPR) void rmsnorm_fwd_kernel(const NormFwdArgs a)
{
    constexpr bool kRes = !__is_same(H, NoResidual);
    __shared__ float red[kTPR / 64];
    const int64_t row = xcd_run(blockIdx.x, gridDim.x);
    const int t = threadIdx.x, cols = a.cols;
    const auto* x = static_cast<const typename X::store_t*>(a.x) + row * a.ld_x;

    Chunk c[kNV];
    Raw8<X> rx[kNV];
    Raw8<Bf16> rg[kNV];
    float v[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        c[i] = chunk_at((i * kTPR + t) * 8, cols);
        rx[i] = load_chunk<X>(x, c[i], cols);
    }
    if constexpr (kRes) {
        const auto* res = static_cast<const typename H::store_t*>(a.res) + row * a.ld_res;
        Raw8<H> rr[kNV];
#pragma unroll
        for (int i = 0; i < kNV; ++i) rr[i] = load_chunk<H>(res, c[i], cols);
#pragma unroll
        for (int i = 0; i < kNV; ++i) rg[i] = load_chunk<Bf16>(a.gamma, c[i], cols);
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            float r[8];
            unpack8(rx[i], v[i]);
            unpack8(rr[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += r[j];
            rr[i] = pack8(H{}, v[i]);   // the stored sum is what the norm is of
            unpack8(rr[i], v[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kNV; ++i) rg[i] = load_chunk<Bf16>(a.gamma, c[i], cols);
#pragma unroll
        for (int i = 0; i < kNV; ++i) unpack8(rx[i], v[i]);
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += j >= c[i].skip ? v[i][j] * v[i][j] : 0.0f;
    ss = row_sum<kTPR>(ss, red);
    const float rstd = 1.0f / sqrtf(ss / (float)cols + a.eps);
    if (t == 0) a.rstd[row] = rstd;

#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        if constexpr (kRes)
            store_chunk(static_cast<typename H::store_t*>(a.h) + row * a.ld_h, c[i], cols, pack8(H{}, v[i]));
        float g[8], y[8];
        unpack8(rg[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = v[i][j] * rstd * g[j];
        if constexpr (kOut == Out::Bf16)
            store_chunk(static_cast<uint16_t*>(a.y) + row * a.ld_y, c[i], cols, pack8(Bf16{}, y));
        else if constexpr (kOut == Out::F32)
            store_chunk(static_cast<float*>(a.y) + row * a.ld_y, c[i], cols, pack8(F32{}, y));
        else if (a.y) {   // fp8: cols is a multiple of 128, a group is sixteen lanes wide
            float amax = 0.0f, scale;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));
            amax = max_lanes<16>(amax);
            const uint2 q = cast8(a.fmt, a.pow2, y, amax, scale);
            if (c[i].on) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + row * a.ld_y + c[i].c0) = q;
                if ((t & 15) == 0) a.scales[(c[i].c0 >> 7) * a.ld_s + row] = scale;
            }
        }
    }
}

// ------------------------------------------------------------ cast of the transpose
constexpr int kCT = 128;   // tile side: one group of rows

// 16-byte chunk k of row r of the tile sits at slot k ^ swizzle(r), so that the column reads of a
// wave (8 columns x 8 segments of 16 rows) fall into different banks.
template <class S> __device__ __forceinline__ int swizzle(int r);
template <> __device__ __forceinline__ int swizzle<Bf16>(int r) { return r >> 4; }
template <> __device__ __forceinline__ int swizzle<F32>(int r) { return (r >> 4) * 2; }

template <class S, int kFmt, bool kPow2>
__global__ __launch_bounds__(kThreads) void rmsnorm_cast_transpose_kernel(const NormFwdArgs a)
{
    typedef typename S::store_t T;
    constexpr int kPer = 16 / sizeof(T);   // elements of a 16-byte chunk
    constexpr int kChunks = kCT / kPer;    // chunks of a row
    __shared__ __attribute__((aligned(16))) T tile[kCT * kCT];
    const int t = threadIdx.x;
    const int64_t tiles_c = (a.cols + kCT - 1) / kCT;
    const int64_t tr = blockIdx.x / tiles_c;
    const int64_t r0 = tr * kCT;
    const int c0 = (int)(blockIdx.x - tr * tiles_c) * kCT;
    const T* src = static_cast<const T*>(a.src);

#pragma unroll
    for (int u = 0; u < kCT * kChunks / kThreads; ++u) {
        const int id = u * kThreads + t, r = id / kChunks, k = id % kChunks;
        u32x4_t w = {0, 0, 0, 0};
        if (c0 + k * kPer < a.cols) w = *reinterpret_cast<const u32x4_t*>(src + (r0 + r) * a.ld_src + c0 + k * kPer);
        *reinterpret_cast<u32x4_t*>(tile + r * kCT + (k ^ swizzle<S>(r)) * kPer) = w;
    }
    __syncthreads();

    // 8 lanes per column, lane `part` takes rows 16 part .. 16 part + 15
    const int part = t & 7;
    float rs[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) rs[k] = a.rstd[r0 + 16 * part + k];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int col = 32 * u + (t >> 3);
        const bool in = c0 + col < a.cols;
        const float g = in ? as_float((uint32_t)a.gamma[c0 + col] << 16) : 0.0f;
        float y[2][8], amax = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int r = 16 * part + k;
            const T e = tile[r * kCT + ((col / kPer) ^ swizzle<S>(r)) * kPer + col % kPer];
            float v;
            if constexpr (sizeof(T) == 2) v = as_float((uint32_t)e << 16);
            else v = e;
            y[k >> 3][k & 7] = v * rs[k] * g;
            amax = fmaxf(amax, fabsf(y[k >> 3][k & 7]));
        }
        amax = max_lanes<8>(amax);
        float scale;
        const uint2 e0 = cast8<kFmt, kPow2>(y[0], amax, scale);
        const uint2 e1 = cast8<kFmt, kPow2>(y[1], amax, scale);
        if (in) {
            *reinterpret_cast<uint4*>(a.qt + (int64_t)(c0 + col) * a.ld_qt + r0 + part * 16) =
                make_uint4(e0.x, e0.y, e1.x, e1.y);
            if (part == 0) a.scales_t[tr * a.ld_st + c0 + col] = scale;
        }
    }
}

// ------------------------------------------------------------ backward
// With xh = h * rstd and g = dy * gamma:
//   dh = rstd * (g - xh * mean over the row of g * xh) (+ dres),  dgamma = sum over the rows of dy * xh
// A workgroup walks over rows, so a thread keeps its columns of gamma and its sums for dgamma in
// registers; the sums of each workgroup go to a row of the workspace, which a second kernel adds
// up in a fixed order.
template <class Y, class H, bool kRes, int kTPR, int kNV>
__global__ __launch_bounds__(kTPR) void rmsnorm_bwd_kernel(const NormBwdArgs a)
{
    __shared__ float red[2][kTPR / 64];
    const int t = threadIdx.x, cols = a.cols;
    Chunk c[kNV];
    Raw8<Bf16> rg[kNV];
    float dg[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        c[i] = chunk_at((i * kTPR + t) * 8, cols);
        rg[i] = load_chunk<Bf16>(a.gamma, c[i], cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) dg[i][j] = 0.0f;
    }
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const auto* dy = static_cast<const typename Y::store_t*>(a.dy) + row * a.ld_dy;
        const auto* h = static_cast<const typename H::store_t*>(a.h) + row * a.ld_h;
        Raw8<Y> ry[kNV];
        Raw8<H> rh[kNV], rr[kNV];
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            ry[i] = load_chunk<Y>(dy, c[i], cols);
            rh[i] = load_chunk<H>(h, c[i], cols);
        }
        if constexpr (kRes) {
            const auto* res = static_cast<const typename H::store_t*>(a.dres) + row * a.ld_dres;
#pragma unroll
            for (int i = 0; i < kNV; ++i) rr[i] = load_chunk<H>(res, c[i], cols);
        }
        const float rstd = a.rstd[row];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            float dyv[8], hv[8], g[8];
            unpack8(ry[i], dyv);
            unpack8(rh[i], hv);
            unpack8(rg[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = dyv[j] * (hv[j] * rstd);
                dg[i][j] += p;
                dot += j >= c[i].skip ? p * g[j] : 0.0f;
            }
        }
        // (the two halves of `red` take turns: a wave that is a row ahead writes the other one)
        dot = row_sum<kTPR>(dot, red[parity]);
        parity ^= 1;
        const float mean = dot / (float)cols;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            float dyv[8], hv[8], g[8], d[8], r[8] = {};
            unpack8(ry[i], dyv);
            unpack8(rh[i], hv);
            unpack8(rg[i], g);
            if constexpr (kRes) unpack8(rr[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = rstd * (dyv[j] * g[j] - hv[j] * rstd * mean) + r[j];
            store_chunk(static_cast<typename H::store_t*>(a.dh) + row * a.ld_dh, c[i], cols, pack8(H{}, d));
        }
    }
    if (!a.partial) return;   // no dgamma wanted
    float* sums = a.partial + (int64_t)blockIdx.x * a.ld_partial;
#pragma unroll
    for (int i = 0; i < kNV; ++i) store_chunk(sums, c[i], cols, pack8(F32{}, dg[i]));
}

// out[c] = sum over p of partial[p][c], in a fixed order: a workgroup has 32 columns, 8 threads of
// four columns by 32 threads that each take every 32nd row.
constexpr int kRedCols = 32;
__global__ __launch_bounds__(kThreads) void column_sum_kernel(const float* __restrict__ partial, int64_t rows,
                                                              int64_t ld, int cols, float* __restrict__ out)
{
    __shared__ float4 red[32][kRedCols / 4];
    const int t = threadIdx.x, cl = t & 7, rl = t >> 3;
    const int c = blockIdx.x * kRedCols + cl * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < cols) {
#pragma unroll 8
        for (int64_t p = rl; p < rows; p += 32) {
            const float4 w = *reinterpret_cast<const float4*>(partial + p * ld + c);
            s.x += w.x;
            s.y += w.y;
            s.z += w.z;
            s.w += w.w;
        }
    }
    red[rl][cl] = s;
    __syncthreads();
    if (t < kRedCols && blockIdx.x * kRedCols + t < cols) {
        float v = 0.0f;
        for (int i = 0; i < 32; ++i) v += reinterpret_cast<const float*>(&red[i][0])[t];
        out[blockIdx.x * kRedCols + t] = v;
    }
}

template <class X, class H, Out kOut>
hipError_t fwd_rows(const NormFwdArgs& a, hipStream_t stream)
{
    const dim3 grid((unsigned)a.rows);
    if (a.cols <= 2048) rmsnorm_fwd_kernel<X, H, kOut, 256, 1><<<grid, 256, 0, stream>>>(a);
    else if (a.cols <= 4096) rmsnorm_fwd_kernel<X, H, kOut, 256, 2><<<grid, 256, 0, stream>>>(a);
    else if (a.cols <= 8192) rmsnorm_fwd_kernel<X, H, kOut, 256, 4><<<grid, 256, 0, stream>>>(a);
    else if (a.cols <= 16384) rmsnorm_fwd_kernel<X, H, kOut, 1024, 2><<<grid, 1024, 0, stream>>>(a);
    else rmsnorm_fwd_kernel<X, H, kOut, 1024, 4><<<grid, 1024, 0, stream>>>(a);
    return hipGetLastError();
}

template <class X, class H>
hipError_t fwd_out(const NormFwdArgs& a, hipStream_t stream)
{
    switch (a.out) {
    case NormOut::Bf16: return fwd_rows<X, H, Out::Bf16>(a, stream);
    case NormOut::F32: return fwd_rows<X, H, Out::F32>(a, stream);
    default: return fwd_rows<X, H, Out::Fp8>(a, stream);
    }
}

template <class X>
hipError_t fwd_res(const NormFwdArgs& a, hipStream_t stream)
{
    if (!a.res) return fwd_out<X, NoResidual>(a, stream);
    return a.h_bf16 ? fwd_out<X, Bf16>(a, stream) : fwd_out<X, F32>(a, stream);
}

template <class S>
hipError_t fwd_transpose(const NormFwdArgs& a, hipStream_t stream)
{
    const int64_t tiles = a.rows / kCT * ((a.cols + kCT - 1) / kCT);
    if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
    const dim3 grid((unsigned)tiles);
    if (a.fmt == FMT_E4M3) {
        if (a.pow2) rmsnorm_cast_transpose_kernel<S, FMT_E4M3, true><<<grid, kThreads, 0, stream>>>(a);
        else rmsnorm_cast_transpose_kernel<S, FMT_E4M3, false><<<grid, kThreads, 0, stream>>>(a);
    } else {
        if (a.pow2) rmsnorm_cast_transpose_kernel<S, FMT_E5M2, true><<<grid, kThreads, 0, stream>>>(a);
        else rmsnorm_cast_transpose_kernel<S, FMT_E5M2, false><<<grid, kThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <class Y, class H, bool kRes>
hipError_t bwd_rows(const NormBwdArgs& a, hipStream_t stream)
{
    const dim3 grid((unsigned)a.blocks);
    if (a.cols <= 2048) rmsnorm_bwd_kernel<Y, H, kRes, 256, 1><<<grid, 256, 0, stream>>>(a);
    else if (a.cols <= 4096) rmsnorm_bwd_kernel<Y, H, kRes, 256, 2><<<grid, 256, 0, stream>>>(a);
    else if (a.cols <= 8192) rmsnorm_bwd_kernel<Y, H, kRes, 256, 4><<<grid, 256, 0, stream>>>(a);
    else if (a.cols <= 16384) rmsnorm_bwd_kernel<Y, H, kRes, 1024, 2><<<grid, 1024, 0, stream>>>(a);
    else rmsnorm_bwd_kernel<Y, H, kRes, 1024, 4><<<grid, 1024, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const NormFwdArgs& a, hipStream_t stream)
{
    if (a.rows <= 0) return hipSuccess;
    if (a.rows > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipError_t e = a.x_bf16 ? fwd_res<Bf16>(a, stream) : fwd_res<F32>(a, stream);
    if (e != hipSuccess || !a.qt) return e;
    return a.src_bf16 ? fwd_transpose<Bf16>(a, stream) : fwd_transpose<F32>(a, stream);
}

// Four workgroups of 256 threads per compute unit are resident; fewer rows, fewer workgroups.
int64_t rmsnorm_bwd_blocks(int64_t rows, int64_t) { return std::min<int64_t>(rows, 1024); }

hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, hipStream_t stream)
{
    hipError_t e = hipSuccess;
    if (a.blocks > 0) {
#define TE_BWD(Y, H) (a.dres ? bwd_rows<Y, H, true>(a, stream) : bwd_rows<Y, H, false>(a, stream))
        if (a.dy_bf16) e = a.h_bf16 ? TE_BWD(Bf16, Bf16) : TE_BWD(Bf16, F32);
        else e = a.h_bf16 ? TE_BWD(F32, Bf16) : TE_BWD(F32, F32);
#undef TE_BWD
    }
    if (e != hipSuccess || !a.dgamma) return e;
    column_sum_kernel<<<(unsigned)((a.cols + kRedCols - 1) / kRedCols), kThreads, 0, stream>>>(
        a.partial, a.blocks, a.ld_partial, a.cols, a.dgamma);
    return hipGetLastError();
}

}  // namespace tefp8
