// Root-mean-square norm with the residual's addition, for gfx950.
//
//   v = x + residual, rounded to the residual's type and stored as h (v = x without a residual)
//   rstd = 1 / sqrt(mean over the row of v^2 + eps),  y = (v * rstd) * gamma
//
// y is stored in bf16 or fp32, or as its per-token fp8 cast (1x128 groups, the operand of the next
// GEMM) and / or the cast of its transpose (the weight gradient's operand).
//
// Memory-bound.  A row is read once into registers, eight consecutive columns (16 bytes
// of bf16) per thread and as many threads as the row needs; the row's sum of squares is reduced
// over the wave by lane exchanges and over the waves through LDS, and everything that follows
// works from the registers (but for the backward pass beyond 16384 columns, which reads the row again).
// Sixteen consecutive lanes hold one 128-column group, so the fp8 cast needs a four-step lane exchange and no LDS.
//
// Rows whose length is no multiple of eight: the last chunk starts at cols - 8 and overlaps its
// neighbour; the columns that the neighbour has too are left out of the sums and written twice
// with the same value.  Every write of a row comes after all its reads (the reduction lies
// between), so h may be the residual's own buffer.
//
// The cast of the transpose has groups of 128 rows and needs the rstd of each of them, so it runs
// as a second kernel over 128 x 64 tiles of the stored h.
//
// Measured at 8192 x 4096 bf16 with the residual: forward into fp8 45.6 us (235 MB, 5.2 TB/s), the transposed cast
// 18.2 us (101 MB, 5.5 TB/s), backward 47.1 us (277 MB, 5.9 TB/s) and 5.1 us for the sums.
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
// The same past the caches, for inputs that are large beside the last one.  (fp32 comes in two halves of its
// lines, of which the second would be fetched again: it takes the ordinary way.)
__device__ __forceinline__ Raw8<Bf16> load8_past(const uint16_t* p)
{
    return {__builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p))};
}
__device__ __forceinline__ Raw8<F32> load8_past(const float* p) { return load8(p); }
template <class T, int kNV, class P>
__device__ __forceinline__ void load_row(Raw8<T> (&r)[kNV], const P* row, const Chunk (&c)[kNV], int cols, bool past)
{
    if (past) {   // (only set where cols >= 8)
#pragma unroll
        for (int i = 0; i < kNV; ++i) r[i] = c[i].on ? load8_past(row + c[i].c0) : zero8<T>();
    } else {
#pragma unroll
        for (int i = 0; i < kNV; ++i) r[i] = load_chunk<T>(row, c[i], cols);
    }
}
template <class P, class R>
__device__ __forceinline__ void store_chunk(P* row, const Chunk& c, int cols, const R& r)
{
    if (!c.on) return;
    if (cols < 8) store_few(row, r, cols);
    else store8(row + c.c0, r);
}

// A workgroup has kThreadsOf<kTPR> threads, kTPR for each of its rows.
template <int kTPR> constexpr int kThreadsOf = kTPR < 256 ? 256 : kTPR;

// Sum over the kTPR threads of a row.  `red` has room for the waves of the workgroup.
template <int kTPR>
__device__ __forceinline__ float row_sum(float v, float* red)
{
    v = sum_lanes<(kTPR < 64 ? kTPR : 64)>(v);
    if (kTPR <= 64) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    red += threadIdx.x / kTPR * (kTPR / 64);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kTPR / 64; ++i) s += red[i];
    return s;
}

// The largest |y|, NaN if one is NaN: a group with what is not finite is to stand for NaN, and codes
// alone cannot say so (they saturate, and e4m3 has no infinity), so its scale does.
__device__ __forceinline__ float amax_keep(float amax, float y) { return __builtin_elementwise_maximum(amax, fabsf(y)); }
// (the bits of numbers without a sign are in the numbers' order, and NaN's are above all)
template <int kLanes>
__device__ __forceinline__ float amax_lanes(float amax) { return as_float(max_lanes<kLanes>(as_bits(amax))); }

template <int kFmt, bool kPow2>
__device__ __forceinline__ uint2 cast8(const float (&y)[8], float amax, float& scale)
{
    float mult, s[8];
    group_scale<kFmt, kPow2>(amax, scale, mult);
    if (!(amax < __builtin_inff())) scale = __builtin_nanf("");
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
__global__ __launch_bounds__(kThreadsOf<kTPR>) void rmsnorm_fwd_kernel(const NormFwdArgs a)
{
    constexpr bool kRes = !__is_same(H, NoResidual);
    constexpr int kRows = kThreadsOf<kTPR> / kTPR;
    __shared__ float red[kThreadsOf<kTPR> / 64];
    // rows past the end repeat the last one and store nothing
    const int64_t row_raw = a.first_row + xcd_run(blockIdx.x, gridDim.x) * kRows + threadIdx.x / kTPR;
    const bool in = row_raw < a.rows;
    const int64_t row = in ? row_raw : a.rows - 1;
    const int t = threadIdx.x % kTPR, cols = a.cols;
    const auto* x = static_cast<const typename X::store_t*>(a.x) + row * a.ld_x;

    Chunk c[kNV];
    Raw8<X> rx[kNV];
    Raw8<Bf16> rg[kNV];
    float v[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i) c[i] = chunk_at((i * kTPR + t) * 8, cols);
    load_row(rx, x, c, cols, a.past);
    if constexpr (kRes) {
        const auto* res = static_cast<const typename H::store_t*>(a.res) + row * a.ld_res;
        Raw8<H> rr[kNV];
        load_row(rr, res, c, cols, a.past);
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
    if (!in) return;
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
            for (int j = 0; j < 8; ++j) amax = amax_keep(amax, y[j]);
            amax = amax_lanes<16>(amax);
            const uint2 q = cast8(a.fmt, a.pow2, y, amax, scale);
            if (c[i].on) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + row * a.ld_y + c[i].c0) = q;
                if ((t & 15) == 0) a.scales[(c[i].c0 >> 7) * a.ld_s + row] = scale;
            }
        }
    }
}

// ------------------------------------------------------------ cast of the transpose
constexpr int kCT = 128;   // rows of a tile: one group
constexpr int kCW = 64;    // columns

// Where 16-byte chunk k of row r of the tile lies, in elements: the column reads of a wave (8 pairs of
// columns x 8 segments of 16 rows) fall into different banks.
template <class S> __device__ __forceinline__ int tile_at(int r, int k);
template <> __device__ __forceinline__ int tile_at<Bf16>(int r, int k)   // a row takes half the banks: a row's gap after each segment
{
    return (r + (r >> 4)) * kCW + (k ^ (r >> 5) * 2) * 8;
}
template <> __device__ __forceinline__ int tile_at<F32>(int r, int k) { return r * kCW + (k ^ (r >> 4) * 2) * 4; }

// One tile per workgroup, 8192 x 4096 bf16 in 17.3 us (5.8 TB/s); 128 columns per tile and two
// tiles per workgroup, the second's loads ahead, took 20.1.  Four waves per SIMD: cut for eight, the
// registers hold too few of a lane's sixteen LDS reads at a time (22.8 us).
template <class S, int kFmt, bool kPow2>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4, 4)))
void rmsnorm_cast_transpose_kernel(const NormFwdArgs a)
{
    typedef typename S::store_t T;
    constexpr int kPer = 16 / sizeof(T);   // elements of a 16-byte chunk
    constexpr int kChunks = kCW / kPer;    // chunks of a row
    constexpr int kLoads = kCT * kChunks / kThreads;
    __shared__ __attribute__((aligned(16))) T tile[(kCT + kCT / 16) * kCW];
    const int t = threadIdx.x;
    const int64_t tiles_c = (a.cols + kCW - 1) / kCW;
    const int64_t tr = blockIdx.x / tiles_c, r0 = tr * kCT;
    const int c0 = (int)(blockIdx.x - tr * tiles_c) * kCW;
    // 8 lanes per pair of columns, lane `part` takes rows 16 part .. 16 part + 15
    const int part = t & 7;

    const int col = (t >> 3) * 2;   // and its neighbour (cols is even)
    const bool in = c0 + col < a.cols;
    const uint32_t gw = in ? *reinterpret_cast<const uint32_a2*>(a.gamma + c0 + col) : 0;
    const int cc = c0 + t % kChunks * kPer;
    const T* src = static_cast<const T*>(a.src) + (r0 + t / kChunks) * a.ld_src + cc;
    u32x4_t v[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
        v[u] = u32x4_t{0, 0, 0, 0};
        if (cc < a.cols) v[u] = *reinterpret_cast<const u32x4_t*>(src + u * (kThreads / kChunks) * a.ld_src);
    }
    float rs[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const u32x4_t w = *reinterpret_cast<const u32x4_a4*>(a.rstd + r0 + 16 * part + 4 * k);
#pragma unroll
        for (int j = 0; j < 4; ++j) rs[4 * k + j] = as_float(w[j]);
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
        *reinterpret_cast<u32x4_t*>(tile + tile_at<S>(u * (kThreads / kChunks) + t / kChunks, t % kChunks)) = v[u];
    __syncthreads();
    const float g[2] = {as_float(gw << 16), as_float(gw & 0xFFFF0000u)};
    float y[2][2][8], amax[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int r = 16 * part + k;
        const T* at = tile + tile_at<S>(r, col / kPer) + col % kPer;
        float v[2];
        if constexpr (sizeof(T) == 2) {
            const uint32_t e = *reinterpret_cast<const uint32_t*>(at);
            v[0] = as_float(e << 16);
            v[1] = as_float(e & 0xFFFF0000u);
        } else {
            const float2 e = *reinterpret_cast<const float2*>(at);
            v[0] = e.x;
            v[1] = e.y;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            y[q][k >> 3][k & 7] = v[q] * rs[k] * g[q];
            amax[q] = amax_keep(amax[q], y[q][k >> 3][k & 7]);
        }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        amax[q] = amax_lanes<8>(amax[q]);
        float scale;
        const uint2 e0 = cast8<kFmt, kPow2>(y[q][0], amax[q], scale);
        const uint2 e1 = cast8<kFmt, kPow2>(y[q][1], amax[q], scale);
        if (in) {
            *reinterpret_cast<uint4*>(a.qt + (int64_t)(c0 + col + q) * a.ld_qt + r0 + part * 16) =
                make_uint4(e0.x, e0.y, e1.x, e1.y);
            if (part == 0) a.scales_t[tr * a.ld_st + c0 + col + q] = scale;
        }
    }
}

// ------------------------------------------------------------ backward
// With xh = h * rstd and g = dy * gamma:
//   dh = rstd * (g - xh * mean over the row of g * xh) (+ dres),  dgamma = sum over the rows of dy * xh
// A workgroup walks over rows, so a thread keeps its columns of gamma and its sums for dgamma in
// registers; the sums of each workgroup (its rows side by side added through LDS) go to a row of the
// workspace, and a second kernel adds those up in a fixed order.
template <class Y, class H, bool kRes, int kTPR, int kNV>
__global__ __launch_bounds__(kThreadsOf<kTPR>) void rmsnorm_bwd_kernel(const NormBwdArgs a)
{
    constexpr int kRows = kThreadsOf<kTPR> / kTPR;
    // Four chunks per thread do not fit the registers beside the sums for dgamma: such rows are read again
    // after the reduction (838 x 20000 bf16: 45 us, and 150 with all of it kept and the registers spilled).  With
    // an fp32 operand 3 to 25 registers are spilled all the same (838 x 20000 in fp32: 101 us).
    constexpr bool kTwice = kNV == 4;
    __shared__ float red[2][kThreadsOf<kTPR> / 64];
    __shared__ float slots[kRows > 1 ? kRows : 1][kRows > 1 ? kTPR * 8 : 1];
    const int t = threadIdx.x % kTPR, slot = threadIdx.x / kTPR, cols = a.cols;
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
    for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += (int64_t)gridDim.x * kRows) {
        // rows past the end repeat the last one, add nothing and store nothing
        const bool in = kRows == 1 || base + slot < a.rows;
        const int64_t row = in ? base + slot : a.rows - 1;
        const auto* dy = static_cast<const typename Y::store_t*>(a.dy) + row * a.ld_dy;
        const auto* h = static_cast<const typename H::store_t*>(a.h) + row * a.ld_h;
        const auto* res = static_cast<const typename H::store_t*>(a.dres) + (kRes ? row * a.ld_dres : 0);
        Raw8<Y> ry[kNV];
        Raw8<H> rh[kNV], rr[kNV];
        if constexpr (!kTwice) {
            load_row(ry, dy, c, cols, false);
            load_row(rh, h, c, cols, false);
            if constexpr (kRes) load_row(rr, res, c, cols, false);
        }
        const float rstd = a.rstd[row];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            if constexpr (kTwice) {
                ry[i] = load_chunk<Y>(dy, c[i], cols);
                rh[i] = load_chunk<H>(h, c[i], cols);
                rg[i] = load_chunk<Bf16>(a.gamma, c[i], cols);
            }
            float dyv[8], hv[8], g[8];
            unpack8(ry[i], dyv);
            unpack8(rh[i], hv);
            unpack8(rg[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = dyv[j] * (hv[j] * rstd);
                dg[i][j] += in ? p : 0.0f;
                dot += j >= c[i].skip ? p * g[j] : 0.0f;
            }
        }
        // (the two halves of `red` take turns: a wave that is a row ahead writes the other one)
        dot = row_sum<kTPR>(dot, red[parity]);
        parity ^= 1;
        const float mean = dot / (float)cols;
        if (!in) continue;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            if constexpr (kTwice) {
                asm volatile("" ::: "memory");   // (loaded here again, not kept)
                ry[i] = load_chunk<Y>(dy, c[i], cols);
                rh[i] = load_chunk<H>(h, c[i], cols);
                rg[i] = load_chunk<Bf16>(a.gamma, c[i], cols);
                if constexpr (kRes) rr[i] = load_chunk<H>(res, c[i], cols);
            }
            float dyv[8], hv[8], g[8], d[8], r[8] = {};
            unpack8(ry[i], dyv);
            unpack8(rh[i], hv);
            unpack8(rg[i], g);
            if constexpr (kRes) unpack8(rr[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = rstd * (dyv[j] * g[j] - hv[j] * rstd * mean) + r[j];
            auto* out = static_cast<typename H::store_t*>(a.dh) + row * a.ld_dh;
            if (kTwice && c[i].skip > 0) {
                // (dh may be dres, which the neighbour reads for itself only now)
                if (c[i].on)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j >= c[i].skip) store_one(out + c[i].c0 + j, pack8(H{}, d), j);
            } else {
                store_chunk(out, c[i], cols, pack8(H{}, d));
            }
        }
    }
    if (!a.partial) return;   // no dgamma wanted
    float* sums = a.partial + (int64_t)blockIdx.x * a.ld_partial;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) store_chunk(sums, c[i], cols, pack8(F32{}, dg[i]));
    } else {
        static_assert(kNV == 1, "rows side by side have one chunk per thread");
        if (c[0].on)
#pragma unroll
            for (int j = 0; j < 8; ++j) slots[slot][c[0].c0 + j] = dg[0][j];
        __syncthreads();
        for (int e = threadIdx.x; e < cols; e += kThreadsOf<kTPR>) {
            float v = 0.0f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) v += slots[r][e];
            sums[e] = v;
        }
    }
}

// out[c] = sum over p of partial[p][c], in a fixed order: a workgroup has 16 columns, 4 threads of
// four columns by 64 threads that each take every 64th row.
constexpr int kRedCols = 16;
__global__ __launch_bounds__(kThreads) void column_sum_kernel(const float* __restrict__ partial, int64_t rows,
                                                              int64_t ld, int cols, float* __restrict__ out)
{
    constexpr int kPer = kRedCols / 4, kLanes = kThreads / kPer;
    __shared__ float red[kLanes][kRedCols];
    const int t = threadIdx.x, cl = t % kPer, rl = t / kPer;
    const int c = blockIdx.x * kRedCols + cl * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < cols) {
#pragma unroll 8
        for (int64_t p = rl; p < rows; p += kLanes) {
            const float4 w = *reinterpret_cast<const float4*>(partial + p * ld + c);
            s.x += w.x;
            s.y += w.y;
            s.z += w.z;
            s.w += w.w;
        }
    }
    *reinterpret_cast<float4*>(&red[rl][cl * 4]) = s;
    __syncthreads();
    // sixteen threads per column, four rows of sums each
    const int col = t % kRedCols, part = t / kRedCols;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kLanes * kRedCols / kThreads; ++i) v += red[part * (kLanes * kRedCols / kThreads) + i][col];
    __syncthreads();
    red[part][col] = v;
    __syncthreads();
    if (t < kRedCols && blockIdx.x * kRedCols + t < cols) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < kThreads / kRedCols; ++i) v += red[i][t];
        out[blockIdx.x * kRedCols + t] = v;
    }
}

// Threads per row: as many as give each one chunk of eight columns (up to 1024 threads, then two or four
// chunks).  Against two chunks and half the threads, 8192 x 4096 bf16 took 38.8 us instead of 39.2 forward
// and 46.2 instead of 48.5 backward, one row 2.5 us instead of 3.0; four and eight chunks were slower.
// F<kTPR, kNV>::run(a, stream) is called for the row length.
template <template <int, int> class F, class A>
void by_cols(const A& a, hipStream_t stream)
{
    if (a.cols <= 128) F<16, 1>::run(a, stream);
    else if (a.cols <= 256) F<32, 1>::run(a, stream);
    else if (a.cols <= 512) F<64, 1>::run(a, stream);
    else if (a.cols <= 1024) F<128, 1>::run(a, stream);
    else if (a.cols <= 2048) F<256, 1>::run(a, stream);
    else if (a.cols <= 4096) F<512, 1>::run(a, stream);
    else if (a.cols <= 8192) F<1024, 1>::run(a, stream);
    else if (a.cols <= 16384) F<1024, 2>::run(a, stream);
    else F<1024, 4>::run(a, stream);
}
int threads_per_row(int64_t cols)
{
    return cols <= 128 ? 16 : cols <= 256 ? 32 : cols <= 512 ? 64 : cols <= 1024 ? 128 : cols <= 2048 ? 256 : cols <= 4096 ? 512 : 1024;
}

// Inputs of this many bytes are read past the caches, so that h and the outputs stay in the last one: with them a
// call of this size fills its 256 MiB.  Forward with the residual, 4096 columns of bf16, without the transposed cast,
// ordinarily and past the caches, in microseconds: where x was just written by another kernel and the residual was not
// touched lately, 96 MiB 32.2 and 31.6, 128 MiB 48.1 and 40.5, 160 MiB 53.2 and 51.3, 256 MiB 96.7 and 82.4, 512 MiB
// 176.7 and 159.5; where neither was touched lately, 33.0 and 33.0, 46.7 and 40.3, 56.1 and 50.3, 110.4 and 77.8,
// 179.3 and 182.7; of the same inputs again and again (still in the cache where they fit), 29.8 and 33.0, 38.8 and
// 41.8, 55.7 and 50.1, 107.2 and 79.4, 180.2 and 184.7.  From 64 MiB down they differ by at most 2 us either way.  The
// residual alone past the caches lies between the two.  The backward pass is slower that way at every size (8192 rows:
// 55.5 and 60.3).
bool past_caches(int64_t bytes) { return bytes >= (int64_t)128 << 20; }

template <class X, class H, Out kOut> struct Fwd {
    template <int kTPR, int kNV> struct Rows {
        // Rows of 4097 to 8192 columns take two chunks for each of 512 threads, though 1024 would have one each: from
        // 1024 rows on two are up to 30 % faster where 1024 threads are half idle, and still 3 to 10 % at 7936
        // columns (bf16 with the residual, microseconds with one chunk and with two: 4096 x 5120 33.6 and 28.0,
        // 4096 x 7168 44.0 and 38.8, 2114 x 7936 26.3 and 24.8); few rows take 0.1 to 0.2 us more. At 8192 columns,
        // where no thread is idle, they are even (4096 x 8192 46.9 and 46.0) but for fp32 x with a residual (with
        // an fp32 residual 106.7 and 113.9, with a bf16 one 55.2 and 58.4), which keeps one chunk there.  The backward
        // pass gains nothing from two.
        static constexpr bool kWide = kTPR == 1024 && kNV == 1, kFullRows = __is_same(X, F32) && !__is_same(H, NoResidual);
        static void run(const NormFwdArgs& a, hipStream_t stream)
        {
            if constexpr (!kWide || kFullRows) {
                if (!kWide || a.cols > 7936) return launch(a, stream);
            }
            if constexpr (kWide) Rows<512, 2>::launch(a, stream);
        }
        static void launch(const NormFwdArgs& a, hipStream_t stream)
        {
            constexpr int kThreads = kThreadsOf<kTPR>, kRows = kThreads / kTPR;
            // (a launch has at most 2^32 threads: more rows than that take several)
            constexpr int64_t kMost = ((int64_t)1 << 31) / kThreads * kRows;
            NormFwdArgs part = a;
            for (part.first_row = 0; part.first_row < a.rows; part.first_row += kMost) {
                const int64_t rows = std::min(kMost, a.rows - part.first_row);
                rmsnorm_fwd_kernel<X, H, kOut, kTPR, kNV>
                    <<<(unsigned)((rows + kRows - 1) / kRows), kThreads, 0, stream>>>(part);
            }
        }
    };
};

template <class X, class H, Out kOut>
hipError_t fwd_rows(const NormFwdArgs& a, hipStream_t stream)
{
    by_cols<Fwd<X, H, kOut>::template Rows>(a, stream);
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

template <class S, int kFmt, bool kPow2>
hipError_t transpose_run(const NormFwdArgs& a, hipStream_t stream)
{
    const int64_t tiles = a.rows / kCT * ((a.cols + kCW - 1) / kCW);
    rmsnorm_cast_transpose_kernel<S, kFmt, kPow2><<<(unsigned)tiles, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <class S>
hipError_t fwd_transpose(const NormFwdArgs& a, hipStream_t stream)
{
    if (a.fmt == FMT_E4M3)
        return a.pow2 ? transpose_run<S, FMT_E4M3, true>(a, stream) : transpose_run<S, FMT_E4M3, false>(a, stream);
    return a.pow2 ? transpose_run<S, FMT_E5M2, true>(a, stream) : transpose_run<S, FMT_E5M2, false>(a, stream);
}

template <class Y, class H, bool kRes> struct Bwd {
    template <int kTPR, int kNV> struct Rows {
        static void run(const NormBwdArgs& a, hipStream_t stream)
        {
            rmsnorm_bwd_kernel<Y, H, kRes, kTPR, kNV><<<(unsigned)a.blocks, kThreadsOf<kTPR>, 0, stream>>>(a);
        }
    };
};

template <class Y, class H, bool kRes>
hipError_t bwd_rows(const NormBwdArgs& a, hipStream_t stream)
{
    by_cols<Bwd<Y, H, kRes>::template Rows>(a, stream);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const NormFwdArgs& args, hipStream_t stream)
{
    NormFwdArgs a = args;
    if (a.rows <= 0) return hipSuccess;
    if (a.qt && a.rows / kCT * ((a.cols + kCW - 1) / kCW) >= ((int64_t)1 << 32) / kThreads) return hipErrorInvalidValue;
    a.past = a.cols >= 8 && past_caches(a.rows * a.cols * ((a.x_bf16 ? 2 : 4) + (a.res ? a.h_bf16 ? 2 : 4 : 0)));
    hipError_t e = a.x_bf16 ? fwd_res<Bf16>(a, stream) : fwd_res<F32>(a, stream);
    if (e != hipSuccess || !a.qt) return e;
    return a.src_bf16 ? fwd_transpose<Bf16>(a, stream) : fwd_transpose<F32>(a, stream);
}

// 1024 threads per compute unit (8192 x 4096 bf16: 46.2 us; with 2560 at two chunks each 51.5), and fewer for
// few rows.
int64_t rmsnorm_bwd_blocks(int64_t rows, int64_t cols)
{
    const int tpr = threads_per_row(cols), threads = std::max(tpr, 256);
    const int64_t per = threads / tpr;
    return std::min<int64_t>((rows + per - 1) / per, device_cus() * (1024 / threads));
}

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
