// Layer norm with the dropped branch's and the residual's addition, for gfx950.
//
//   h = dropout(x) + residual, rounded to the residual's type and stored (h = x without a residual)
//   mean, rstd = 1 / sqrt(mean of (h - mean)^2 + eps),  y = ((h - mean) * rstd) * gamma + beta
//
// Stored as the root-mean-square norm stores its y (norm.hip), whose layout of a row over the threads this is too: the
// row is read once into registers, eight columns to a thread.  The mean is summed in 64 bits, so that it is exact but for
// its rounding (a constant row comes out as exactly beta; in 32 bits its error is that of values far larger than
// itself, and a reduction of the differences would have to correct it); the variance, of the differences from it and
// corrected for that rounding, takes a second reduction.  Dropout's bits are computed in registers, one counter of
// the generator per chunk.
//
// Memory-bound: x, residual, h and y once each.  8192 x 4096 bf16 with the residual to e4m3: 49 us, with dropout 51
// (the generator's multiplications, in a kernel whose one row per workgroup leaves little to hide them behind), with the
// transposed layout as well 64 and 68, whose second kernel reads h once more; to fp32 without a residual, 4999 x 2112, 16.4 us
// (5.1 TB/s).  Backward, 8192 x 4096: 44.6 us, with dropout 53.8; with the residual's gradient 57 and 75.
// Rows of more than 8192 columns take 1024 threads of 128 registers.  They hold the forward's chunks up to 16384 columns (8192 x
// 14336 with the residual to bf16 217 us, the root-mean-square norm's 173) and spill some beyond (4096 x 32768 250 and 206);
// the backward's two column sums do not fit beside its chunks (with the residual's gradient 468 and 178; 856 and 254).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#ifndef TE_LAYERNORM_PART
#define TE_LAYERNORM_PART -1
#endif

#include "block_internal.h"
#include "dropout_device.h"
#include "fp8_codec.h"
#include "norm_device.h"
#include "ops_device.h"

namespace tefp8 {
namespace {

// 1 / sqrt(x) by the hardware's instruction (off by an ulp), whose inputs must not be subnormal.
__device__ __forceinline__ float inverse_root(float x)
{
    const bool small = x < 0x1p-96f;
    return __builtin_amdgcn_rsqf(small ? x * 0x1p64f : x) * (small ? 0x1p32f : 1.0f);
}

// The cast of a chunk, its group's largest value known.  x * (FP8_MAX / amax) is at most FP8_MAX (1 + 2^-23), which rounds
// to FP8_MAX: there is nothing to clamp.  A group with what is not finite stands for NaN, as in cast8.
template <int kFmt>
__device__ __forceinline__ uint2 encode_scaled(const float (&y)[8], float mult)
{
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float a = y[4 * h] * mult, b = y[4 * h + 1] * mult, c = y[4 * h + 2] * mult, d = y[4 * h + 3] * mult;
        int p;
        if (kFmt == FMT_E4M3) {
            p = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
            p = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, p, true);
        } else {
            p = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
            p = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, p, true);
        }
        w[h] = (uint32_t)p;
    }
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ uint2 cast_scaled(int fmt, int pow2, const float (&y)[8], float amax, float& scale)
{
    float mult;
    if (fmt == FMT_E4M3) pow2 ? group_scale<FMT_E4M3, true>(amax, scale, mult) : group_scale<FMT_E4M3, false>(amax, scale, mult);
    else pow2 ? group_scale<FMT_E5M2, true>(amax, scale, mult) : group_scale<FMT_E5M2, false>(amax, scale, mult);
    if (!(amax < __builtin_inff())) scale = __builtin_nanf("");
    return fmt == FMT_E4M3 ? encode_scaled<FMT_E4M3>(y, mult) : encode_scaled<FMT_E5M2>(y, mult);
}

// One row to kTPR threads.  What a thread does once for its row counts as much as its eight columns: the divisions by the
// columns are products with their inverse, and the inverse root is the hardware's.
template <class X, class H, Out kOut, int kTPR, int kNV>
__global__ __launch_bounds__(kThreadsOf<kTPR>) void layernorm_fwd_kernel(const LayerNormFwdArgs a)
{
    constexpr bool kRes = !__is_same(H, NoResidual);
    typedef typename std::conditional<kRes, H, X>::type R;   // what the norm is of
    constexpr int kRows = kThreadsOf<kTPR> / kTPR;
    __shared__ double red[kThreadsOf<kTPR> / 64];
    __shared__ float red2[kThreadsOf<kTPR> / 64];
    // rows past the end repeat the last one and store nothing
    const int64_t row_raw = a.first_row + xcd_run(blockIdx.x, gridDim.x) * kRows + threadIdx.x / kTPR;
    const bool in = row_raw < a.rows;
    const int64_t row = in ? row_raw : a.rows - 1;
    const int t = threadIdx.x % kTPR, cols = a.cols;
    const auto* x = static_cast<const typename X::store_t*>(a.x) + row * a.ld_x;

    Chunk c[kNV];
    Raw8<X> rx[kNV];
    Raw8<R> rh[kNV];
    Raw8<Bf16> rg[kNV], rb[kNV];
    float v[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i) c[i] = chunk_at((i * kTPR + t) * 8, cols);
    load_row(rx, x, c, cols, a.past);
    if constexpr (kRes) load_row(rh, static_cast<const typename R::store_t*>(a.res) + row * a.ld_res, c, cols, a.past);
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        rg[i] = load_chunk<Bf16>(a.gamma, c[i], cols);
        rb[i] = a.beta ? load_chunk<Bf16>(a.beta, c[i], cols) : zero8<Bf16>();
    }
    const DropKey key = drop_key(a.drop);
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        unpack8(rx[i], v[i]);
        if constexpr (kRes) {
            float r[8];
            unpack8(rh[i], r);
            if (a.drop.below) drop8(a.drop, drop_chunk(a.drop, key, c[i].c0, c[i].on ? c[i].skip : 0, row), v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += r[j];
            rh[i] = pack8(R{}, v[i]);   // the stored sum is what the norm is of
            unpack8(rh[i], v[i]);
        }
    }
    // Sums, then squares of the differences (which take v's place).  Where the columns fill their chunks, a chunk counts as
    // a whole or not at all; else the columns that the chunk before has too, or, in a row of less than eight, that are
    // none, are left out one by one.
    double s = 0.0;
    float d2 = 0.0f;
    const bool whole = (cols & 7) == 0;
    if (whole) {
#pragma unroll
        for (int i = 0; i < kNV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += (double)v[i][j];   // (0 in a chunk past the end)
    } else {
#pragma unroll
        for (int i = 0; i < kNV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += j >= c[i].skip ? (double)v[i][j] : 0.0;
    }
    s = row_sum64<kTPR>(s, red) * a.inv_cols;
    const float mean = (float)s, off = (float)(s - (double)mean);   // (the mean's rounding, of which the variance knows)
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] -= mean;
    if (whole) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            float part = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) part = fmaf(v[i][j], v[i][j], part);
            d2 += c[i].on ? part : 0.0f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kNV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                d2 += c[i].on && j >= c[i].skip && (cols >= 8 || j < cols) ? v[i][j] * v[i][j] : 0.0f;
    }
    d2 = row_sum<kTPR>(d2, red2);
    float var = d2 * (float)a.inv_cols - off * off;
    var = var < 0.0f ? 0.0f : var;   // (NaN stays)
    const float rstd = inverse_root(var + a.eps);
    if (!in) return;
    if (t == 0) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }

#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        if constexpr (kRes) store_chunk(static_cast<typename R::store_t*>(a.h) + row * a.ld_h, c[i], cols, rh[i]);
        float g[8], b[8], y[8];
        unpack8(rg[i], g);
        unpack8(rb[i], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = fmaf(v[i][j] * rstd, g[j], b[j]);
        if constexpr (kOut == Out::Bf16)
            store_chunk(static_cast<uint16_t*>(a.y) + row * a.ld_y, c[i], cols, pack8(Bf16{}, y));
        else if constexpr (kOut == Out::F32)
            store_chunk(static_cast<float*>(a.y) + row * a.ld_y, c[i], cols, pack8(F32{}, y));
        else if (a.y) {   // fp8: cols is a multiple of 128, a group is sixteen lanes wide
            float amax = 0.0f, scale;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = amax_keep(amax, y[j]);
            amax = amax_lanes<16>(amax);
            const uint2 q = cast_scaled(a.fmt, a.pow2, y, amax, scale);
            if (c[i].on) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + row * a.ld_y + c[i].c0) = q;
                if ((t & 15) == 0) a.scales[(c[i].c0 >> 7) * a.ld_s + row] = scale;
            }
        }
    }
}

// The cast of the transpose: groups of 128 rows need the mean and rstd of each of them, so it runs as a second kernel
// over 128 x 64 tiles of the stored h, as norm.hip's does.
template <class S, int kFmt, bool kPow2>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4, 4)))
void layernorm_cast_transpose_kernel(const LayerNormFwdArgs a)
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
    const int part = t & 7;         // 8 lanes per pair of columns, lane `part` takes rows 16 part .. 16 part + 15
    const int col = (t >> 3) * 2;   // and its neighbour (cols is even)
    const bool in = c0 + col < a.cols;
    const uint32_t gw = in ? *reinterpret_cast<const uint32_a2*>(a.gamma + c0 + col) : 0;
    const uint32_t bw = in && a.beta ? *reinterpret_cast<const uint32_a2*>(a.beta + c0 + col) : 0;
    const int cc = c0 + t % kChunks * kPer;
    const T* src = static_cast<const T*>(a.src) + (r0 + t / kChunks) * a.ld_src + cc;
    u32x4_t v[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
        v[u] = u32x4_t{0, 0, 0, 0};
        if (cc < a.cols) v[u] = *reinterpret_cast<const u32x4_t*>(src + u * (kThreads / kChunks) * a.ld_src);
    }
    float mu[16], rs[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const u32x4_t m = *reinterpret_cast<const u32x4_a4*>(a.mean + r0 + 16 * part + 4 * k);
        const u32x4_t w = *reinterpret_cast<const u32x4_a4*>(a.rstd + r0 + 16 * part + 4 * k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            mu[4 * k + j] = as_float(m[j]);
            rs[4 * k + j] = as_float(w[j]);
        }
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
        *reinterpret_cast<u32x4_t*>(tile + tile_at<S>(u * (kThreads / kChunks) + t / kChunks, t % kChunks)) = v[u];
    __syncthreads();
    const float g[2] = {as_float(gw << 16), as_float(gw & 0xFFFF0000u)};
    const float b[2] = {as_float(bw << 16), as_float(bw & 0xFFFF0000u)};
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
            y[q][k >> 3][k & 7] = fmaf((v[q] - mu[k]) * rs[k], g[q], b[q]);
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
// With xh = (h - mean) * rstd and g = dy * gamma:
//   dh = rstd * (g - mean of g - xh * mean of g * xh) (+ dres),  dx = dropout(dh)
//   dgamma = sum over the rows of dy * xh,  dbeta = sum over the rows of dy
// A workgroup walks over rows with its columns' sums for dgamma and dbeta in registers; they go to a row of the
// workspace each, and a second kernel adds those up in a fixed order.
template <class Y, class H, bool kRes, int kTPR, int kNV>
__global__ __launch_bounds__(kThreadsOf<kTPR>) void layernorm_bwd_kernel(const LayerNormBwdArgs a)
{
    constexpr int kRows = kThreadsOf<kTPR> / kTPR;
    // (rows of more than 16384 columns are read again after the reduction, as in norm.hip)
    constexpr bool kTwice = kNV == 4;
    // The next row's loads are out before this row's sums, where a thread has one chunk (8192 x 4096 without dropout 51.2 us,
    // and 55.3 without that).  With two the registers do not hold two rows (spilled, 2048 x 8200 bf16 182 us, and 130
    // without; 8192 x 14336 721 and 471; fp32 1099 and 627), and rows that are read twice gain nothing from their mean
    // and deviation alone (4096 x 32768 878 and 861, fp32 1117 and 975).
    constexpr bool kAhead = kNV == 1;
    __shared__ float2 red[2][kThreadsOf<kTPR> / 64];
    __shared__ float slots[kRows > 1 ? kRows : 1][kRows > 1 ? kTPR * 8 : 1];
    const int t = threadIdx.x % kTPR, slot = threadIdx.x / kTPR, cols = a.cols;
    Chunk c[kNV];
    Raw8<Bf16> rg[kNV];
    float dg[kNV][8], db[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        c[i] = chunk_at((i * kTPR + t) * 8, cols);
        rg[i] = load_chunk<Bf16>(a.gamma, c[i], cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = 0.0f;
    }
    const DropKey key = drop_key(a.drop);
    Raw8<Y> ry[kNV];
    Raw8<H> rh[kNV], rr[kNV];
    float mean, rstd;
    const auto load = [&](int64_t base) {
        const int64_t row = min(base + slot, a.rows - 1);   // (rows past the end repeat the last one, add and store nothing)
        if constexpr (!kTwice) {
            load_row(ry, static_cast<const typename Y::store_t*>(a.dy) + row * a.ld_dy, c, cols, false);
            load_row(rh, static_cast<const typename H::store_t*>(a.h) + row * a.ld_h, c, cols, false);
            if constexpr (kRes) load_row(rr, static_cast<const typename H::store_t*>(a.dres) + row * a.ld_dres, c, cols, false);
        }
        mean = a.mean[row];
        rstd = a.rstd[row];
    };
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t base = (int64_t)blockIdx.x * kRows;
    if constexpr (kAhead) load(base);
    for (int parity = 0; base < a.rows; base += step, parity ^= 1) {
        const bool in = kRows == 1 || base + slot < a.rows;
        const int64_t row = in ? base + slot : a.rows - 1;
        const auto* dy = static_cast<const typename Y::store_t*>(a.dy) + row * a.ld_dy;
        const auto* h = static_cast<const typename H::store_t*>(a.h) + row * a.ld_h;
        const auto* res = static_cast<const typename H::store_t*>(a.dres) + (kRes ? row * a.ld_dres : 0);
        if constexpr (!kAhead) load(base);
        // (what this row needs of the loads, before the next row's take their registers)
        Raw8<Y> cy[kNV];
        Raw8<H> ch[kNV], cr[kNV];
        const float mu = mean, rs = rstd;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            cy[i] = ry[i];
            ch[i] = rh[i];
            if constexpr (kRes) cr[i] = rr[i];
        }
        if constexpr (kAhead)
            if (base + step < a.rows) load(base + step);
        float sg = 0.0f, sx = 0.0f;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            if constexpr (kTwice) {
                cy[i] = load_chunk<Y>(dy, c[i], cols);
                ch[i] = load_chunk<H>(h, c[i], cols);
                rg[i] = load_chunk<Bf16>(a.gamma, c[i], cols);
            }
            float dyv[8], hv[8], g[8];
            unpack8(cy[i], dyv);
            unpack8(ch[i], hv);
            unpack8(rg[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = dyv[j] * ((hv[j] - mu) * rs);
                dg[i][j] += in ? p : 0.0f;
                db[i][j] += in ? dyv[j] : 0.0f;
                // (behind the end of a row of less than eight columns p may be 0 times an overflow)
                const bool mine = c[i].on && j >= c[i].skip && (kTPR > 16 || cols >= 8 || j < cols);
                sg += mine ? dyv[j] * g[j] : 0.0f;
                sx += mine ? p * g[j] : 0.0f;
            }
        }
        // (the two halves of `red` take turns: a wave that is a row ahead writes the other one)
        row_sum2<kTPR>(sg, sx, red[parity]);
        const float mg = sg * a.inv_cols, mx = sx * a.inv_cols;
        if (!in) continue;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            if constexpr (kTwice) {
                asm volatile("" ::: "memory");   // (loaded here again, not kept)
                cy[i] = load_chunk<Y>(dy, c[i], cols);
                ch[i] = load_chunk<H>(h, c[i], cols);
                rg[i] = load_chunk<Bf16>(a.gamma, c[i], cols);
                if constexpr (kRes) cr[i] = load_chunk<H>(res, c[i], cols);
            }
            float dyv[8], hv[8], g[8], d[8], r[8] = {};
            unpack8(cy[i], dyv);
            unpack8(ch[i], hv);
            unpack8(rg[i], g);
            if constexpr (kRes) unpack8(cr[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = rs * ((dyv[j] * g[j] - mg) - (hv[j] - mu) * rs * mx) + r[j];
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
            if (a.dx) {
                // (what the neighbour has too is in dres as long as that is read once: the same value again; read
                // twice, it may be dh by now, and is left to the neighbour)
                drop8(a.drop, drop_chunk(a.drop, key, c[i].c0, c[i].on ? c[i].skip : 0, row), d);
                const bool some = kTwice && c[i].skip > 0;
                if (a.dx_bf16) {
                    uint16_t* o = static_cast<uint16_t*>(a.dx) + row * a.ld_dx;
                    if (!some) store_chunk(o, c[i], cols, pack8(Bf16{}, d));
                    else if (c[i].on)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j >= c[i].skip) store_one(o + c[i].c0 + j, pack8(Bf16{}, d), j);
                } else {
                    float* o = static_cast<float*>(a.dx) + row * a.ld_dx;
                    if (!some) store_chunk(o, c[i], cols, pack8(F32{}, d));
                    else if (c[i].on)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j >= c[i].skip) store_one(o + c[i].c0 + j, pack8(F32{}, d), j);
                }
            }
        }
    }
    if (!a.partial) return;   // neither sum wanted
    float* sums = a.partial + (int64_t)blockIdx.x * (2 * a.ld_partial);
    if constexpr (kRows == 1) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            store_chunk(sums, c[i], cols, pack8(F32{}, dg[i]));
            store_chunk(sums + a.ld_partial, c[i], cols, pack8(F32{}, db[i]));
        }
    } else {
        static_assert(kNV == 1, "rows side by side have one chunk per thread");
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
            if (c[0].on)
#pragma unroll
                for (int j = 0; j < 8; ++j) slots[slot][c[0].c0 + j] = k ? db[0][j] : dg[0][j];
            __syncthreads();
            for (int e = threadIdx.x; e < cols; e += kThreadsOf<kTPR>) {
                float v = 0.0f;
#pragma unroll
                for (int r = 0; r < kRows; ++r) v += slots[r][e];
                sums[k * a.ld_partial + e] = v;
            }
        }
    }
}

// (inputs of this many bytes are read past the caches, as in norm.hip)
[[maybe_unused]] bool past_caches(int64_t bytes) { return bytes >= (int64_t)128 << 20; }

template <class X, class H, Out kOut> struct Fwd {
    template <int kTPR, int kNV> struct Rows {
        // (rows of 4097 to 8192 columns take two chunks for each of 512 threads, as in norm.hip)
        static constexpr bool kWide = kTPR == 1024 && kNV == 1;
        static void run(const LayerNormFwdArgs& a, hipStream_t stream)
        {
            if constexpr (kWide) Rows<512, 2>::launch(a, stream);
            else launch(a, stream);
        }
        static void launch(const LayerNormFwdArgs& a, hipStream_t stream)
        {
            constexpr int kThreads = kThreadsOf<kTPR>, kRows = kThreads / kTPR;
            // (a launch has at most 2^32 threads: more rows than that take several)
            constexpr int64_t kMost = ((int64_t)1 << 31) / kThreads * kRows;
            LayerNormFwdArgs part = a;
            for (part.first_row = 0; part.first_row < a.rows; part.first_row += kMost) {
                const int64_t rows = std::min(kMost, a.rows - part.first_row);
                layernorm_fwd_kernel<X, H, kOut, kTPR, kNV>
                    <<<(unsigned)((rows + kRows - 1) / kRows), kThreads, 0, stream>>>(part);
            }
        }
    };
};

template <class X, class H, Out kOut>
hipError_t fwd_rows(const LayerNormFwdArgs& a, hipStream_t stream)
{
    by_cols<Fwd<X, H, kOut>::template Rows>(a, stream);
    return hipGetLastError();
}

template <class X, class H>
hipError_t fwd_out(const LayerNormFwdArgs& a, hipStream_t stream)
{
    switch (a.out) {
    case NormOut::Bf16: return fwd_rows<X, H, Out::Bf16>(a, stream);
    case NormOut::F32: return fwd_rows<X, H, Out::F32>(a, stream);
    default: return fwd_rows<X, H, Out::Fp8>(a, stream);
    }
}

template <class X>
hipError_t fwd_res(const LayerNormFwdArgs& a, hipStream_t stream)
{
    if (!a.res) return fwd_out<X, NoResidual>(a, stream);
    return a.h_bf16 ? fwd_out<X, Bf16>(a, stream) : fwd_out<X, F32>(a, stream);
}

template <class S, int kFmt, bool kPow2>
hipError_t transpose_run(const LayerNormFwdArgs& a, hipStream_t stream)
{
    const int64_t tiles = a.rows / kCT * ((a.cols + kCW - 1) / kCW);
    layernorm_cast_transpose_kernel<S, kFmt, kPow2><<<(unsigned)tiles, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <class S>
hipError_t fwd_transpose(const LayerNormFwdArgs& a, hipStream_t stream)
{
    if (a.fmt == FMT_E4M3)
        return a.pow2 ? transpose_run<S, FMT_E4M3, true>(a, stream) : transpose_run<S, FMT_E4M3, false>(a, stream);
    return a.pow2 ? transpose_run<S, FMT_E5M2, true>(a, stream) : transpose_run<S, FMT_E5M2, false>(a, stream);
}

template <class Y, class H, bool kRes> struct Bwd {
    template <int kTPR, int kNV> struct Rows {
        static void run(const LayerNormBwdArgs& a, hipStream_t stream)
        {
            layernorm_bwd_kernel<Y, H, kRes, kTPR, kNV><<<(unsigned)a.blocks, kThreadsOf<kTPR>, 0, stream>>>(a);
        }
    };
};

template <class Y, class H, bool kRes>
hipError_t bwd_rows(const LayerNormBwdArgs& a, hipStream_t stream)
{
    by_cols<Bwd<Y, H, kRes>::template Rows>(a, stream);
    return hipGetLastError();
}

}  // namespace

// The instantiations in units that compile side by side: forward of bf16 x (0), of fp32 x (1), the backward pass (2).
hipError_t layernorm_fwd_bf16(const LayerNormFwdArgs& a, hipStream_t stream);
hipError_t layernorm_fwd_f32(const LayerNormFwdArgs& a, hipStream_t stream);

#if TE_LAYERNORM_PART < 0 || TE_LAYERNORM_PART == 1
hipError_t layernorm_fwd_f32(const LayerNormFwdArgs& a, hipStream_t stream) { return fwd_res<F32>(a, stream); }
#endif

#if TE_LAYERNORM_PART < 0 || TE_LAYERNORM_PART == 0
hipError_t layernorm_fwd_bf16(const LayerNormFwdArgs& a, hipStream_t stream) { return fwd_res<Bf16>(a, stream); }

hipError_t launch_layernorm_fwd(const LayerNormFwdArgs& args, hipStream_t stream)
{
    LayerNormFwdArgs a = args;
    if (a.rows <= 0) return hipSuccess;
    a.inv_cols = 1.0 / a.cols;
    if (a.qt && a.rows / kCT * ((a.cols + kCW - 1) / kCW) >= ((int64_t)1 << 32) / kThreads) return hipErrorInvalidValue;
    a.past = a.cols >= 8 && past_caches(a.rows * a.cols * ((a.x_bf16 ? 2 : 4) + (a.res ? a.h_bf16 ? 2 : 4 : 0)));
    hipError_t e = hipSuccess;
    // (the transposed cast alone needs h and the row's numbers too)
    e = a.x_bf16 ? layernorm_fwd_bf16(a, stream) : layernorm_fwd_f32(a, stream);
    if (e != hipSuccess || !a.qt) return e;
    return a.src_bf16 ? fwd_transpose<Bf16>(a, stream) : fwd_transpose<F32>(a, stream);
}
#endif

#if TE_LAYERNORM_PART < 0 || TE_LAYERNORM_PART == 2
int64_t layernorm_bwd_blocks(int64_t rows, int64_t cols)
{
    const int tpr = threads_per_row(cols), threads = std::max(tpr, 256);
    const int64_t per = threads / tpr;
    return std::min<int64_t>((rows + per - 1) / per, device_cus() * (1024 / threads));
}

hipError_t launch_layernorm_bwd(const LayerNormBwdArgs& args, hipStream_t stream)
{
    LayerNormBwdArgs a = args;
    a.inv_cols = 1.0f / (float)a.cols;
    hipError_t e = hipSuccess;
    if (a.blocks > 0) {
#define TE_BWD(Y, H) (a.dres ? bwd_rows<Y, H, true>(a, stream) : bwd_rows<Y, H, false>(a, stream))
        if (a.dy_bf16) e = a.h_bf16 ? TE_BWD(Bf16, Bf16) : TE_BWD(Bf16, F32);
        else e = a.h_bf16 ? TE_BWD(F32, Bf16) : TE_BWD(F32, F32);
#undef TE_BWD
    }
    if (e != hipSuccess || (!a.dgamma && !a.dbeta)) return e;
    // (both sums in one launch, or the one that is wanted)
    const float* from = a.dgamma ? a.partial : a.partial + a.ld_partial;
    const dim3 grid((unsigned)((a.cols + kRedCols - 1) / kRedCols), a.dgamma && a.dbeta ? 2 : 1);
    column_sum_kernel<<<grid, kThreads, 0, stream>>>(from, a.blocks, 2 * a.ld_partial, a.cols, a.dgamma ? a.dgamma : a.dbeta,
                                                     a.ld_partial, a.dbeta);
    return hipGetLastError();
}
#endif

}  // namespace tefp8
