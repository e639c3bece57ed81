// Gated feed-forward products for gfx950:
//
//   forward   z = x w^T,  y = act(gate) * up
//   dgrad     D = dy wt^T,  dz = (D * up * act'(gate), D * act(gate))
//
// on the block-scaled fp8 GEMM of gemm.hip, whose tiles, copies and K loop the kernel of large products runs (the file is
// included for its device code; no part of its own entry points is compiled here).  Gate and up features alternate in blocks of
// 16 rows of w, the width of a matrix-core tile, so a wave's 4 x 8 accumulator tiles hold gate and up of the same 64
// features in the same lanes: the gated product is formed in registers, and a workgroup's 256 x 256 tile of z is a
// 256 x 128 tile of y.  The data gradient's tile has 256 x 256 values of D and twice as many of dz: it is written in
// two halves of the wave's column groups, each of which is one 128-column group of dz (the fp8 cast's unit).
//
// Formulas: with s = 1 / (1 + exp(-u)), u = g (SiLU) or 2 c (g + a g^3) (the tanh form of GELU),
//   act = g s,  act' = s (1 + g (1 - s) u')
//
// 8192 rows, 4096 -> 14336, SiLU: forward with z in bf16 1008 us (1.91 PFLOP/s; gemm.hip's plain product of that size 1001:
// the epilogue hides), in e4m3 in both layouts 1063; with FAST on power-of-two scales 896 and 941 (the plain product 882).
// Data gradient to e5m2 in both layouts 709 us: 496 of products (gemm.hip's of that size), and the 940 MB of z and dz behind
// each tile, where every workgroup asks memory at once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#define TE_GEMM_PART 100   // none of gemm.hip's host parts
#include "gemm.hip"

#include "block_internal.h"

#ifndef TE_GATED_PART
#define TE_GATED_PART -1
#endif

namespace tefp8 {
namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

template <int kAct>
__device__ __forceinline__ float sigma(float g)
{
    // exp(-u) = exp2(arg); an infinite one gives s = 0, as it should
    const float arg = kAct == (int)Act::Silu ? -kLog2e * g : gelu_exp2_arg(g);
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(arg));
}
// act(g) * up
template <int kAct>
__device__ __forceinline__ float gated(float g, float up) { return g * sigma<kAct>(g) * up; }

// (d act'(g) up, d act(g)); 1 - s loses nothing that counts (where s is near 1, so is act'), and g s is formed first,
// so that a large negative g gives 0
template <int kAct>
__device__ __forceinline__ void gated_grad(float d, float g, float up, float& dg, float& du)
{
    const float s = sigma<kAct>(g), a = g * s;
    float t = a * (1.0f - s);
    if (kAct == (int)Act::Gelu) t *= 2.0f * kGeluC * fmaf(3.0f * kGeluA, fminf(g * g, 0x1p100f), 1.0f);
    dg = d * up * (s + t);
    du = d * a;
}

// max |v| that keeps NaN
__device__ __forceinline__ float amax_of(float amax, float v) { return __builtin_elementwise_maximum(amax, fabsf(v)); }
__device__ __forceinline__ float max_bits(float a, float b)   // of numbers without a sign
{
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}
template <int kCtrl>
__device__ __forceinline__ float dpp_max_bits(float v)
{
    return max_bits(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), kCtrl, 0xF, 0xF, false)));
}
[[maybe_unused]] __device__ __forceinline__ float row16_max_bits(float v)
{
    v = dpp_max_bits<kDppQuadXor1>(v);
    v = dpp_max_bits<kDppQuadXor2>(v);
    v = dpp_max_bits<kDppRowHalfMirror>(v);
    return dpp_max_bits<kDppRowMirror>(v);
}
// A group that holds what is not finite stands for NaN: its scale says so, codes cannot.
template <int kFmtQ>
__device__ __forceinline__ void group_scale_of(const GemmArgs& p, float amax, float& scale, float& mult)
{
    if (p.q_pow2) group_scale<kFmtQ, true>(amax, scale, mult);
    else group_scale<kFmtQ, false>(amax, scale, mult);
    if (!(amax < __builtin_inff())) scale = __builtin_nanf("");
}

// Two neighbouring column groups' registers, exchanged so that each lane has eight consecutive columns: those of
// group (q4 & 1), from 8 (q4 >> 1) on.
[[maybe_unused]] __device__ __forceinline__ void pair(const v4f& v0, const v4f& v1, float (&v)[8])
{
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const auto sw = __builtin_amdgcn_permlane16_swap(__float_as_uint(v0[c]), __float_as_uint(v1[c]), false, false);
        v[c] = __uint_as_float(sw[0]);
        v[4 + c] = __uint_as_float(sw[1]);
    }
}

// The 64 rows from mw on of a row-major array, as a buffer whose range ends behind the last valid row (at once, if `in` is
// not set): loads past it give 0 and stores nothing, with no branch around each.  (Row strides are below 64 MiB.)
struct Rows {
    __amdgpu_buffer_rsrc_t r;
    uint32_t ld;   // bytes
    __device__ __forceinline__ Rows(const void* base, int64_t mw, int64_t M, int64_t ld_bytes, int64_t column_bytes, bool in)
        : ld((uint32_t)ld_bytes)
    {
        const int64_t rows = in ? max(min(M - mw, (int64_t)kWM), (int64_t)0) : 0;
        r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(base)) + mw * ld_bytes + column_bytes, 0,
                                              (int)(uint32_t)(rows * ld_bytes), 0x00020000);
    }
    // Byte `at` of row `row`.
    __device__ __forceinline__ u32x4_t load16(uint32_t row, uint32_t at, uint32_t uniform = 0) const
    {
        return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, row * ld + at, uniform, 0));
    }
    template <bool kStream = false>
    __device__ __forceinline__ void store16(uint32_t row, uint32_t at, u32x4_t v) const
    {
        __builtin_amdgcn_raw_buffer_store_b128(v, r, row * ld + at, 0, kStream ? 2 : 0);
    }
    __device__ __forceinline__ void store8(uint32_t row, uint32_t at, uint32_t v0, uint32_t v1, uint32_t uniform = 0) const
    {
        __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{v0, v1}, r, row * ld + at, uniform, 0);
    }
    __device__ __forceinline__ void store4(uint32_t at, float v) const
    {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, at, 0, 0);
    }
};
__device__ __forceinline__ u32x4_t pack_bf16x8(const float (&v)[8])
{
    return u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}
constexpr uint32_t kNowhere = 0xFFFFFFF0u;   // past every range

// ------------------------------------------------------------ casts of a tile
// Four values of a group, times its multiplier FP8_MAX / amax: at most FP8_MAX (1 + 2^-23), which rounds to FP8_MAX, so
// there is nothing to clamp (two of three instructions of encode4 in gemm.hip).
template <int kFmtQ>
__device__ __forceinline__ uint32_t encode_scaled(const v4f& v, float mult)
{
    int w;
    if (kFmtQ == FMT_E4M3) {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * mult, v[1] * mult, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * mult, v[3] * mult, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(v[0] * mult, v[1] * mult, 0, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(v[2] * mult, v[3] * mult, w, true);
    }
    return (uint32_t)w;
}
// The row-wise cast of kJ column groups of one row in accumulator layout, from the buffer's column 0 on.
template <int kFmtQ, int kJ>
__device__ __forceinline__ void store_codes(const Rows& q, const v4f (&v)[kJ], float mult, uint32_t row, int q4)
{
#pragma unroll
    for (int jp = 0; jp < kJ / 2; ++jp) {
        const auto sw = __builtin_amdgcn_permlane16_swap(encode_scaled<kFmtQ>(v[2 * jp], mult), encode_scaled<kFmtQ>(v[2 * jp + 1], mult),
                                                         false, false);
        q.store8(row, (2 * jp + (q4 & 1)) * 16 + (q4 >> 1) * 8, sw[0], sw[1]);
    }
}

// A wave's 128 columns, one group of each row.
template <int kFmtQ>
__device__ __forceinline__ void cast_rows128(const GemmArgs& p, const v4f (&v)[kTM][kTN], int64_t mw, int64_t n, bool in, int lane)
{
    const int r16 = lane & 15, q4 = lane >> 4;
    const Rows q(p.q_out, mw, p.M, p.ld_q, n, in);
    const Rows s(p.q_scales + (n / 128) * p.ld_qs, mw, p.M, 4, 0, in);
#pragma unroll
    for (int i = 0; i < kTM; ++i) {
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < kTN; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) amax = amax_of(amax, v[i][j][c]);
        amax = max_bits(amax, __shfl_xor(amax, 16));
        amax = max_bits(amax, __shfl_xor(amax, 32));
        float scale, mult;
        group_scale_of<kFmtQ>(p, amax, scale, mult);
        store_codes<kFmtQ, kTN>(q, v[i], mult, i * 16 + r16, q4);
        s.store4(q4 == 0 ? (i * 16 + r16) * 4 : kNowhere, scale);
    }
}

// The transposed cast of a tile of 256 rows: the waves (wm, wn) hold 64 rows x kJ column groups each, the columns of
// wn from first + wn * stride on.  The column maxima of a 128-row group meet in LDS (X), the multipliers come back
// through Y, and the codes go through T (64 rows of a column: 16 dwords, dword r16 holds rows 16 i + r16 in byte i) so
// that a thread stores runs of 64 rows.  In two halves, so that the caller can start loads when the values are spent:
// codes() leaves them in T, store() writes them out.  T may be written again after the first barrier of the next
// codes(); `xs` has room for T, `xy` for X and Y.
template <int kFmtQ, int kJ>
struct ColumnCast {
    static constexpr int kW = kJ * 16, kPer = kW / 64;   // columns of a wave, and of a lane for the scales

    static __device__ __forceinline__ void codes(const GemmArgs& p, const v4f (&v)[kTM][kJ], int64_t m0, int64_t first, int64_t stride,
                                                 int64_t cols, uint8_t* xs, uint8_t* xy, int wave, int lane)
    {
        asm volatile("" : "+v"(lane));                // (recomputed here: not held across the K loop)
        const int wm = wave / kWavesN, wn = wave % kWavesN;
        const int r16 = lane & 15, q4 = lane >> 4;
        float* X = reinterpret_cast<float*>(xy);                     // [kWaves][kW] column maxima
        float* Y = reinterpret_cast<float*>(xy + kWaves * kW * 4);   // [kWaves][kW] multipliers
        uint32_t* T = reinterpret_cast<uint32_t*>(xs);               // [kWavesN * kW][kWavesM][16]
        const int64_t mg = m0 + (wm >> 1) * 128;      // this wave pair's 128-row group
        const int64_t nw = first + wn * stride;
        const bool live = mg < p.M && nw < cols;      // (M and cols are whole groups)
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            float cm[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float a = amax_of(fabsf(v[0][j][c]), v[1][j][c]);
                a = amax_of(amax_of(a, v[2][j][c]), v[3][j][c]);
                cm[c] = row16_max_bits(a);
            }
            if (r16 == 0) *reinterpret_cast<float4*>(X + wave * kW + j * 16 + q4 * 4) = make_float4(cm[0], cm[1], cm[2], cm[3]);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int col = u * 64 + lane;
            float s, mu;
            group_scale_of<kFmtQ>(p, max_bits(X[wave * kW + col], X[(wave ^ kWavesN) * kW + col]), s, mu);
            Y[wave * kW + col] = mu;
            if ((wm & 1) == 0 && live) p.qt_scales[(mg / 128) * p.ld_qts + nw + col] = s;
        }
        // (the multipliers were written by this wave: its LDS reads see them in order)
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const v4f mu = *reinterpret_cast<const v4f*>(Y + wave * kW + j * 16 + q4 * 4);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                T[((wn * kW + j * 16 + q4 * 4 + c) * kWavesM + wm) * 16 + r16] =
                    encode_scaled<kFmtQ>(v4f{v[0][j][c], v[1][j][c], v[2][j][c], v[3][j][c]}, mu[c]);
        }
    }
    static __device__ __forceinline__ void store(const GemmArgs& p, int64_t m0, int64_t first, int64_t stride, int64_t cols, uint8_t* xs)
    {
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const uint32_t* T = reinterpret_cast<const uint32_t*>(xs);
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kJ / 4; ++h) {
            const int k = tid + h * kThreads;   // 0 .. kWavesN * kW * kWavesM - 1
            const int nt = k / kWavesM, w = k % kWavesM;
            const int64_t n = first + (nt / kW) * stride + nt % kW, m = m0 + w * kWM;
            const uint4* src = reinterpret_cast<const uint4*>(T + k * 16);
            uint32_t o[16];
#pragma unroll
            for (int g = 0; g < 4; ++g) {   // byte i of dwords 4 g .. 4 g + 3 to output dword 4 i + g
                const uint4 d = src[g];
                const uint32_t ab_lo = __builtin_amdgcn_perm(d.y, d.x, 0x05010400u);
                const uint32_t ab_hi = __builtin_amdgcn_perm(d.y, d.x, 0x07030602u);
                const uint32_t cd_lo = __builtin_amdgcn_perm(d.w, d.z, 0x05010400u);
                const uint32_t cd_hi = __builtin_amdgcn_perm(d.w, d.z, 0x07030602u);
                o[0 * 4 + g] = __builtin_amdgcn_perm(cd_lo, ab_lo, 0x05040100u);
                o[1 * 4 + g] = __builtin_amdgcn_perm(cd_lo, ab_lo, 0x07060302u);
                o[2 * 4 + g] = __builtin_amdgcn_perm(cd_hi, ab_hi, 0x05040100u);
                o[3 * 4 + g] = __builtin_amdgcn_perm(cd_hi, ab_hi, 0x07060302u);
            }
            if (n < cols && m < p.M) {
                uint8_t* dst = p.qt_out + n * p.ld_qt + m;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<uint4*>(dst + 16 * r) = make_uint4(o[4 * r], o[4 * r + 1], o[4 * r + 2], o[4 * r + 3]);
            }
        }
    }
};
constexpr int kXyBytes = 2 * kWaves * kWN * 4;   // X and Y of a wave's 128 columns

// ------------------------------------------------------------ forward epilogue
// kJ column groups of z from column n on (gate and up in turn), rows mw ..; kQuant: 0 y in bf16 or fp32, 1 its row-wise
// cast, 2 the transposed one and, if wanted, the row-wise one.  A row's 128 features are those of both waves along N.
template <int kAct, int kQuant, int kFmtQ, int kJ>
__device__ __forceinline__ void forward_epilogue(const GemmArgs& p, v4f (&acc)[kTM][kJ], int64_t m0, int64_t mw, int64_t n, uint8_t* xs,
                                                 uint8_t* xy, int wave, int lane)
{
    asm volatile("" : "+v"(lane));
    const int r16 = lane & 15, q4 = lane >> 4;
    const uint32_t run = (q4 & 1) * 16 + (q4 >> 1) * 8;   // first of the lane's eight columns of a pair of groups
    constexpr int kF = kJ / 2;   // groups of features
    if (p.aux) {
        const Rows z(p.aux, mw, p.M, p.ld_aux * 2, n * 2, true);
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
            for (int f = 0; f < kF; ++f) {
                float v[8];
                pair(acc[i][2 * f], acc[i][2 * f + 1], v);
                z.store16<true>(i * 16 + r16, (f * 32 + run) * 2, pack_bf16x8(v));   // (streamed, as gemm.hip's pre-activation)
            }
    }
    const int64_t nf = n / 2;    // first feature
    v4f y[kTM][kF];
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
        for (int f = 0; f < kF; ++f) {
            const v4f g = acc[i][2 * f], u = acc[i][2 * f + 1];
            y[i][f] = v4f{gated<kAct>(g[0], u[0]), gated<kAct>(g[1], u[1]), gated<kAct>(g[2], u[2]), gated<kAct>(g[3], u[3])};
        }
    if constexpr (kQuant == 0) {
        const int size = p.out_bf16 ? 2 : 4;
        const Rows o(p.out, mw, p.M, p.ld_out * size, nf * size, true);
        if (p.out_bf16) {
#pragma unroll
            for (int i = 0; i < kTM; ++i) {
                if constexpr (kF % 2 == 0) {
#pragma unroll
                    for (int fp = 0; fp < kF / 2; ++fp) {
                        float v[8];
                        pair(y[i][2 * fp], y[i][2 * fp + 1], v);
                        o.store16(i * 16 + r16, (fp * 32 + run) * 2, pack_bf16x8(v));
                    }
                } else {
#pragma unroll
                    for (int f = 0; f < kF; ++f)
                        o.store8(i * 16 + r16, (f * 16 + q4 * 4) * 2, pack_bf16x2(y[i][f][0], y[i][f][1]), pack_bf16x2(y[i][f][2], y[i][f][3]));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kTM; ++i)
#pragma unroll
                for (int f = 0; f < kF; ++f) o.store16(i * 16 + r16, (f * 16 + q4 * 4) * 4, __builtin_bit_cast(u32x4_t, y[i][f]));
        }
        return;
    } else {
        static_assert(kJ == kTN, "a wave of the 256 x 256 tile");
        const int wm = wave / kWavesN, wn = wave % kWavesN;
        if constexpr (kQuant == 2) {
            typedef ColumnCast<kFmtQ, kF> Cast;
            Cast::codes(p, y, m0, nf - wn * (kWN / 2), kWN / 2, p.N / 2, xs, xy, wave, lane);
            Cast::store(p, m0, nf - wn * (kWN / 2), kWN / 2, p.N / 2, xs);
            if (!p.q_out) return;
        }
        float* A = reinterpret_cast<float*>(xy);   // [kWavesN][kBM] maxima of 64 features (X and Y are read)
        float amax[kTM];
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
            float a = 0.0f;
#pragma unroll
            for (int f = 0; f < kF; ++f)
#pragma unroll
                for (int c = 0; c < 4; ++c) a = amax_of(a, y[i][f][c]);
            a = max_bits(a, __shfl_xor(a, 16));
            amax[i] = max_bits(a, __shfl_xor(a, 32));
            if (q4 == 0) A[wn * kBM + wm * kWM + i * 16 + r16] = amax[i];
        }
        __syncthreads();
        const Rows q(p.q_out, mw, p.M, p.ld_q, nf, true);
        const Rows s(p.q_scales + (nf / 128) * p.ld_qs, mw, p.M, 4, 0, wn == 0);
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
            float scale, mult;
            group_scale_of<kFmtQ>(p, max_bits(amax[i], A[(wn ^ 1) * kBM + wm * kWM + i * 16 + r16]), scale, mult);
            store_codes<kFmtQ, kF>(q, y[i], mult, i * 16 + r16, q4);
            s.store4(q4 == 0 ? (i * 16 + r16) * 4 : kNowhere, scale);
        }
    }
}

// ------------------------------------------------------------ data gradient's epilogue
// dz of the lane's four values of D's column group j and one row; z: the 16-byte run of z's columns 32 j + run .. that
// the lane has loaded, exchanged as in pair() for the gate and up values of its own columns.
template <int kAct>
__device__ __forceinline__ void grad4(const v4f& d, const u32x4_t& z, v4f& dg, v4f& du)
{
    const auto lo = __builtin_amdgcn_permlane16_swap(z[0], z[2], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(z[1], z[3], false, false);
    const uint32_t g[2] = {(uint32_t)lo[0], (uint32_t)hi[0]}, u[2] = {(uint32_t)lo[1], (uint32_t)hi[1]};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float a, b;
        gated_grad<kAct>(d[c], __uint_as_float(c & 1 ? g[c >> 1] & 0xFFFF0000u : g[c >> 1] << 16),
                         __uint_as_float(c & 1 ? u[c >> 1] & 0xFFFF0000u : u[c >> 1] << 16), a, b);
        dg[c] = a;
        du[c] = b;
    }
}

// kJ column groups of D from column n on, rows mw .., to dz in bf16 or fp32.
template <int kAct, int kJ>
__device__ __forceinline__ void dgrad_store(const GemmArgs& p, const v4f (&acc)[kTM][kJ], int64_t mw, int64_t n, int lane)
{
    asm volatile("" : "+v"(lane));
    const int r16 = lane & 15, q4 = lane >> 4;
    const uint32_t run = (q4 & 1) * 16 + (q4 >> 1) * 8;
    const bool in = n < p.N;
    const int size = p.out_bf16 ? 2 : 4;
    const Rows zr(p.preact, mw, p.M, p.ld_aux * 2, 4 * n, in), o(p.out, mw, p.M, p.ld_out * size, 2 * n * size, in);
    // (the runs of z a group ahead of their use, before the stores in between: a load behind a store is waited for
    // with it)
    u32x4_t z[2][kTM];
#pragma unroll
    for (int i = 0; i < kTM; ++i) z[0][i] = zr.load16(i * 16 + r16, run * 2);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        if (j + 1 < kJ) {
#pragma unroll
            for (int i = 0; i < kTM; ++i) z[(j + 1) & 1][i] = zr.load16(i * 16 + r16, ((j + 1) * 32 + run) * 2);
        }
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
            v4f dg, du;
            grad4<kAct>(acc[i][j], z[j & 1][i], dg, du);
            if (p.out_bf16) {
                float v[8];
                pair(dg, du, v);
                o.store16(i * 16 + r16, (j * 32 + run) * 2, pack_bf16x8(v));
            } else {
                o.store16(i * 16 + r16, (j * 32 + q4 * 4) * 4, __builtin_bit_cast(u32x4_t, dg));
                o.store16(i * 16 + r16, (j * 32 + 16 + q4 * 4) * 4, __builtin_bit_cast(u32x4_t, du));
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// The casts of a wave's dz: half h of its column groups gives 128 columns of dz, one group of each row.  A half's z and
// D together fill the registers that its dz takes, so all of its z is loaded at once, the second half's while the
// first half's codes are stored.  The halves are a loop (the second's D moves to the first's place): unrolled, the code
// of a tile would pass the instruction cache.
template <int kAct, int kQuant, int kFmtQ>
__device__ __forceinline__ void dgrad_casts(const GemmArgs& p, v4f (&acc)[kTM][kTN], int64_t m0, int64_t mw, int64_t n0, int64_t n,
                                            uint8_t* xs, uint8_t* xy, int wave, int lane)
{
    asm volatile("" : "+v"(lane));
    const int r16 = lane & 15, q4 = lane >> 4;
    const uint32_t run = (q4 & 1) * 16 + (q4 >> 1) * 8;
    const bool in = n < p.N;
    constexpr int kJ = kTN / 2;
    typedef ColumnCast<kFmtQ, kTN> Cast;
    const Rows zr(p.preact, mw, p.M, p.ld_aux * 2, 4 * n, in);
    u32x4_t z[kTM][kJ];
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j) z[i][j] = zr.load16(i * 16 + r16, (j * 32 + run) * 2);
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        v4f v[kTM][kTN];
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                grad4<kAct>(acc[i][j], z[i][j], v[i][2 * j], v[i][2 * j + 1]);
                __builtin_amdgcn_sched_barrier(0);   // (each in the registers of what it was made from)
            }
        if (p.q_out) cast_rows128<kFmtQ>(p, v, mw, 2 * n + h * 128, in, lane);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (kQuant == 2) Cast::codes(p, v, m0, 2 * n0 + h * 128, 2 * kWN, 2 * p.N, xs, xy, wave, lane);
        __builtin_amdgcn_sched_barrier(0);
        // (the second half's; the first's once more behind it would read past the tile's columns: nothing is loaded)
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                z[i][j] = zr.load16(h == 0 ? i * 16 + r16 : kWM, (j * 32 + run) * 2, kJ * 32 * 2);
                acc[i][j] = acc[i][j + kJ];
            }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (kQuant == 2) Cast::store(p, m0, 2 * n0 + h * 128, 2 * kWN, 2 * p.N, xs);
    }
}

// ------------------------------------------------------------ kernels
// gemm.hip's persistent kernel with the epilogues above.
template <int kFmtA, int kFmtB, bool kFast, bool kFwd, int kAct, int kQuant, int kFmtQ>
__global__ __launch_bounds__(kThreads) void gated_kernel(const GemmArgs p, int64_t total_tiles)
{
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStageBytes + kWaves * 4 + (kQuant ? kXyBytes : 0)];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t G = gridDim.x;
    const int64_t per_xcd = G / kXcds;
    int64_t tile = blockIdx.x;
    if (tile < per_xcd * kXcds) tile = (tile % kXcds) * per_xcd + tile / kXcds;

    const LaneOff o = lane_offsets(wave, lane);
    int s0_off = 0, s1_off = kStageBytes;
    asm volatile("" : "+s"(s0_off), "+s"(s1_off));
    uint32_t* slots = reinterpret_cast<uint32_t*>(smem + 2 * kStageBytes);

    TileCtx c = tile_ctx(p, tile);
    load_stage(p, c.src, smem + s0_off, c.kb0, wave, lane);
    bool ok = kFast ? row_scales_pow2(p, c) : false;
    for (;;) {
        const bool chain = kFast && workgroup_all(ok, slots, wave, lane);
        stage_barrier();
        load_stage_a_scales(p, select_src(c.src, c.nkb > 1), smem + s1_off, c.kb0 + 1, wave, lane);
        v4f acc[kTM][kTN];
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
            for (int j = 0; j < kTN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
        if (chain) main_loop<true, kFmtA, kFmtB>(p, smem + s0_off, smem + s1_off, acc, o, c.src, c.kb0, c.nkb, wave, lane);
        else main_loop<false, kFmtA, kFmtB>(p, smem + s0_off, smem + s1_off, acc, o, c.src, c.kb0, c.nkb, wave, lane);
        // every wave is done reading the stages: start the next tile's copies, then write this tile out
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        const int64_t next = tile + G;
        const bool more = next < total_tiles;
        TileCtx cn = c;
        if (more) {
            cn = tile_ctx(p, next);
            load_stage(p, cn.src, smem + s0_off, cn.kb0, wave, lane);
        }
        uint8_t* xs = smem + s1_off;   // (the stage that the next tile's first copies do not use)
        uint8_t* xy = smem + 2 * kStageBytes + kWaves * 4;
        const int64_t mw = c.m0 + wave / kWavesN * kWM, n = c.n0 + wave % kWavesN * kWN;
        if constexpr (kFwd) forward_epilogue<kAct, kQuant, kFmtQ, kTN>(p, acc, c.m0, mw, n, xs, xy, wave, lane);
        else if constexpr (kQuant == 0) dgrad_store<kAct, kTN>(p, acc, mw, n, lane);
        else dgrad_casts<kAct, kQuant, kFmtQ>(p, acc, c.m0, mw, c.n0, n, xs, xy, wave, lane);
        if (!more) break;
        if (kFast) ok = row_scales_pow2(p, cn);
        tile = next;
        c = cn;
    }
}

// ------------------------------------------------------------ parts of 64 x 128
// For few tiles: a workgroup has one 64 x 128 part of the product, its wave w the column groups 2 w and 2 w + 1 (16
// features of the forward), with the same sums as in a tile.  Two blocks are on their way, one is read from
// LDS into registers and one, in registers, multiplied.  Few waves are there to hide anything, so the loop holds no branch
// and no wait that another wave's work would have to fill: each wave issues the same seven copies a block (two of a, four
// of b, one run of scales), and the products stand between the LDS reads of the block after theirs.  (Data gradient, 300
// rows, 4096 -> 7168: 34.9 us with the K loop of gemm.hip's wave tiles, whose copies stand behind branches; 33.4 with
// copies of the same shape; 27.8 with all of a block's products started before the first is added; 25.7 so.)
//
// Wave w's copies of one block: kilobytes w + 4 u of a and of b in a stage, and 64 scales: those of a's rows (wave 0), of
// b's first and last 64 (1, 2); wave 3's run is empty.
struct PartCopies {
    const uint8_t *a, *b;
    int a_bytes, b_bytes;
    uint32_t va[2], vb, b_step;   // this lane's byte of the wave's copies
    const float* scales;
    int64_t ld_scales;
    int scale_bytes, scale_to;
};
constexpr int kPartCopies = 7;
__device__ __forceinline__ PartCopies part_copies(const GemmArgs& p, int64_t m0, int64_t n0, int w, int lane)
{
    PartCopies s;
    s.a = p.a + m0 * p.lda;
    s.b = p.b + n0 * p.ldb;
    s.a_bytes = (int)(min((int64_t)kWM, p.M - m0) * p.lda);
    s.b_bytes = (int)(min((int64_t)kWN, p.N - n0) * p.ldb);
    const int row = w * 8 + (lane >> 3), chunk = (lane & 7) ^ ((row >> 1) & 7);   // (32 rows on the chunk is the same)
    s.va[0] = (uint32_t)(row * p.lda + chunk * 16);
    s.va[1] = s.va[0] + (uint32_t)(32 * p.lda);
    s.vb = (uint32_t)(row * p.ldb + chunk * 16);
    s.b_step = (uint32_t)(32 * p.ldb);
    const bool of_a = w == 0;
    const int64_t first = of_a ? m0 : n0 + (w == 2 ? 64 : 0);
    s.scales = (of_a ? p.sa : p.sb) + first;
    s.ld_scales = of_a ? p.lsa : p.lsb;
    s.scale_bytes = w == 3 ? 0 : (int)(min((int64_t)64, max(s.ld_scales - first, (int64_t)0)) * 4);
    s.scale_to = kVScale + (of_a ? 0 : 1024 + (w - 1) * 256);
    return s;
}
__device__ __forceinline__ void part_load(const PartCopies& s, uint8_t* stage, int kb, bool live, int w, int lane)
{
    const __amdgpu_buffer_rsrc_t a = make_rsrc(s.a, live ? s.a_bytes : 0), b = make_rsrc(s.b, live ? s.b_bytes : 0);
    const __amdgpu_buffer_rsrc_t sc = make_rsrc(s.scales + kb * s.ld_scales, live ? s.scale_bytes : 0);
#pragma unroll
    for (int u = 0; u < 2; ++u)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(a, (lds_ptr_t)(stage + (w + 4 * u) * 1024), 16, s.va[u], kb * kBK, 0, 0);
#pragma unroll
    for (int u = 0; u < 4; ++u)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_ptr_t)(stage + kVA + (w + 4 * u) * 1024), 16, s.vb + u * s.b_step, kb * kBK, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sc, (lds_ptr_t)(stage + s.scale_to), 4, (uint32_t)(lane * 4), 0, 0, 0);
}

// A block's operands and scales in registers.
template <bool kChain>
struct PartFrags {
    v8i a[kTM], b[kVJ];
    uint32_t sa[kTM], eb[kVJ];   // (eb: kChain alone, sb: otherwise)
    float4 sb[kVJ];
    __device__ __forceinline__ void read_b(const uint8_t* st, const WaveLane& o, int w)
    {
#pragma unroll
        for (int jj = 0; jj < kVJ; ++jj) {
            const int j = w * kVJ + jj;
            b[jj] = lds_frag(st, o.b_lo, o.b_hi, j * 2048);
            if (kChain) eb[jj] = lds_u32(st + kVScale + 1024 + (j * 16 + o.r16) * 4);
            else sb[jj] = lds_f32x4(st + kVScale + 1024 + (j * 16 + o.q4 * 4) * 4);
        }
    }
    __device__ __forceinline__ void read_a(const uint8_t* st, const WaveLane& o, int i)
    {
        a[i] = lds_frag(st, o.a_lo, o.a_hi, i * 2048);
        sa[i] = lds_u32(st + kVScale + (i * 16 + o.r16) * 4);
    }
};
// Row group i's products; FULL's are added by promote_all once all of a block are started.
template <bool kChain, int kFmtA, int kFmtB>
__device__ __forceinline__ void part_products(const PartFrags<kChain>& f, int i, v4f (&acc)[kTM][kVJ], v4f (&P)[kTM][kVJ])
{
#pragma unroll
    for (int jj = 0; jj < kVJ; ++jj) {
        if (kChain)
            acc[i][jj] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f.b[jj], f.a[i], acc[i][jj], kFmtB, kFmtA, 0, e8m0(f.eb[jj]), 0,
                                                                          e8m0(f.sa[i]));
        else
            P[i][jj] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f.b[jj], f.a[i], v4f{0.f, 0.f, 0.f, 0.f}, kFmtB, kFmtA, 0, 0, 0, 0);
    }
}
template <bool kChain>
__device__ __forceinline__ void promote_all(const PartFrags<kChain>& f, v4f (&acc)[kTM][kVJ], const v4f (&P)[kTM][kVJ])
{
    if (kChain) return;
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
        for (int jj = 0; jj < kVJ; ++jj) promote(acc[i][jj], P[i][jj], __uint_as_float(f.sa[i]), f.sb[jj]);
}

// The block in stage `st`: wait for this wave's copies of it, meet the other waves (all copies have landed, and all have
// read the block before, in `nx`), start the copies of block `ahead` into that one, then read this block into `f` while
// the products of the one before, `g`, are formed.
template <bool kChain, int kFmtA, int kFmtB, bool kFirst = false>
__device__ __forceinline__ void part_block(const PartCopies& s, uint8_t* st, uint8_t* nx, PartFrags<kChain>& f, const PartFrags<kChain>& g,
                                           v4f (&acc)[kTM][kVJ], const WaveLane& o, int w, int ahead, bool live, int lane)
{
    static_assert(kPartCopies == 7 && kVStages == 3, "the wait");
    asm volatile("s_waitcnt vmcnt(7) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    part_load(s, nx, ahead, live, w, lane);
    v4f P[kTM][kVJ];
    f.read_b(st, o, w);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kTM; ++i) {
        f.read_a(st, o, i);
        if (!kFirst) part_products<kChain, kFmtA, kFmtB>(g, i, acc, P);
        __builtin_amdgcn_sched_barrier(0);
    }
    if (!kFirst) promote_all<kChain>(g, acc, P);
}

// Each stage is a pointer of its own, so that its reads wait for no copy into another.  Blocks 0 and 1 are on their way on
// entry; block i is read into f0 or f1 in turn.
template <bool kChain, int kFmtA, int kFmtB>
__device__ __forceinline__ void part_loop(const PartCopies& s, uint8_t* __restrict__ s0, uint8_t* __restrict__ s1, uint8_t* __restrict__ s2,
                                          v4f (&acc)[kTM][kVJ], const WaveLane& o, int w, int nkb, int lane)
{
    PartFrags<kChain> f0, f1;
#define TE_BLOCK(i, st, nx, f, g) part_block<kChain, kFmtA, kFmtB>(s, st, nx, f, g, acc, o, w, it + i + 2, it + i + 2 < nkb, lane)
    int it = 0;
    part_block<kChain, kFmtA, kFmtB, true>(s, s0, s2, f0, f1, acc, o, w, 2, 2 < nkb, lane);
    for (it = 1; it + 6 <= nkb; it += 6) {
        TE_BLOCK(0, s1, s0, f1, f0);
        TE_BLOCK(1, s2, s1, f0, f1);
        TE_BLOCK(2, s0, s2, f1, f0);
        TE_BLOCK(3, s1, s0, f0, f1);
        TE_BLOCK(4, s2, s1, f1, f0);
        TE_BLOCK(5, s0, s2, f0, f1);
    }
    if (it < nkb) TE_BLOCK(0, s1, s0, f1, f0);
    if (it + 1 < nkb) TE_BLOCK(1, s2, s1, f0, f1);
    if (it + 2 < nkb) TE_BLOCK(2, s0, s2, f1, f0);
    if (it + 3 < nkb) TE_BLOCK(3, s1, s0, f0, f1);
    if (it + 4 < nkb) TE_BLOCK(4, s2, s1, f1, f0);
#undef TE_BLOCK
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (the empty copies write LDS too)
    v4f P[kTM][kVJ];
    const auto last = [&](const PartFrags<kChain>& f) {
#pragma unroll
        for (int i = 0; i < kTM; ++i) part_products<kChain, kFmtA, kFmtB>(f, i, acc, P);
        promote_all<kChain>(f, acc, P);
    };
    if (nkb & 1) last(f0);
    else last(f1);
}

// Every scale of the part's rows and columns is a power of two.
__device__ __forceinline__ bool part_scales_pow2(const GemmArgs& p, int64_t m0, int64_t n0, int nkb, int lane)
{
    const int rows = (int)min((int64_t)kWM, p.M - m0), cols = (int)min((int64_t)kWN, p.N - n0);
    bool ok = true;
#pragma unroll 4
    for (int kb = 0; kb < nkb; ++kb) {
        const float* a = p.sa + kb * p.lsa + m0;
        const float* b = p.sb + kb * p.lsb + n0;
        const float v = lane < rows ? a[lane] : 1.0f, x = lane < cols ? b[lane] : 1.0f, y = lane + 64 < cols ? b[lane + 64] : 1.0f;
        ok = ok && is_pow2_scale(v) && is_pow2_scale(x) && is_pow2_scale(y);
    }
    return __builtin_amdgcn_ballot_w64(!ok) == 0;
}

// Workgroups go to the XCDs in turn: each XCD takes a run of parts, down a column of parts first, so that the parts that
// read the same rows of b share an L2.
template <int kFmtA, int kFmtB, bool kFast, bool kFwd, int kAct, int kQuant, int kFmtQ>
__global__ __launch_bounds__(kVThreads) __attribute__((amdgpu_waves_per_eu(2))) void gated_part_kernel(const GemmArgs p)
{
    static_assert(kQuant == 0 || !kFwd, "a forward's part has half a group of each row");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kVStages * kVStage];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part_rows = (int)((p.M + kWM - 1) / kWM);
    const int at = (int)(blockIdx.x % kXcds * (gridDim.x / kXcds) + blockIdx.x / kXcds);
    const int64_t m0 = (int64_t)(at % part_rows) * kWM, n0 = (int64_t)(at / part_rows) * kWN;
    if (n0 >= p.N) return;
    const int nkb = p.groups[0].kb_len;
    const PartCopies s = part_copies(p, m0, n0, w, lane);
    WaveLane o;
    o.r16 = lane & 15;
    o.q4 = lane >> 4;
    o.a_lo = swz(o.r16, o.q4);
    o.a_hi = swz(o.r16, o.q4 + 4);
    o.b_lo = kVA + swz(o.r16, o.q4);
    o.b_hi = kVA + swz(o.r16, o.q4 + 4);
    int s0_off = 0, s1_off = kVStage, s2_off = 2 * kVStage;
    asm volatile("" : "+s"(s0_off), "+s"(s1_off), "+s"(s2_off));
    const bool chain = kFast && part_scales_pow2(p, m0, n0, nkb, lane);
    part_load(s, smem + s0_off, 0, 0 < nkb, w, lane);
    part_load(s, smem + s1_off, 1, 1 < nkb, w, lane);

    v4f part[kTM][kVJ];
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
        for (int jj = 0; jj < kVJ; ++jj) part[i][jj] = v4f{0.f, 0.f, 0.f, 0.f};
    if (chain) part_loop<true, kFmtA, kFmtB>(s, smem + s0_off, smem + s1_off, smem + s2_off, part, o, w, nkb, lane);
    else part_loop<false, kFmtA, kFmtB>(s, smem + s0_off, smem + s1_off, smem + s2_off, part, o, w, nkb, lane);
    if constexpr (kQuant == 0) {
        const int64_t n = n0 + w * (kVJ * 16);
        if constexpr (kFwd) forward_epilogue<kAct, 0, kFmtQ, kVJ>(p, part, m0, m0, n, smem, smem, 0, lane);
        else dgrad_store<kAct, kVJ>(p, part, m0, n, lane);
    } else {
        // Row-wise cast of the data gradient: half h of the part's column groups is one group of each row of dz; waves 2 h
        // and 2 h + 1 hold it, each 64 columns of it for the 64 rows: they share the maxima through LDS.
        const int r16 = o.r16, q4 = o.q4;
        const uint32_t run = (q4 & 1) * 16 + (q4 >> 1) * 8;
        const int64_t n = n0 + w * (kVJ * 16);
        const Rows zr(p.preact, m0, p.M, p.ld_aux * 2, 4 * n, true), q(p.q_out, m0, p.M, p.ld_q, 2 * n, true);
        const Rows sr(p.q_scales + (2 * n / 128) * p.ld_qs, m0, p.M, 4, 0, (w & 1) == 0);
        v4f v[kTM][2 * kVJ];
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
            for (int j = 0; j < kVJ; ++j)
                grad4<kAct>(part[i][j], zr.load16(i * 16 + r16, (j * 32 + run) * 2), v[i][2 * j], v[i][2 * j + 1]);
        float* A = reinterpret_cast<float*>(smem);   // [kVWaves][kWM]
        __syncthreads();   // every wave is done reading the stages
        float amax[kTM];
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
            float a = 0.0f;
#pragma unroll
            for (int j = 0; j < 2 * kVJ; ++j)
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) a = amax_of(a, v[i][j][cc]);
            a = max_bits(a, __shfl_xor(a, 16));
            amax[i] = max_bits(a, __shfl_xor(a, 32));
            if (q4 == 0) A[w * kWM + i * 16 + r16] = amax[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
            float scale, mult;
            group_scale_of<kFmtQ>(p, max_bits(amax[i], A[(w ^ 1) * kWM + i * 16 + r16]), scale, mult);
            store_codes<kFmtQ, 2 * kVJ>(q, v[i], mult, i * 16 + r16, q4);
            sr.store4(q4 == 0 ? (i * 16 + r16) * 4 : kNowhere, scale);
        }
    }
}

struct Shape {
    int64_t tiles;
    bool parts;
    dim3 grid;
};
[[maybe_unused]] Shape shape_of(const GemmArgs& a, bool parts)
{
    Shape s;
    s.tiles = ((a.M + kBM - 1) / kBM) * ((a.N + kBN - 1) / kBN);
    s.parts = parts;
    const int64_t n = ((a.M + kWM - 1) / kWM) * ((a.N + kWN - 1) / kWN);
    s.grid = dim3((unsigned)(parts ? (n + kXcds - 1) / kXcds * kXcds : std::min<int64_t>(s.tiles, device_cus())));
    return s;
}

template <int kFmtA, int kFmtB, bool kFast, bool kFwd, int kAct, int kQuant, int kFmtQ>
hipError_t run_tiles(const GemmArgs& a, const Shape& s, hipStream_t stream)
{
    gated_kernel<kFmtA, kFmtB, kFast, kFwd, kAct, kQuant, kFmtQ><<<s.grid, kThreads, 0, stream>>>(a, s.tiles);
    return hipGetLastError();
}
template <int kFmtA, int kFmtB, bool kFast, bool kFwd, int kAct, int kQuant, int kFmtQ>
hipError_t run_parts(const GemmArgs& a, const Shape& s, hipStream_t stream)
{
    gated_part_kernel<kFmtA, kFmtB, kFast, kFwd, kAct, kQuant, kFmtQ><<<s.grid, kVThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <int kFmtA, int kFmtB, bool kFast, int kAct>
hipError_t forward_act(const GemmArgs& a, const Shape& s, hipStream_t stream)
{
    const bool e4 = a.q_fmt == FMT_E4M3;
    if (s.parts) return run_parts<kFmtA, kFmtB, kFast, true, kAct, 0, 0>(a, s, stream);
    if (a.qt_out)
        return e4 ? run_tiles<kFmtA, kFmtB, kFast, true, kAct, 2, FMT_E4M3>(a, s, stream)
                  : run_tiles<kFmtA, kFmtB, kFast, true, kAct, 2, FMT_E5M2>(a, s, stream);
    if (a.q_out)
        return e4 ? run_tiles<kFmtA, kFmtB, kFast, true, kAct, 1, FMT_E4M3>(a, s, stream)
                  : run_tiles<kFmtA, kFmtB, kFast, true, kAct, 1, FMT_E5M2>(a, s, stream);
    return run_tiles<kFmtA, kFmtB, kFast, true, kAct, 0, 0>(a, s, stream);
}
template <int kFmtA, int kFmtB>
hipError_t forward(const GemmArgs& a, bool parts, hipStream_t stream)
{
    const Shape s = shape_of(a, parts);
    const bool silu = a.flags == (uint32_t)Act::Silu;
    // (power-of-two scales, on which FAST chains the blocks, are a choice for e4m3 operands; other pairs run FULL's
    // update, which FAST's result is on any other scales too)
    if constexpr (kFmtA == FMT_E4M3 && kFmtB == FMT_E4M3) {
        if (a.fast)
            return silu ? forward_act<kFmtA, kFmtB, true, (int)Act::Silu>(a, s, stream)
                        : forward_act<kFmtA, kFmtB, true, (int)Act::Gelu>(a, s, stream);
    }
    return silu ? forward_act<kFmtA, kFmtB, false, (int)Act::Silu>(a, s, stream)
                : forward_act<kFmtA, kFmtB, false, (int)Act::Gelu>(a, s, stream);
}
template <int kFmtA, int kFmtB, int kAct>
hipError_t dgrad_act(const GemmArgs& a, const Shape& s, hipStream_t stream)
{
    const bool e4 = a.q_fmt == FMT_E4M3;
    if (s.parts) {
        if (!a.q_out) return run_parts<kFmtA, kFmtB, false, false, kAct, 0, 0>(a, s, stream);
        return e4 ? run_parts<kFmtA, kFmtB, false, false, kAct, 1, FMT_E4M3>(a, s, stream)
                  : run_parts<kFmtA, kFmtB, false, false, kAct, 1, FMT_E5M2>(a, s, stream);
    }
    if (a.qt_out)
        return e4 ? run_tiles<kFmtA, kFmtB, false, false, kAct, 2, FMT_E4M3>(a, s, stream)
                  : run_tiles<kFmtA, kFmtB, false, false, kAct, 2, FMT_E5M2>(a, s, stream);
    if (a.q_out)
        return e4 ? run_tiles<kFmtA, kFmtB, false, false, kAct, 1, FMT_E4M3>(a, s, stream)
                  : run_tiles<kFmtA, kFmtB, false, false, kAct, 1, FMT_E5M2>(a, s, stream);
    return run_tiles<kFmtA, kFmtB, false, false, kAct, 0, 0>(a, s, stream);
}
template <int kFmtA, int kFmtB>
hipError_t dgrad(const GemmArgs& a, bool parts, hipStream_t stream)
{
    const Shape s = shape_of(a, parts);
    return a.flags == (uint32_t)Act::Silu ? dgrad_act<kFmtA, kFmtB, (int)Act::Silu>(a, s, stream)
                                          : dgrad_act<kFmtA, kFmtB, (int)Act::Gelu>(a, s, stream);
}

}  // namespace

// One unit for each pair of operand formats and direction (0-3 forward, 4-7 data gradient), and one for the host side (8).
#define TE_GATED_PAIRS(F) F(0, e4_e4, FMT_E4M3, FMT_E4M3) F(1, e5_e4, FMT_E5M2, FMT_E4M3) F(2, e4_e5, FMT_E4M3, FMT_E5M2) F(3, e5_e5, FMT_E5M2, FMT_E5M2)
#define TE_GATED_DECLARE(n, pair, A, B)                                                   \
    hipError_t gated_forward_##pair(const GemmArgs& a, bool parts, hipStream_t stream);    \
    hipError_t gated_dgrad_##pair(const GemmArgs& a, bool parts, hipStream_t stream);
TE_GATED_PAIRS(TE_GATED_DECLARE)
#define TE_GATED_FORWARD(pair, A, B)                                                                            \
    hipError_t gated_forward_##pair(const GemmArgs& a, bool parts, hipStream_t stream)                           \
    {                                                                                                           \
        return forward<A, B>(a, parts, stream);                                                                  \
    }
#define TE_GATED_DGRAD(pair, A, B) \
    hipError_t gated_dgrad_##pair(const GemmArgs& a, bool parts, hipStream_t stream) { return dgrad<A, B>(a, parts, stream); }
#if TE_GATED_PART < 0 || TE_GATED_PART == 0
TE_GATED_FORWARD(e4_e4, FMT_E4M3, FMT_E4M3)
#endif
#if TE_GATED_PART < 0 || TE_GATED_PART == 1
TE_GATED_FORWARD(e5_e4, FMT_E5M2, FMT_E4M3)
#endif
#if TE_GATED_PART < 0 || TE_GATED_PART == 2
TE_GATED_FORWARD(e4_e5, FMT_E4M3, FMT_E5M2)
#endif
#if TE_GATED_PART < 0 || TE_GATED_PART == 3
TE_GATED_FORWARD(e5_e5, FMT_E5M2, FMT_E5M2)
#endif
#if TE_GATED_PART < 0 || TE_GATED_PART == 4
TE_GATED_DGRAD(e4_e4, FMT_E4M3, FMT_E4M3)
#endif
#if TE_GATED_PART < 0 || TE_GATED_PART == 5
TE_GATED_DGRAD(e5_e4, FMT_E5M2, FMT_E4M3)
#endif
#if TE_GATED_PART < 0 || TE_GATED_PART == 6
TE_GATED_DGRAD(e4_e5, FMT_E4M3, FMT_E5M2)
#endif
#if TE_GATED_PART < 0 || TE_GATED_PART == 7
TE_GATED_DGRAD(e5_e5, FMT_E5M2, FMT_E5M2)
#endif

#if TE_GATED_PART < 0 || TE_GATED_PART == 8
namespace {
// The kernel of parts where there are at most four for each compute unit; for a row-wise cast of y, which then needs a
// second kernel, at most three.  K = 4096, M x N, us by tiles
// and by parts:
//   data gradient, bf16   512 x 8192 (2 parts a unit) 60.4, 30.5;  300 x 16384 (2.5) 69.3, 48.5;  512 x 16384 (4) 76.1, 71.0;
//                         512 x 24576 (6) 86.5, 107.9;  2048 x 8192 (8) 93.4, 151.9
//   forward, bf16         512 x 8192 49.8, 27.3;  300 x 16384 51.2, 38.6;  512 x 16384 52.2, 49.5;  512 x 24576 64.9, 87.1
//   forward, fp8          512 x 8192 51.7, 31.2;  512 x 12288 (3) 51.8, 45.1;  512 x 16384 52.3, 55.8
// At four parts a unit short contractions gain a little by it and long ones lose as much:
//   K = 1024, bf16        data gradient 512 x 8192 30.6, 15.5;  512 x 16384 32.3, 26.8;  512 x 24576 47.4, 46.4
//                         forward 19.4, 11.5;  21.0, 20.3;  23.1, 27.2
//   K = 14336, bf16       data gradient 194, 111;  200, 212;  228, 313;  forward 178, 105;  181, 199;  210, 295
// The cast of the transpose needs 128 rows and a part has 64, so it takes tiles however few: 512 rows, forward 512 x 8192
// with z 56 us (row-wise alone 32), data gradient 81 (31).
bool by_parts(int64_t M, int64_t N, int most = 4)
{
    return ((M + kWM - 1) / kWM) * ((N + kWN - 1) / kWN) <= (int64_t)most * device_cus();
}
}  // namespace

bool gated_fwd_through_f32(int64_t M, int64_t H) { return by_parts(M, 2 * H, 3); }

hipError_t launch_gated_fwd(const GemmArgs& a, hipStream_t stream)
{
    const bool parts = !a.q_out && !a.qt_out && by_parts(a.M, a.N);
#define TE_TAKE(n, pair, A, B) \
    if (a.fmt_a == A && a.fmt_b == B) return gated_forward_##pair(a, parts, stream);
    TE_GATED_PAIRS(TE_TAKE)
#undef TE_TAKE
    return hipErrorInvalidValue;
}

hipError_t launch_gated_dgrad(const GemmArgs& a, hipStream_t stream)
{
    const bool parts = !a.qt_out && by_parts(a.M, a.N);
#define TE_TAKE(n, pair, A, B) \
    if (a.fmt_a == A && a.fmt_b == B) return gated_dgrad_##pair(a, parts, stream);
    TE_GATED_PAIRS(TE_TAKE)
#undef TE_TAKE
    return hipErrorInvalidValue;
}
#endif

}  // namespace tefp8
