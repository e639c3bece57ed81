// Top-k router with per-expert counts and balance loss, for gfx950.
//
//   p = softmax of a token's logits; its experts are the top_k largest logits, equal ones by the
//   lower index; logits of -inf (closed experts) and NaN are never chosen
//   weight = p of the chosen experts, or those divided by their sum
//   counts[e] = tokens sent to e, n = tokens sent anywhere,
//   loss = experts / (top_k n^2) * sum over e of counts[e] * (sum over those tokens of p[.][e])
//
// kL lanes share a token, each with kNC chunks of eight consecutive logits (16 bytes of bf16;
// chunk i of lane p starts at column 8 (i kL + p), so the lanes' loads of one chunk are one run).
// The logits stay in registers.  Selection: every lane keeps its kK largest in a sorted list; with
// a[j-1] >= a[j] the list after x came in is a'[j] = med3(a[j-1], a[j], x), one instruction per
// entry.  For bf16 the entry is one 32-bit word, the logit's order-preserving bits above and the
// column's position below (so equal logits differ and the lower column wins); for fp32 the position
// travels beside it.  The lists of the kL lanes merge pairwise: the larger of a[j] and the
// partner's a[kK-1-j] are the kK largest in a bitonic order, which log2(kK) exchanges sort.
//
// A lane has the same columns for every token it takes, so the column sums of p that the loss
// needs add up in its registers; they and the counts (integer atomics in LDS) leave the workgroup
// once, as one row of the workspace that a second kernel adds up in a fixed order.  Calls of few
// tokens run in one workgroup that finishes by itself.
//
// Measured at 65536 tokens, 256 experts, bf16, top 8: forward 19.7 us and 4.8 us for the second kernel (38 MB
// would take 7.2 us).  The first issues 918 vector instructions per wave and step of eight tokens, 13 to 14 us of it by
// their cycles; the rest is waiting, with two waves on a SIMD and no loads ahead of the step.  Backward 13.7
// us, bound by memory (71 MB at 5.2 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "internal.h"
#include "ops_device.h"
#include "ops_internal.h"

namespace tefp8 {
namespace {

constexpr uint32_t kNegInf = 0xFF800000u;

// Signed integers in the order of the floats: the magnitude's bits, negated for negative numbers
// (so -0 = +0).  -inf is kClosed: nothing at or below is chosen; NaN lies above +inf or below -inf.
constexpr int32_t kOpenInf = 0x7F800000, kClosed = -kOpenInf;
__device__ __forceinline__ int32_t order_key(uint32_t bits)
{
    const int32_t neg = (int32_t)bits >> 31;
    return ((int32_t)(bits & 0x7FFFFFFFu) ^ neg) - neg;
}
__device__ __forceinline__ float from_order_key(int32_t k)
{
    return as_float(k < 0 ? (uint32_t)-k | 0x80000000u : (uint32_t)k);
}
// The middle one; written so that it becomes one instruction.
__device__ __forceinline__ int32_t med3(int32_t a, int32_t b, int32_t x) { return max(min(a, b), min(max(a, b), x)); }

// exp for arguments at or below zero.  t = x log2(e) is rounded, which would be |x| 2^-24 of the result; what it is
// off by, x - t ln 2, comes back as a factor.  The constant is the float above log2(e), so that this is never
// negative (at most |x| 2^-22), and its bounds 0 and 1 cost nothing (the instruction clamps) and make a zero of the
// NaN at x = -inf; a NaN x stays NaN by t.  ln 2 as a float adds |x| 2^-28.
__device__ __forceinline__ float exp_exact(float x)
{
    float ln2 = -0.693147182f;
    asm("" : "+s"(ln2));   // (in a register: an instruction with a literal has no clamp)
    const float t = x * 1.44269514f;
    const float r = __builtin_amdgcn_fmed3f(fmaf(t, ln2, x), 0.0f, 1.0f);
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, r, e);
}
// The product alone, for what is stored in bf16 next: off by |x| 2^-24 of the result, where the store rounds by
// 2^-8 (the backward pass in bf16: 13.6 us so, 14.3 with exp_exact).
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// A sum in pairs: one after the other, equal small terms on top of a large one are all rounded the same way (2047
// logits 7.6 below the largest: the row's sum off by 6 steps of 2^-24 rms that way, by 1 in pairs).
template <int kN> __device__ __forceinline__ float sum_pairs(const float (&v)[kN])
{
    static_assert((kN & (kN - 1)) == 0, "halves");
    float s[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i] = v[i];
#pragma unroll
    for (int n = kN / 2; n >= 1; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) s[i] += s[i + n];
    return s[0];
}

// A sorted list of the kK largest (key, column), equal keys by the lower column.
template <class T, int kK> struct TopList;

template <int kK> struct TopList<Bf16, kK> {
    int32_t a[kK];   // the upper half of the key, and below it what makes equal keys differ
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < kK; ++j) a[j] = INT32_MIN;
    }
    __device__ __forceinline__ void insert(int32_t x)
    {
#pragma unroll
        for (int j = kK - 1; j > 0; --j) a[j] = med3(a[j - 1], a[j], x);
        a[0] = max(a[0], x);
    }
    // Eight logits; the lane's own elements are numbered from `pos` on, in ascending column order (0 .. 63).
    __device__ __forceinline__ void insert8(const Raw8<Bf16>& r, int pos, bool drop_nan)
    {
        typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = r.a[i], m = w & 0x7FFF7FFFu;
            const i16x2 neg = __builtin_bit_cast(i16x2, w) >> 15;
            uint32_t k = __builtin_bit_cast(uint32_t, (__builtin_bit_cast(i16x2, m) ^ neg) - neg);
            if (drop_nan) {
                if ((m & 0xFFFFu) > 0x7F80u) k = (k & 0xFFFF0000u) | 0x8000u;
                if (m >> 16 > 0x7F80u) k = (k & 0xFFFFu) | 0x80000000u;
            }
            insert((int32_t)((k << 16) | (63 - (pos + 2 * i))));
            insert((int32_t)((k & 0xFFFF0000u) | (63 - (pos + 2 * i + 1))));
        }
    }
    // own numbers -> columns
    template <class F> __device__ __forceinline__ void to_columns(F column)
    {
#pragma unroll
        for (int j = 0; j < kK; ++j) a[j] = (a[j] & (int32_t)0xFFFF0000) | (0xFFFF - column(63 - (a[j] & 63)));
    }
    __device__ __forceinline__ int32_t key(int j) const { return a[j] & (int32_t)0xFFFF0000; }
    __device__ __forceinline__ int column(int j) const { return 0xFFFF - (a[j] & 0xFFFF); }
    template <int kStep> __device__ __forceinline__ void take_partner()
    {
        int32_t b[kK];
#pragma unroll
        for (int j = 0; j < kK; ++j) b[j] = max(a[j], partner<kStep>(a[kK - 1 - j]));
#pragma unroll
        for (int j = 0; j < kK; ++j) a[j] = b[j];
    }
    __device__ __forceinline__ void order(int i, int j)
    {
        const int32_t hi = max(a[i], a[j]), lo = min(a[i], a[j]);
        a[i] = hi;
        a[j] = lo;
    }
};

template <int kK> struct TopList<F32, kK> {
    int32_t a[kK];
    int c[kK];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < kK; ++j) {
            a[j] = INT32_MIN;
            c[j] = 0;
        }
    }
    __device__ __forceinline__ void insert(int32_t x, int pos)
    {
        bool above = x > a[kK - 1];   // x goes above entry j (an equal earlier one stays above x)
#pragma unroll
        for (int j = kK - 1; j > 0; --j) {
            const bool next = x > a[j - 1];
            c[j] = next ? c[j - 1] : above ? pos : c[j];
            a[j] = med3(a[j - 1], a[j], x);
            above = next;
        }
        c[0] = above ? pos : c[0];
        a[0] = max(a[0], x);
    }
    __device__ __forceinline__ void insert8(const Raw8<F32>& r, int pos, bool drop_nan)
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t w = j < 4 ? (uint32_t)r.a[j & 3] : (uint32_t)r.b[j & 3];
            int32_t k = order_key(w);
            if (drop_nan && (w & 0x7FFFFFFFu) > 0x7F800000u) k = INT32_MIN;
            insert(k, pos + j);
        }
    }
    template <class F> __device__ __forceinline__ void to_columns(F column)
    {
#pragma unroll
        for (int j = 0; j < kK; ++j) c[j] = column(c[j]);
    }
    __device__ __forceinline__ int32_t key(int j) const { return a[j]; }
    __device__ __forceinline__ int column(int j) const { return c[j]; }
    static __device__ __forceinline__ bool before(int32_t ka, int ca, int32_t kb, int cb)
    {
        return ka > kb || (ka == kb && ca < cb);
    }
    template <int kStep> __device__ __forceinline__ void take_partner()
    {
        int32_t b[kK];
        int d[kK];
#pragma unroll
        for (int j = 0; j < kK; ++j) {
            b[j] = partner<kStep>(a[kK - 1 - j]);
            d[j] = partner<kStep>(c[kK - 1 - j]);
        }
#pragma unroll
        for (int j = 0; j < kK; ++j) {
            const bool mine = before(a[j], c[j], b[j], d[j]);
            a[j] = mine ? a[j] : b[j];
            c[j] = mine ? c[j] : d[j];
        }
    }
    __device__ __forceinline__ void order(int i, int j)
    {
        const bool keep = before(a[i], c[i], a[j], c[j]);
        const int32_t ka = a[i];
        const int ca = c[i];
        a[i] = keep ? ka : a[j];
        c[i] = keep ? ca : c[j];
        a[j] = keep ? a[j] : ka;
        c[j] = keep ? c[j] : ca;
    }
};

template <int kStep, class T, int kK>
__device__ __forceinline__ void merge(TopList<T, kK>& l)
{
    l.template take_partner<kStep>();
#pragma unroll
    for (int s = kK / 2; s >= 1; s >>= 1)
#pragma unroll
        for (int j = 0; j < kK; ++j)
            if ((j & s) == 0) l.order(j, j + s);
}
template <int kL, class T, int kK>
__device__ __forceinline__ void merge_lanes(TopList<T, kK>& l)
{
    if constexpr (kL > 1) merge<1>(l);
    if constexpr (kL > 2) merge<2>(l);
    if constexpr (kL > 4) merge<4>(l);
    if constexpr (kL > 8) merge<8>(l);
    if constexpr (kL > 16) merge<16>(l);
    if constexpr (kL > 32) merge<32>(l);
}

// The lane's chunks of a row: the eight logits from each column (i kL + p) 8 on, columns past the last as
// -inf.  (The last chunk of a row whose length is no multiple of eight is loaded from experts - 8 and
// moved to the front.  All loads come first: one that is waited for by itself costs its whole latency.)
template <class T, int kL, int kNC, class P>
__device__ __forceinline__ void load_logits(Raw8<T> (&r)[kNC], const P* row, int p, int experts)
{
    if (kL * kNC == 1 && experts < 8) {
        r[0] = load_few(row, experts, kNegInf);
        return;
    }
#pragma unroll
    for (int i = 0; i < kNC; ++i) r[i] = load8(row + min((i * kL + p) * 8, experts - 8));
#pragma unroll
    for (int i = 0; i < kNC; ++i) {
        const int col = (i * kL + p) * 8, behind = col - (experts - 8);
        if (behind > 0) r[i] = behind < 8 ? drop_front(r[i], behind, kNegInf) : fill8<T>(kNegInf);
    }
}

// The workspace: a row per workgroup of counts (and, behind them, of its routed tokens) and of
// sums of p, then a sum per workgroup of the second kernel, and its ticket.
struct Space {
    int32_t* counts;
    float* probs;
    double* sums;
    int32_t* ticket;
};
constexpr int kFinishCols = 16;
__host__ __device__ inline int64_t finish_blocks(int64_t experts) { return experts / kFinishCols + 1; }
__host__ __device__ inline Space space_at(void* ws, int64_t blocks, int64_t experts)
{
    Space s;
    s.sums = static_cast<double*>(ws);
    s.ticket = reinterpret_cast<int32_t*>(s.sums + finish_blocks(experts));
    s.counts = s.ticket + 2;
    s.probs = reinterpret_cast<float*>(s.counts + blocks * (experts + 1));
    return s;
}

__device__ __forceinline__ float balance_loss(double sum, int64_t n, int experts, int top_k)
{
    const double m = n > 0 ? (double)n : 1.0;
    return (float)((double)experts / (double)top_k * sum / (m * m));
}

// Sum over the workgroup, in every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double v, double* red)
{
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < (int)blockDim.x / 64; ++i) s += red[i];
    return s;
}

constexpr int kFwdThreads = 512;
constexpr int kFwdWaves = kFwdThreads / 64;

// (Waves per SIMD that the registers are cut for: four take 128 each, which the long lists and the rows of
// fp32 do not fit, and the lists of 4 and 8 on 32 lanes but for one register, which is spilled.)
template <class T, int kNC, int kK> constexpr int kFwdWavesPerSimd = kK == 16 || (kNC == 4 && __is_same(T, F32)) ? 2 : 4;

template <class T, int kL, int kNC, int kK, bool kLoss>
__global__ __launch_bounds__(kFwdThreads, (kFwdWavesPerSimd<T, kNC, kK>)) void router_fwd_kernel(const RouterArgs a)
{
    extern __shared__ int32_t lds[];   // with the loss: counts [experts], sums of p [kFwdWaves][experts]
    __shared__ int32_t routed;
    __shared__ double red[kFwdWaves];
    constexpr int kRows = 64 / kL;     // tokens per wave and step
    constexpr bool kAhead = kNC <= 2;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int p = lane % kL, slot = lane / kL;
    const int E = a.experts, k = a.top_k;
    const auto* logits = static_cast<const typename T::store_t*>(a.logits);
    int32_t* hist = lds;
    float* sums = reinterpret_cast<float*>(lds + E);

    float acc[kNC][8];
    int n_routed = 0;
    if constexpr (kLoss) {
        for (int e = threadIdx.x; e < E; e += kFwdThreads) hist[e] = 0;
        if (threadIdx.x == 0) {
            routed = 0;
            // (for the second kernel, which starts after this one has ended)
            if (a.workspace && blockIdx.x == 0) *space_at(a.workspace, a.blocks, E).ticket = 0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kNC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    }

    const int64_t step = (int64_t)gridDim.x * kFwdWaves * kRows;
    int64_t base = ((int64_t)blockIdx.x * kFwdWaves + wave) * kRows;
    // Tokens past the end repeat the last one and store nothing.
    Raw8<T> raw[kNC], next[kNC];
    uint8_t unmasked = 1, next_unmasked = 1;
    auto fetch = [&](int64_t b, Raw8<T> (&r)[kNC], uint8_t& m) {
        const int64_t t = min(b + slot, a.tokens - 1);
        const auto* row = logits + t * a.ld;
        if (a.mask) m = a.mask[t];
        load_logits<T, kL>(r, row, p, E);
    };
    if (kAhead && base < a.tokens) fetch(base, next, next_unmasked);
    for (; base < a.tokens; base += step) {
        const int64_t t = base + slot;
        if constexpr (kAhead) {
            unmasked = next_unmasked;
#pragma unroll
            for (int i = 0; i < kNC; ++i) raw[i] = next[i];
            if (base + step < a.tokens) fetch(base + step, next, next_unmasked);
        } else {
            fetch(base, raw, unmasked);
        }
        const bool in = t < a.tokens, live = in && unmasked != 0;

        TopList<T, kK> top;
        auto select = [&](bool drop_nan) {
            top.clear();
#pragma unroll
            for (int i = 0; i < kNC; ++i) top.insert8(raw[i], i * 8, drop_nan);
            top.to_columns([&](int pos) { return ((pos >> 3) * kL + p) * 8 + (pos & 7); });
            merge_lanes<kL>(top);
        };
        select(false);
        // A NaN above all others was chosen: choose again without any (those below -inf never are).  The
        // sum of the row is NaN in both cases, and with it the token's weights.
        if (__any(top.key(0) > kOpenInf)) select(true);

        const float m = top.key(0) > kClosed ? from_order_key(top.key(0)) : 0.0f;
        float e[kNC][8], part[kNC];
#pragma unroll
        for (int i = 0; i < kNC; ++i) {
            float v[8];
            unpack8(raw[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) e[i][j] = exp_exact(v[j] - m);
            part[i] = sum_pairs(e[i]);
        }
        const float s = sum_lanes<kL>(sum_pairs(part));
        const bool sent = live && top.key(0) > kClosed;

        // lane p has entries p, p + kL, ...
        constexpr int kOwn = (kK + kL - 1) / kL;
        float ev[kOwn], sum = 0.0f;
        int col[kOwn];
#pragma unroll
        for (int q = 0; q < kOwn; ++q) {
            int32_t key = top.key(q * kL);
            col[q] = top.column(q * kL);
#pragma unroll
            for (int i = 1; i < kL && q * kL + i < kK; ++i) {
                key = p == i ? top.key(q * kL + i) : key;
                col[q] = p == i ? top.column(q * kL + i) : col[q];
            }
            const bool chosen = sent && key > kClosed && q * kL + p < min(k, kK);
            ev[q] = chosen ? exp_exact(from_order_key(key) - m) : 0.0f;
            if (!chosen) col[q] = -1;
            sum += ev[q];
        }
        const float inv = 1.0f / s;
        float scale = inv;
        if (a.renorm) scale = s == s ? 1.0f / sum_lanes<kL>(sum) : s;
#pragma unroll
        for (int q = 0; q < kOwn; ++q) {
            const int j = q * kL + p;
            if (in && j < k && j < kK) {
                a.index[t * k + j] = col[q];
                a.weight[t * k + j] = col[q] >= 0 ? ev[q] * scale : 0.0f;
                if constexpr (kLoss)
                    if (col[q] >= 0) atomicAdd(&hist[col[q]], 1);
            }
        }
        if (a.lse && p == 0 && in) a.lse[t] = sent ? m + logf(s) : 0.0f;
        if constexpr (kLoss) {
            if (sent) {
                n_routed += p == 0;
#pragma unroll
                for (int i = 0; i < kNC; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[i][j] += e[i][j] * inv;
            }
        }
    }

    if constexpr (kLoss) {
        // The wave's tokens side by side (lanes p, p + kL, ...): the halves and the rows of the wave
        // exchange, so that each keeps half of the sums, then the lanes of a row.
        float v[kNC * 8];
        int n = kNC * 8, first = 0;
#pragma unroll
        for (int i = 0; i < kNC * 8; ++i) v[i] = acc[i >> 3][i & 7];
        if constexpr (kL <= 32) {
            n /= 2;
            first += (lane & 32) ? n : 0;
#pragma unroll
            for (int i = 0; i < kNC * 4; ++i) {
                const auto x = __builtin_amdgcn_permlane32_swap(as_bits(v[i]), as_bits(v[i + kNC * 4]), false, false);
                v[i] = as_float(x[0]) + as_float(x[1]);
            }
        }
        if constexpr (kL <= 16) {
            n /= 2;
            first += (lane & 16) ? n : 0;
#pragma unroll
            for (int i = 0; i < kNC * 2; ++i) {
                const auto x = __builtin_amdgcn_permlane16_swap(as_bits(v[i]), as_bits(v[i + kNC * 2]), false, false);
                v[i] = as_float(x[0]) + as_float(x[1]);
            }
        }
        constexpr int kKept = kNC * 8 / (kL <= 16 ? 4 : kL <= 32 ? 2 : 1);
#pragma unroll
        for (int i = 0; i < kKept; ++i) {
            if constexpr (kL <= 8) v[i] += as_float((uint32_t)dpp<0x128>((int)as_bits(v[i])));   // row_ror:8
            if constexpr (kL <= 4) v[i] += as_float((uint32_t)dpp<0x124>((int)as_bits(v[i])));
            if constexpr (kL <= 2) v[i] += as_float((uint32_t)dpp<0x122>((int)as_bits(v[i])));
            if constexpr (kL <= 1) v[i] += as_float((uint32_t)dpp<0x121>((int)as_bits(v[i])));
            const int f = first + i, col = ((f >> 3) * kL + p) * 8 + (f & 7);
            if ((lane & 15) < kL && col < E) sums[wave * E + col] = v[i];
        }
        if (n_routed) atomicAdd(&routed, n_routed);
        __syncthreads();
        if (a.workspace) {
            const Space w = space_at(a.workspace, a.blocks, E);
            for (int e = threadIdx.x; e < E; e += kFwdThreads) {
                float s = 0.0f;
                for (int q = 0; q < kFwdWaves; ++q) s += sums[q * E + e];
                w.counts[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
                w.probs[(int64_t)blockIdx.x * E + e] = s;
            }
            if (threadIdx.x == 0) w.counts[(int64_t)blockIdx.x * (E + 1) + E] = routed;
        } else {
            double part = 0.0;
            for (int e = threadIdx.x; e < E; e += kFwdThreads) {
                double s = 0.0;
                for (int q = 0; q < kFwdWaves; ++q) s += (double)sums[q * E + e];
                a.counts[e] = hist[e];
                part += (double)hist[e] * s;
            }
            part = block_sum(part, red);
            if (threadIdx.x == 0) {
                a.routed[0] = routed;
                a.loss[0] = balance_loss(part, routed, E, k);
            }
        }
    }
}

// Adds up the workgroups' rows: 16 columns per workgroup (column `experts` is the number of routed
// tokens), 64 threads per column; the last workgroup to end adds the columns' parts of the loss.
__global__ __launch_bounds__(1024) void router_finish_kernel(const RouterArgs a)
{
    __shared__ double red_p[16][kFinishCols];
    __shared__ int32_t red_c[16][kFinishCols];
    __shared__ double part[kFinishCols];
    const int E = a.experts, cl = threadIdx.x % kFinishCols, rl = threadIdx.x / kFinishCols;
    const int e = blockIdx.x * kFinishCols + cl;
    const Space w = space_at(a.workspace, a.blocks, E);
    double s = 0.0;
    int32_t c = 0;
    if (e <= E) {
#pragma unroll 8
        for (int64_t b = rl; b < a.blocks; b += 1024 / kFinishCols) {
            c += w.counts[b * (E + 1) + e];
            if (e < E) s += (double)w.probs[b * E + e];
        }
    }
#pragma unroll
    for (int d = kFinishCols; d < 64; d <<= 1) {
        s += __shfl_xor(s, d);
        c += __shfl_xor(c, d);
    }
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) < kFinishCols) {
        red_p[wave][cl] = s;
        red_c[wave][cl] = c;
    }
    __syncthreads();
    if (threadIdx.x < kFinishCols) {
        s = 0.0;
        c = 0;
        for (int i = 0; i < 16; ++i) {
            s += red_p[i][cl];
            c += red_c[i][cl];
        }
        if (e < E) a.counts[e] = c;
        else if (e == E) __hip_atomic_store(a.routed, c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        part[cl] = e < E ? (double)c * s : 0.0;
    }
    __syncthreads();
    if (threadIdx.x >= 64) return;
    double v = 0.0;
    for (int i = 0; i < kFinishCols; ++i) v += part[i];
    if (gridDim.x > 1) {
        // What the last workgroup reads of the others (this sum, and `routed`, stored above by this wave)
        // goes to memory by agent-wide stores; waiting for them is all the order that is needed, and a
        // release would write the whole L2 back.
        int32_t before = 0;
        if (threadIdx.x == 0) {
            __hip_atomic_store(&w.sums[blockIdx.x], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            before = __hip_atomic_fetch_add(w.ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        if (__shfl(before, 0) != (int)gridDim.x - 1) return;
        asm volatile("" ::: "memory");
        v = 0.0;
        for (int i = threadIdx.x; i < (int)gridDim.x; i += 64)
            v += __hip_atomic_load(&w.sums[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    }
    if (threadIdx.x == 0) {
        const int32_t n = __hip_atomic_load(a.routed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        a.loss[0] = balance_loss(v, n, E, a.top_k);
    }
}

// ------------------------------------------------------------ backward
//   a[e] = d_loss * experts / top_k * counts[e] / n^2   (the loss is linear in p)
//   weights p:            b = a + d_weight at the chosen columns,  d = p * (b - sum of p b)
//   weights renormalised: d = p * (a - sum of p a) + w * (d_weight - sum of w d_weight) at the chosen ones
// with p = exp(logit - lse) divided by its sum over the row.
// One read of the logits and one write of the gradient; a token's lanes hold its row in registers
// as in the forward pass.  What the chosen columns get extra is handed to the lanes that hold them
// through LDS (a row of zeros per token, set, read by columns, and cleared again).
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

template <class T, int kL, int kNC, bool kRenorm>
__global__ __launch_bounds__(kThreads, 4) void router_bwd_kernel(const RouterBwdArgs a)
{
    constexpr int kRows = 64 / kL, kCols = kL * kNC * 8;
    constexpr bool kBf16 = __is_same(T, Bf16);
    constexpr int kSlots = (kRouterMaxTopK + kL - 1) / kL;   // entries of a token per lane
    __shared__ __attribute__((aligned(16))) float extra_lds[kWaves][kRows][kCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int p = lane % kL, slot = lane / kL;
    const int E = a.experts, k = a.top_k;
    float* extra = extra_lds[wave][slot];
    for (int c = p * 8; c < kCols; c += kL * 8)
#pragma unroll
        for (int j = 0; j < 8; ++j) extra[c + j] = 0.0f;

    auto read_extra = [&](int i, float (&x)[8]) {
        const float4* src = reinterpret_cast<const float4*>(extra + (i * kL + p) * 8);
        const float4 lo = src[0], hi = src[1];
        x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
        x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
    };

    float g[kNC][8];
#pragma unroll
    for (int i = 0; i < kNC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] = 0.0f;
    if (a.d_loss) {
        const float n = (float)max(a.routed[0], 1);
        const float f = a.d_loss[0] * ((float)E / (float)k) / (n * n);
        // (read as the logits are; past the last column any count will do, as p is zero there)
        Raw8<F32> c[kNC];
        load_logits<F32, kL>(c, reinterpret_cast<const float*>(a.counts), p, E);
#pragma unroll
        for (int i = 0; i < kNC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) g[i][j] = f * (float)(int32_t)(j < 4 ? (uint32_t)c[i].a[j & 3] : (uint32_t)c[i].b[j & 3]);
    }

    const auto* logits = static_cast<const typename T::store_t*>(a.logits);
    const int64_t step = (int64_t)gridDim.x * kWaves * kRows;
    for (int64_t base = ((int64_t)blockIdx.x * kWaves + wave) * kRows; base < a.tokens; base += step) {
        const bool in = base + slot < a.tokens;
        const int64_t t = in ? base + slot : a.tokens - 1;
        const auto* row = logits + t * a.ld;
        // The chosen columns: entries p, p + kL, ... of the token are this lane's.  (Everything that is
        // read by the token is asked for here, before any of it is used.)
        int pos[kSlots];
        float dw[kSlots], w[kSlots];
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            pos[q] = -1;
            dw[q] = w[q] = 0.0f;
            if (q * kL >= k) continue;
            const int64_t at = t * k + min(q * kL + p, k - 1);
            pos[q] = a.index[at];
            if (a.d_weight) dw[q] = a.d_weight[at];
        }
        const int first = a.index[t * k];
        const float lse = a.lse[t];
        Raw8<T> raw[kNC];
        load_logits<T, kL>(raw, row, p, E);
        const bool live = in && first >= 0;
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            if (!live || q * kL + p >= k || pos[q] >= E) pos[q] = -1;
            if (pos[q] < 0) dw[q] = 0.0f;
            if constexpr (kRenorm) {
                if (pos[q] >= 0) {
                    float v;
                    if constexpr (kBf16) v = as_float((uint32_t)row[pos[q]] << 16);
                    else v = row[pos[q]];
                    w[q] = expf(v - lse);
                }
            }
        }
        if constexpr (kRenorm) {
            float sw = 0.0f, sd = 0.0f;
#pragma unroll
            for (int q = 0; q < kSlots; ++q) sw += w[q];
            sw = sum_lanes<kL>(sw);
            const float iw = sw > 0.0f ? 1.0f / sw : sw;   // (NaN stays)
#pragma unroll
            for (int q = 0; q < kSlots; ++q) {
                w[q] *= iw;
                sd += w[q] * dw[q];
            }
            sd = sum_lanes<kL>(sd);
#pragma unroll
            for (int q = 0; q < kSlots; ++q) dw[q] = w[q] * (dw[q] - sd);
        }
#pragma unroll
        for (int q = 0; q < kSlots; ++q)
            if (pos[q] >= 0) extra[pos[q]] = dw[q];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();

        float pr[kNC][8];
        float dot = 0.0f, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kNC; ++i) {
            float v[8], x[8];
            read_extra(i, x);
            unpack8(raw[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                pr[i][j] = kBf16 ? exp_fast(v[j] - lse) : exp_exact(v[j] - lse);
                sum += pr[i][j];
                dot += pr[i][j] * (kRenorm ? g[i][j] : g[i][j] + x[j]);
            }
        }
        // (the sum is 1 but for lse's rounding, which matters where lse is large beside the log in it)
        sum = sum_lanes<kL>(sum);
        const float inv = lse == lse ? 1.0f / sum : lse;
        dot = sum_lanes<kL>(dot) * inv;

        auto* out = static_cast<typename T::store_t*>(a.d_logits) + t * a.ld_d;
#pragma unroll
        for (int i = 0; i < kNC; ++i) {
            const int col = (i * kL + p) * 8;
            float d[8], x[8];
            read_extra(i, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float pj = pr[i][j] * inv;
                d[j] = kRenorm ? pj * (g[i][j] - dot) + x[j] : pj * (g[i][j] + x[j] - dot);
            }
            if (!in || col >= E) continue;
            const Raw8<T> r = live ? pack8(T{}, d) : zero8<T>();
            if (col + 8 <= E) store8(out + col, r);
            else store_few(out + col, r, E - col);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < kSlots; ++q)
            if (pos[q] >= 0) extra[pos[q]] = 0.0f;
    }
}

// Lanes per token and chunks per lane for a number of experts: as few lanes as hold the row with
// at most four chunks each, and at least eight (one 128-byte line of bf16 per chunk) beyond 32 experts.
struct Shape { int lanes, chunks; };
Shape shape_of(int64_t experts)
{
    if (experts <= 8) return {1, 1};
    if (experts <= 16) return {1, 2};
    if (experts <= 32) return {4, 1};
    if (experts <= 64) return {8, 1};
    if (experts <= 128) return {8, 2};
    if (experts <= 256) return {8, 4};
    if (experts <= 512) return {16, 4};
    if (experts <= 1024) return {32, 4};
    return {64, 4};
}

template <class T, int kL, int kNC, int kK>
hipError_t fwd_run(const RouterArgs& a, hipStream_t stream)
{
    const dim3 grid((unsigned)a.blocks);
    if (a.counts) {
        const size_t lds = (size_t)a.experts * 4 * (1 + kFwdWaves);
        router_fwd_kernel<T, kL, kNC, kK, true><<<grid, kFwdThreads, lds, stream>>>(a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || !a.workspace) return e;
        router_finish_kernel<<<(unsigned)finish_blocks(a.experts), 1024, 0, stream>>>(a);
    } else {
        router_fwd_kernel<T, kL, kNC, kK, false><<<grid, kFwdThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <class T, int kL, int kNC>
hipError_t fwd_k(const RouterArgs& a, hipStream_t stream)
{
    if (a.top_k == 1) return fwd_run<T, kL, kNC, 1>(a, stream);
    if (a.top_k == 2) return fwd_run<T, kL, kNC, 2>(a, stream);
    if (a.top_k <= 4) return fwd_run<T, kL, kNC, 4>(a, stream);
    if (a.top_k <= 8) return fwd_run<T, kL, kNC, 8>(a, stream);
    if constexpr (kL * kNC > 1) return fwd_run<T, kL, kNC, 16>(a, stream);
    return hipErrorInvalidValue;
}

template <class T, int kL, int kNC>
hipError_t bwd_run(const RouterBwdArgs& a, hipStream_t stream)
{
    const int64_t per = kWaves * (64 / kL);
    const int64_t blocks = std::min<int64_t>((a.tokens + per - 1) / per, 4 * device_cus());
    if (a.renorm) router_bwd_kernel<T, kL, kNC, true><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    else router_bwd_kernel<T, kL, kNC, false><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

#define TE_ROUTER_SHAPES(F, T, a, stream)                          \
    do {                                                           \
        const Shape s = shape_of((a).experts);                     \
        if (s.lanes == 1 && s.chunks == 1) return F<T, 1, 1>(a, stream); \
        if (s.lanes == 1) return F<T, 1, 2>(a, stream);            \
        if (s.lanes == 4) return F<T, 4, 1>(a, stream);            \
        if (s.lanes == 8 && s.chunks == 1) return F<T, 8, 1>(a, stream); \
        if (s.lanes == 8 && s.chunks == 2) return F<T, 8, 2>(a, stream); \
        if (s.lanes == 8) return F<T, 8, 4>(a, stream);            \
        if (s.lanes == 16) return F<T, 16, 4>(a, stream);          \
        if (s.lanes == 32) return F<T, 32, 4>(a, stream);          \
        return F<T, 64, 4>(a, stream);                             \
    } while (0)

template <class T> hipError_t fwd_shape(const RouterArgs& a, hipStream_t stream) { TE_ROUTER_SHAPES(fwd_k, T, a, stream); }
template <class T> hipError_t bwd_shape(const RouterBwdArgs& a, hipStream_t stream) { TE_ROUTER_SHAPES(bwd_run, T, a, stream); }

}  // namespace

// Workgroups: one where it takes the tokens in at most four steps and the counts are asked for (no second
// kernel then).  Else as many as are resident, and with four chunks per lane half of that: their time is mostly
// instructions, and every workgroup costs the second kernel a row (both kernels with 256 workgroups and with 512:
// 65536 x 256 bf16 23.4 and 24.6 us, 16384 x 512 bf16 17.3 and 18.7, 32768 x 256 fp32 23.1 and 27.3; 100000 x 64 fp32
// 30.5 and 27.3, 100000 x 100 fp32 41.5 and 37.2).
int64_t router_fwd_blocks(int64_t tokens, int64_t experts, bool loss)
{
    const Shape s = shape_of(experts);
    const int64_t per = kFwdWaves * (64 / s.lanes);
    const int64_t blocks = (tokens + per - 1) / per;
    if (loss && blocks <= 4) return 1;
    return std::min<int64_t>(blocks, !loss ? 4096 : s.chunks == 4 ? 256 : 512);
}

int64_t router_fwd_workspace_bytes(int64_t tokens, int64_t experts)
{
    const int64_t blocks = router_fwd_blocks(tokens, experts, true);
    if (blocks <= 1) return 0;
    return finish_blocks(experts) * 8 + 8 + blocks * (experts + 1) * 4 + blocks * experts * 4;
}

hipError_t launch_router_fwd(const RouterArgs& a, hipStream_t stream)
{
    if (a.blocks <= 0) return hipSuccess;
    return a.bf16 ? fwd_shape<Bf16>(a, stream) : fwd_shape<F32>(a, stream);
}

hipError_t launch_router_bwd(const RouterBwdArgs& a, hipStream_t stream)
{
    if (a.tokens <= 0) return hipSuccess;
    return a.bf16 ? bwd_shape<Bf16>(a, stream) : bwd_shape<F32>(a, stream);
}

}  // namespace tefp8
