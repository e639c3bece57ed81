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
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ops_device.h"
#include "ops_internal.h"

namespace tefp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr uint32_t kNegInf = 0xFF800000u;
constexpr uint32_t kClosed = 0x007FFFFFu;   // order-preserving bits of -inf: nothing at or below is chosen
constexpr uint32_t kOpenInf = 0xFF800000u;  // ... of +inf: NaN lies above

// Order-preserving bits: unsigned comparison of the results is comparison of the floats (-0 = +0).
__device__ __forceinline__ uint32_t order_bits(float v)
{
    const uint32_t b = as_bits(v + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t k)
{
    return as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint32_t med3(uint32_t a, uint32_t b, uint32_t x)   // a >= b
{
    return max(min(a, x), b);
}

// A sorted list of the kK largest (key, column), equal keys by the lower column.
template <class T, int kK> struct TopList;

template <int kK> struct TopList<Bf16, kK> {
    uint32_t a[kK];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < kK; ++j) a[j] = 0;
    }
    // `pos` counts the lane's own elements (0 .. 63), in ascending column order
    __device__ __forceinline__ void insert(uint32_t key, int pos)
    {
        const uint32_t x = (key & 0xFFFF0000u) | (63 - pos);
#pragma unroll
        for (int j = kK - 1; j > 0; --j) a[j] = med3(a[j - 1], a[j], x);
        a[0] = max(a[0], x);
    }
    // own positions -> columns
    template <class F> __device__ __forceinline__ void to_columns(F column)
    {
#pragma unroll
        for (int j = 0; j < kK; ++j) a[j] = (a[j] & 0xFFFF0000u) | (0xFFFF - column(63 - (int)(a[j] & 63)));
    }
    // (the order bits of a negative bf16 end in sixteen ones, which the column's bits replaced)
    __device__ __forceinline__ uint32_t key(int j) const
    {
        const uint32_t k = a[j] & 0xFFFF0000u;
        return (int32_t)k < 0 ? k : k | 0xFFFFu;
    }
    __device__ __forceinline__ int column(int j) const { return 0xFFFF - (int)(a[j] & 0xFFFFu); }
    template <int kStep> __device__ __forceinline__ void take_partner()
    {
        uint32_t b[kK];
#pragma unroll
        for (int j = 0; j < kK; ++j) b[j] = (uint32_t)partner<kStep>((int)a[kK - 1 - j]);
#pragma unroll
        for (int j = 0; j < kK; ++j) a[j] = max(a[j], b[j]);
    }
    __device__ __forceinline__ void order(int i, int j)
    {
        const uint32_t hi = max(a[i], a[j]), lo = min(a[i], a[j]);
        a[i] = hi;
        a[j] = lo;
    }
};

template <int kK> struct TopList<F32, kK> {
    uint32_t a[kK];
    int c[kK];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < kK; ++j) {
            a[j] = 0;
            c[j] = 0x7FFFFFFF;
        }
    }
    __device__ __forceinline__ void insert(uint32_t x, int pos)
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
    template <class F> __device__ __forceinline__ void to_columns(F column)
    {
#pragma unroll
        for (int j = 0; j < kK; ++j) c[j] = c[j] == 0x7FFFFFFF ? c[j] : column(c[j]);
    }
    __device__ __forceinline__ uint32_t key(int j) const { return a[j]; }
    __device__ __forceinline__ int column(int j) const { return c[j]; }
    static __device__ __forceinline__ bool before(uint32_t ka, int ca, uint32_t kb, int cb)
    {
        return ka > kb || (ka == kb && ca < cb);
    }
    template <int kStep> __device__ __forceinline__ void take_partner()
    {
        uint32_t b[kK];
        int d[kK];
#pragma unroll
        for (int j = 0; j < kK; ++j) {
            b[j] = (uint32_t)partner<kStep>((int)a[kK - 1 - j]);
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
        const uint32_t ka = a[i];
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

// Where the chunk with nominal first column `col` is loaded from: the last one of a row whose
// length is no multiple of eight starts at experts - 8 and shares its first columns with its
// neighbour.
__device__ __forceinline__ int chunk_start(int col, int experts) { return max(min(col, experts - 8), 0); }

__device__ __forceinline__ void set_raw(Raw8<Bf16>& r, int j, uint32_t bits)
{
    r.a[j >> 1] = (j & 1) ? (r.a[j >> 1] & 0xFFFFu) | (bits & 0xFFFF0000u) : (r.a[j >> 1] & 0xFFFF0000u) | bits >> 16;
}
__device__ __forceinline__ void set_raw(Raw8<F32>& r, int j, uint32_t bits)
{
    if (j < 4) r.a[j & 3] = bits;
    else r.b[j & 3] = bits;
}
// Eight logits; those that are no columns of this chunk read as -inf.
template <class T, class P>
__device__ __forceinline__ Raw8<T> load_logits(const P* row, int col, int experts, bool live)
{
    const int c0 = chunk_start(col, experts);
    Raw8<T> r = zero8<T>();
    if (live && col < experts) r = experts < 8 ? load_few(row, experts) : load8(row + c0);
    const int lo = live ? col - c0 : 8, hi = experts - c0;   // columns lo .. hi - 1 are the chunk's own
    if (lo > 0 || hi < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < lo || j >= hi) set_raw(r, j, kNegInf);
    }
    return r;
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

template <class T, int kL, int kNC, int kK, bool kLoss>
__global__ __launch_bounds__(kThreads) void router_fwd_kernel(const RouterArgs a)
{
    extern __shared__ int32_t lds[];   // with the loss: counts [experts], sums of p [kWaves][experts]
    __shared__ int32_t routed;
    __shared__ double red[kWaves];
    constexpr int kRows = 64 / kL;     // tokens per wave and step
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int p = lane % kL, slot = lane / kL;
    const int E = a.experts, k = a.top_k;
    const auto* logits = static_cast<const typename T::store_t*>(a.logits);
    int32_t* hist = lds;
    float* sums = reinterpret_cast<float*>(lds + E);

    float acc[kNC][8];
    int n_routed = 0;
    if constexpr (kLoss) {
        for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
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

    const int64_t step = (int64_t)gridDim.x * kWaves * kRows;
    for (int64_t base = ((int64_t)blockIdx.x * kWaves + wave) * kRows; base < a.tokens; base += step) {
        const int64_t t = base + slot;
        bool live = t < a.tokens;
        if (live && a.mask) live = a.mask[t] != 0;
        const auto* row = logits + t * a.ld;
        Raw8<T> raw[kNC];
#pragma unroll
        for (int i = 0; i < kNC; ++i) raw[i] = load_logits<T>(row, (i * kL + p) * 8, E, live);

        TopList<T, kK> top;
        auto select = [&](bool drop_nan) {
            top.clear();
#pragma unroll
            for (int i = 0; i < kNC; ++i) {
                float v[8];
                unpack8(raw[i], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint32_t key = order_bits(v[j]);
                    if (drop_nan) key = key > kOpenInf ? 0 : key;
                    top.insert(key, i * 8 + j);
                }
            }
            top.to_columns([&](int pos) { return chunk_start(((pos >> 3) * kL + p) * 8, E) + (pos & 7); });
            merge_lanes<kL>(top);
        };
        select(false);

        const bool open = top.key(0) > kClosed;
        const float m = open ? from_order_bits(top.key(0)) : 0.0f;
        float s = 0.0f;
        float e[kNC][8];
#pragma unroll
        for (int i = 0; i < kNC; ++i) {
            float v[8];
            unpack8(raw[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                e[i][j] = __expf(v[j] - m);
                s += e[i][j];
            }
        }
        s = sum_lanes<kL>(s);
        // A NaN logit sorts above all others: choose again without it (its weights stay NaN).
        if (__any(s != s)) select(true);
        const bool sent = live && top.key(0) > kClosed;

        const float inv = 1.0f / s;
        float scale = inv;
        if (a.renorm) {
            float w = 0.0f;
#pragma unroll
            for (int j = 0; j < kK; ++j)
                if (j < k && top.key(j) > kClosed) w += expf(from_order_bits(top.key(j)) - m);
            scale = 1.0f / w;
            if (s != s) scale = s;
        }
        // lane p writes entries p, p + kL, ...
#pragma unroll
        for (int j0 = 0; j0 < kK; j0 += kL) {
            uint32_t key = top.key(j0);
            int col = top.column(j0);
#pragma unroll
            for (int q = 1; q < kL && j0 + q < kK; ++q) {
                key = p == q ? top.key(j0 + q) : key;
                col = p == q ? top.column(j0 + q) : col;
            }
            const int j = j0 + p;
            if (j < k && p + j0 < kK && t < a.tokens) {
                const bool chosen = sent && key > kClosed;
                a.index[t * k + j] = chosen ? col : -1;
                a.weight[t * k + j] = chosen ? expf(from_order_bits(key) - m) * scale : 0.0f;
                if constexpr (kLoss)
                    if (chosen) atomicAdd(&hist[col], 1);
            }
        }
        if (a.lse && p == 0 && t < a.tokens) a.lse[t] = sent ? m + logf(s) : 0.0f;
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
        // the wave's tokens side by side (lanes p, p + kL, ...), then the waves
#pragma unroll
        for (int i = 0; i < kNC; ++i) {
            const int col = (i * kL + p) * 8, c0 = chunk_start(col, E);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int s = kL; s < 64; s <<= 1) acc[i][j] += __shfl_xor(acc[i][j], s);
                if (slot == 0 && c0 + j >= col && c0 + j < E) sums[wave * E + c0 + j] = acc[i][j];
            }
        }
        if (n_routed) atomicAdd(&routed, n_routed);
        __syncthreads();
        if (a.workspace) {
            const Space w = space_at(a.workspace, a.blocks, E);
            for (int e = threadIdx.x; e < E; e += kThreads) {
                float s = 0.0f;
                for (int q = 0; q < kWaves; ++q) s += sums[q * E + e];
                w.counts[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
                w.probs[(int64_t)blockIdx.x * E + e] = s;
            }
            if (threadIdx.x == 0) w.counts[(int64_t)blockIdx.x * (E + 1) + E] = routed;
        } else {
            double part = 0.0;
            for (int e = threadIdx.x; e < E; e += kThreads) {
                double s = 0.0;
                for (int q = 0; q < kWaves; ++q) s += (double)sums[q * E + e];
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
    __shared__ int64_t red_c[16][kFinishCols];
    __shared__ double part[kFinishCols];
    const int E = a.experts, cl = threadIdx.x % kFinishCols, rl = threadIdx.x / kFinishCols;
    const int e = blockIdx.x * kFinishCols + cl;
    const Space w = space_at(a.workspace, a.blocks, E);
    double s = 0.0;
    int64_t c = 0;
    if (e <= E) {
#pragma unroll 4
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
        if (e < E) a.counts[e] = (int32_t)c;
        else if (e == E) __hip_atomic_store(a.routed, (int32_t)c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        part[cl] = e < E ? (double)c * s : 0.0;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double v = 0.0;
        for (int i = 0; i < kFinishCols; ++i) v += part[i];
        __hip_atomic_store(&w.sums[blockIdx.x], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        if (__hip_atomic_fetch_add(w.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1) {
            double v = 0.0;
            for (int i = 0; i < (int)gridDim.x; ++i)
                v += __hip_atomic_load(&w.sums[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const int32_t n = __hip_atomic_load(a.routed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            a.loss[0] = balance_loss(v, n, E, a.top_k);
        }
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
template <class T, int kL, int kNC>
__global__ __launch_bounds__(kThreads) void router_bwd_kernel(const RouterBwdArgs a)
{
    constexpr int kRows = 64 / kL, kCols = kL * kNC * 8;
    constexpr int kSlots = (kRouterMaxTopK + kL - 1) / kL;   // entries of a token per lane
    __shared__ __attribute__((aligned(16))) float extra_lds[kWaves][kRows][kCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int p = lane % kL, slot = lane / kL;
    const int E = a.experts, k = a.top_k;
    float* extra = extra_lds[wave][slot];
    for (int c = p * 8; c < kCols; c += kL * 8)
#pragma unroll
        for (int j = 0; j < 8; ++j) extra[c + j] = 0.0f;

    float g[kNC][8];
    float f = 0.0f;
    if (a.d_loss) {
        const float n = (float)max(a.routed[0], 1);
        f = a.d_loss[0] * ((float)E / (float)k) / (n * n);
    }
#pragma unroll
    for (int i = 0; i < kNC; ++i) {
        const int c0 = chunk_start((i * kL + p) * 8, E);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] = a.d_loss && c0 + j < E ? f * (float)a.counts[c0 + j] : 0.0f;
    }

    const auto* logits = static_cast<const typename T::store_t*>(a.logits);
    const int64_t step = (int64_t)gridDim.x * kWaves * kRows;
    for (int64_t base = ((int64_t)blockIdx.x * kWaves + wave) * kRows; base < a.tokens; base += step) {
        const int64_t t = base + slot;
        const bool in = t < a.tokens;
        const auto* row = logits + t * a.ld;
        const bool live = in && a.index[t * k] >= 0;
        Raw8<T> raw[kNC];
#pragma unroll
        for (int i = 0; i < kNC; ++i) raw[i] = load_logits<T>(row, (i * kL + p) * 8, E, live);
        const float lse = live ? a.lse[t] : 0.0f;

        // the chosen columns: entry j0 + p of the token is this lane's
        int pos[kSlots];
        float dw[kSlots], w[kSlots];
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            const int j = q * kL + p;
            int idx = -1;
            pos[q] = -1;
            dw[q] = w[q] = 0.0f;
            if (live && j < k) idx = a.index[t * k + j];
            if (idx >= 0 && idx < E) {
                pos[q] = (idx & ~7) + idx - chunk_start(idx & ~7, E);
                if (a.d_weight) dw[q] = a.d_weight[t * k + j];
                if (a.renorm) {
                    float v;
                    if constexpr (sizeof(row[0]) == 2) v = as_float((uint32_t)row[idx] << 16);
                    else v = row[idx];
                    w[q] = expf(v - lse);
                }
            }
        }
        if (a.renorm) {
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

        float x[kNC][8], pr[kNC][8];
        float dot = 0.0f, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kNC; ++i) {
            const float* src = extra + (i * kL + p) * 8;
            float v[8];
            unpack8(raw[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[i][j] = src[j];
                pr[i][j] = expf(v[j] - lse);
                sum += pr[i][j];
                dot += pr[i][j] * (a.renorm ? g[i][j] : g[i][j] + x[i][j]);
            }
        }
        // (the sum is 1 but for lse's rounding, which matters where lse is large beside the log in it)
        const float inv = 1.0f / sum_lanes<kL>(sum);
        dot = sum_lanes<kL>(dot) * inv;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < kSlots; ++q)
            if (pos[q] >= 0) extra[pos[q]] = 0.0f;

        auto* out = static_cast<typename T::store_t*>(a.d_logits) + t * a.ld_d;
#pragma unroll
        for (int i = 0; i < kNC; ++i) {
            const int col = (i * kL + p) * 8, c0 = chunk_start(col, E);
            float d[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float pj = pr[i][j] * inv;
                d[j] = a.renorm ? pj * (g[i][j] - dot) + x[i][j] : pj * (g[i][j] + x[i][j] - dot);
                if (!live) d[j] = 0.0f;
            }
            if (!in || col >= E) continue;
            const Raw8<T> r = pack8(T{}, d);
            if (col == c0 && c0 + 8 <= E) {
                store8(out + c0, r);
            } else {   // the columns before `col` are the neighbour's
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c0 + j >= col && c0 + j < E) store_one(out + c0 + j, r, j);
            }
        }
    }
}

// Lanes per token and chunks per lane for a number of experts: as few lanes as hold the row with
// at most four chunks each, and eight lanes (one 128-byte line of bf16 per chunk) beyond 16 experts.
struct Shape { int lanes, chunks; };
Shape shape_of(int64_t experts)
{
    if (experts <= 8) return {1, 1};
    if (experts <= 16) return {1, 2};
    if (experts <= 64) return {8, 1};
    if (experts <= 128) return {8, 2};
    if (experts <= 256) return {8, 4};
    if (experts <= 512) return {16, 4};
    return {64, 4};
}

template <class T, int kL, int kNC, int kK>
hipError_t fwd_run(const RouterArgs& a, hipStream_t stream)
{
    const dim3 grid((unsigned)a.blocks);
    if (a.counts) {
        const size_t lds = (size_t)a.experts * 4 * (1 + kWaves);
        router_fwd_kernel<T, kL, kNC, kK, true><<<grid, kThreads, lds, stream>>>(a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || !a.workspace) return e;
        router_finish_kernel<<<(unsigned)finish_blocks(a.experts), 1024, 0, stream>>>(a);
    } else {
        router_fwd_kernel<T, kL, kNC, kK, false><<<grid, kThreads, 0, stream>>>(a);
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
    const int64_t blocks = std::min<int64_t>((a.tokens + per - 1) / per, 2048);
    router_bwd_kernel<T, kL, kNC><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

#define TE_ROUTER_SHAPES(F, T, a, stream)                          \
    do {                                                           \
        const Shape s = shape_of((a).experts);                     \
        if (s.lanes == 1 && s.chunks == 1) return F<T, 1, 1>(a, stream); \
        if (s.lanes == 1) return F<T, 1, 2>(a, stream);            \
        if (s.lanes == 8 && s.chunks == 1) return F<T, 8, 1>(a, stream); \
        if (s.lanes == 8 && s.chunks == 2) return F<T, 8, 2>(a, stream); \
        if (s.lanes == 8) return F<T, 8, 4>(a, stream);            \
        if (s.lanes == 16) return F<T, 16, 4>(a, stream);          \
        return F<T, 64, 4>(a, stream);                             \
    } while (0)

template <class T> hipError_t fwd_shape(const RouterArgs& a, hipStream_t stream) { TE_ROUTER_SHAPES(fwd_k, T, a, stream); }
template <class T> hipError_t bwd_shape(const RouterBwdArgs& a, hipStream_t stream) { TE_ROUTER_SHAPES(bwd_run, T, a, stream); }

}  // namespace

// Workgroups: one where it takes the tokens in at most four steps and the counts are asked for (no
// second kernel then), else up to 1024 of them.
int64_t router_fwd_blocks(int64_t tokens, int64_t experts, bool loss)
{
    const int64_t per = kWaves * (64 / shape_of(experts).lanes);
    const int64_t blocks = (tokens + per - 1) / per;
    if (loss && blocks <= 4) return 1;
    return std::min<int64_t>(blocks, loss ? 1024 : 4096);
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
