// Device pieces shared by the operators around the GEMMs (norm.hip, router.hip, grad_clip.hip):
// eight-element loads and stores of bf16 and fp32 at any element alignment, and reductions over
// the lanes of a wavefront.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tefp8 {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
// The same sixteen bytes at the alignment of one element.  Global memory instructions of up to
// sixteen bytes take any address on this target, so rows of odd length or stride need no other path.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t uint32_a2 __attribute__((aligned(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// (the arguments by value: a bit cast of a vector's element in place reads its first element)
__device__ __forceinline__ float as_float(uint32_t b) { return __builtin_bit_cast(float, b); }
__device__ __forceinline__ uint32_t as_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

struct Bf16 {
    typedef uint16_t store_t;
};
struct F32 {
    typedef float store_t;
};

// fp32 -> bf16 rounds to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){lo, hi}, bf16x2_t));
}

// Eight raw elements as loaded, so that several loads can be in flight before the first is used.
template <class T> struct Raw8;
template <> struct Raw8<Bf16> { u32x4_t a; };
template <> struct Raw8<F32> { u32x4_t a, b; };

__device__ __forceinline__ Raw8<Bf16> load8(const uint16_t* p)
{
    return {*reinterpret_cast<const u32x4_a2*>(p)};
}
__device__ __forceinline__ Raw8<F32> load8(const float* p)
{
    return {*reinterpret_cast<const u32x4_a4*>(p), *reinterpret_cast<const u32x4_a4*>(p + 4)};
}
// n < 8 elements, and behind them `fill` (the bits of an fp32 number that bf16 holds too).
__device__ __forceinline__ Raw8<Bf16> load_few(const uint16_t* p, int n, uint32_t fill = 0)
{
    Raw8<Bf16> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < n ? p[2 * i] : fill >> 16, hi = 2 * i + 1 < n ? p[2 * i + 1] : fill >> 16;
        r.a[i] = lo | hi << 16;
    }
    return r;
}
__device__ __forceinline__ Raw8<F32> load_few(const float* p, int n, uint32_t fill = 0)
{
    Raw8<F32> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.a[i] = i < n ? as_bits(p[i]) : fill;
        r.b[i] = 4 + i < n ? as_bits(p[4 + i]) : fill;
    }
    return r;
}
// Elements n .. 7 to the front, and `fill` behind them (0 <= n < 8).
__device__ __forceinline__ Raw8<Bf16> drop_front(Raw8<Bf16> r, int n, uint32_t fill)
{
    const uint32_t f = fill | fill >> 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t next = i < 3 ? (uint32_t)r.a[i + 1 & 3] : f;
        r.a[i] = n & 1 ? r.a[i] >> 16 | next << 16 : (uint32_t)r.a[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) r.a[i] = n & 2 ? (i < 3 ? (uint32_t)r.a[i + 1 & 3] : f) : (uint32_t)r.a[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) r.a[i] = n & 4 ? (i < 2 ? (uint32_t)r.a[i + 2 & 3] : f) : (uint32_t)r.a[i];
    return r;
}
__device__ __forceinline__ Raw8<F32> drop_front(Raw8<F32> r, int n, uint32_t fill)
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < 4 ? (uint32_t)r.a[i & 3] : (uint32_t)r.b[i & 3];
#pragma unroll
    for (int s = 1; s <= 4; s *= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = n & s ? (i + s < 8 ? w[i + s & 7] : fill) : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.a[i] = w[i];
        r.b[i] = w[4 + i];
    }
    return r;
}
template <class T> __device__ __forceinline__ Raw8<T> zero8();
template <class T> __device__ __forceinline__ Raw8<T> fill8(uint32_t fill);
template <> __device__ __forceinline__ Raw8<Bf16> fill8<Bf16>(uint32_t f)
{
    f |= f >> 16;
    return {u32x4_t{f, f, f, f}};
}
template <> __device__ __forceinline__ Raw8<F32> fill8<F32>(uint32_t f) { return {u32x4_t{f, f, f, f}, u32x4_t{f, f, f, f}}; }
template <> __device__ __forceinline__ Raw8<Bf16> zero8<Bf16>() { return {u32x4_t{0, 0, 0, 0}}; }
template <> __device__ __forceinline__ Raw8<F32> zero8<F32>() { return {u32x4_t{0, 0, 0, 0}, u32x4_t{0, 0, 0, 0}}; }

__device__ __forceinline__ void unpack8(const Raw8<Bf16>& r, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = as_float(r.a[i] << 16);
        v[2 * i + 1] = as_float(r.a[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack8(const Raw8<F32>& r, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = as_float(r.a[i]);
        v[4 + i] = as_float(r.b[i]);
    }
}
__device__ __forceinline__ Raw8<Bf16> pack8(Bf16, const float (&v)[8])
{
    return {u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])}};
}
__device__ __forceinline__ Raw8<F32> pack8(F32, const float (&v)[8])
{
    Raw8<F32> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.a[i] = as_bits(v[i]);
        r.b[i] = as_bits(v[4 + i]);
    }
    return r;
}
__device__ __forceinline__ void store8(uint16_t* p, const Raw8<Bf16>& r) { *reinterpret_cast<u32x4_a2*>(p) = r.a; }
__device__ __forceinline__ void store8(float* p, const Raw8<F32>& r)
{
    *reinterpret_cast<u32x4_a4*>(p) = r.a;
    *reinterpret_cast<u32x4_a4*>(p + 4) = r.b;
}
__device__ __forceinline__ void store_one(uint16_t* p, const Raw8<Bf16>& r, int i)
{
    *p = (uint16_t)(r.a[i >> 1] >> (16 * (i & 1)));
}
__device__ __forceinline__ void store_one(float* p, const Raw8<F32>& r, int i)
{
    *p = i < 4 ? as_float(r.a[i & 3]) : as_float(r.b[i & 3]);
}
template <class P, class R>
__device__ __forceinline__ void store_few(P* p, const R& r, int n)   // n < 8
{
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) store_one(p + i, r, i);
}

// Lane exchanges: within 16 lanes by DPP (no LDS), across the halves and quarters of the wave by
// permutes.  After step s every lane holds the result over its aligned group of 2 s lanes.
template <int kCtrl>
__device__ __forceinline__ int dpp(int v)
{
    // (every lane's source is inside its row; said this way the exchange folds into the instruction that uses it)
    return __builtin_amdgcn_update_dpp(0, v, kCtrl, 0xF, 0xF, true);
}
// The value of a partner lane in the other half of the aligned group of 2 * kStep lanes, for
// values that are already equal over each aligned group of kStep lanes.
template <int kStep>
__device__ __forceinline__ int partner(int v)
{
    if (kStep == 1) return dpp<0xB1>(v);    // quad_perm [1,0,3,2]
    if (kStep == 2) return dpp<0x4E>(v);    // quad_perm [2,3,0,1]
    if (kStep == 4) return dpp<0x141>(v);   // lane i <-> 7-i within each half row
    if (kStep == 8) return dpp<0x140>(v);   // lane i <-> 15-i within each row
    return __shfl_xor(v, kStep);
}
template <int kStep>
__device__ __forceinline__ float partner(float v)
{
    return __builtin_bit_cast(float, partner<kStep>(__builtin_bit_cast(int, v)));
}
// Sum over aligned groups of kLanes lanes, in every lane; the order of the additions is fixed.
template <int kLanes>
__device__ __forceinline__ float sum_lanes(float v)
{
    if (kLanes > 1) v += partner<1>(v);
    if (kLanes > 2) v += partner<2>(v);
    if (kLanes > 4) v += partner<4>(v);
    if (kLanes > 8) v += partner<8>(v);
    if (kLanes > 16) v += partner<16>(v);
    if (kLanes > 32) v += partner<32>(v);
    return v;
}
template <int kLanes>
__device__ __forceinline__ uint32_t max_lanes(uint32_t v)
{
    if (kLanes > 1) v = max(v, (uint32_t)partner<1>((int)v));
    if (kLanes > 2) v = max(v, (uint32_t)partner<2>((int)v));
    if (kLanes > 4) v = max(v, (uint32_t)partner<4>((int)v));
    if (kLanes > 8) v = max(v, (uint32_t)partner<8>((int)v));
    if (kLanes > 16) v = max(v, (uint32_t)partner<16>((int)v));
    if (kLanes > 32) v = max(v, (uint32_t)partner<32>((int)v));
    return v;
}

// Workgroups go to the eight XCDs in turn; this order gives each XCD (and its L2) a run of
// consecutive work items instead.  A permutation of 0 .. n-1.
__device__ __forceinline__ int64_t xcd_run(int64_t b, int64_t n)
{
    const int64_t q = n / 8, r = n % 8, x = b % 8;
    return x * q + (x < r ? x : r) + b / 8;
}

}  // namespace tefp8
