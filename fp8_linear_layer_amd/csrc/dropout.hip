// Dropout with the residual's addition, for gfx950:  out = dropout(x) + residual.
//
// Elementwise over chunks of eight columns (one counter of the generator each); a workgroup takes 1024 chunks that
// follow each other, four to a thread, whose loads are all in flight before the first is used.  The row's end that
// fills no chunk goes element by element.  A thread reads its chunks before it writes them and nobody else's, so out
// may be x's or the residual's buffer.  Memory-bound, generator and all: 8192 x 4096 bf16 with the residual 33.4 us (201 MB,
// 6.0 TB/s) with p = 0.1 and 33.1 with p = 0; without the residual 23.2 and 21.3.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "block_internal.h"
#include "dropout_device.h"
#include "ops_device.h"

namespace tefp8 {
namespace {

constexpr int kThreads = 256, kPer = 4, kChunks = kThreads * kPer;

struct None {};

template <class X, class R, class O>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const DropoutArgs a)
{
    constexpr bool kRes = !__is_same(R, None);
    typedef typename X::store_t x_t;
    typedef typename O::store_t o_t;
    const int64_t base = (a.first_block + blockIdx.x) * kChunks;
    const int64_t row0 = base / a.per_row, at0 = base - row0 * a.per_row;
    const DropKey key = drop_key(a.drop);
    int64_t row[kPer];
    int64_t col[kPer];
    int n[kPer];   // columns of the chunk, 0 past the last row
    Raw8<X> rx[kPer];
    Raw8<typename std::conditional<kRes, R, X>::type> rr[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t at = at0 + threadIdx.x + i * kThreads;   // (below per_row + 1024)
        uint32_t over;
        if (a.per_row >= kChunks) over = at >= a.per_row;
        else over = a.per_row == 1 ? (uint32_t)at : __umulhi((uint32_t)at, a.magic);   // (at < 2^11, per_row < 2^10: exact)
        row[i] = row0 + over;
        col[i] = (at - (int64_t)over * a.per_row) * 8;
        n[i] = row[i] < a.rows ? (int)min((int64_t)8, a.cols - col[i]) : 0;
        const x_t* x = static_cast<const x_t*>(a.x) + row[i] * a.ld_x + col[i];
        if (n[i] == 8) rx[i] = load8(x);
        else rx[i] = load_few(x, n[i]);
        if constexpr (kRes) {
            const auto* r = static_cast<const typename R::store_t*>(a.res) + row[i] * a.ld_res + col[i];
            if (n[i] == 8) rr[i] = load8(r);
            else rr[i] = load_few(r, n[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        float v[8];
        unpack8(rx[i], v);
        if (a.drop.below) drop8(a.drop, drop_chunk(a.drop, key, col[i], 0, row[i]), v);
        if constexpr (kRes) {
            float r[8];
            unpack8(rr[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += r[j];
        }
        o_t* o = static_cast<o_t*>(a.out) + row[i] * a.ld_out + col[i];
        if (n[i] == 8) store8(o, pack8(O{}, v));
        else store_few(o, pack8(O{}, v), n[i]);
    }
}

template <class X, class R, class O>
hipError_t run(const DropoutArgs& args, hipStream_t stream)
{
    DropoutArgs a = args;
    const int64_t blocks = (a.rows * a.per_row + kChunks - 1) / kChunks;
    constexpr int64_t kMost = ((int64_t)1 << 31) / kThreads;   // (a launch has at most 2^32 threads)
    for (a.first_block = 0; a.first_block < blocks; a.first_block += kMost)
        dropout_kernel<X, R, O><<<(unsigned)std::min(kMost, blocks - a.first_block), kThreads, 0, stream>>>(a);
    return hipGetLastError();
}
template <class X, class R>
hipError_t run_out(const DropoutArgs& a, hipStream_t stream)
{
    return a.out_bf16 ? run<X, R, Bf16>(a, stream) : run<X, R, F32>(a, stream);
}
template <class X>
hipError_t run_res(const DropoutArgs& a, hipStream_t stream)
{
    if (!a.res) return run_out<X, None>(a, stream);
    return a.res_bf16 ? run_out<X, Bf16>(a, stream) : run_out<X, F32>(a, stream);
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& args, hipStream_t stream)
{
    DropoutArgs a = args;
    if (a.rows <= 0) return hipSuccess;
    a.per_row = (a.cols + 7) / 8;
    a.magic = a.per_row > 1 && a.per_row < kChunks ? (uint32_t)((((uint64_t)1 << 32) + a.per_row - 1) / a.per_row) : 0;
    return a.x_bf16 ? run_res<Bf16>(a, stream) : run_res<F32>(a, stream);
}

}  // namespace tefp8
