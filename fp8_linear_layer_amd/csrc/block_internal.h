// Internal interface between the C-ABI front end of a gated block's operators (api_block.cpp) and their
// gfx950 kernels (gated.hip, gated_few.hip, layernorm.hip, dropout.hip).  Not installed; not part of the ABI.
#pragma once

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "internal.h"
#include "ops_internal.h"

namespace tefp8 {

// ------------------------------------------------------------ dropout
// An element whose 16 bits, as the high half of a word, are below `below` is dropped (0: no dropout).
struct Drop {
    const int64_t* rng;   // seed, number of the call
    uint32_t below;
    uint32_t all;         // everything is dropped
    float factor;         // of the kept
};

struct DropoutArgs {
    const void* x;
    const void* res;      // or null
    void* out;
    int64_t rows, cols, ld_x, ld_res, ld_out;
    bool x_bf16, res_bf16, out_bf16;
    Drop drop;
    // set by the launcher:
    int64_t per_row, first_block;   // chunks of eight columns in a row; of this launch
    uint32_t magic;                 // 2^32 / per_row, rounded up
};
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t stream);

// ------------------------------------------------------------ layer norm
struct LayerNormFwdArgs {
    const void* x;          // [rows][ld_x] bf16 or fp32
    const void* res;        // [rows][ld_res] bf16 or fp32, or null
    const uint16_t* gamma;  // [cols] bf16
    const uint16_t* beta;   // [cols] bf16, or null
    void* h;                // [rows][ld_h], the residual's type; null without a residual
    float* mean;            // [rows]
    float* rstd;            // [rows]
    void* y;                // bf16 / fp32 [rows][ld_y], or fp8 codes (may be null: transpose only)
    float* scales;          // [cols/128][ld_s]
    uint8_t* qt;            // [cols][ld_qt] or null
    float* scales_t;        // [rows/128][ld_st]
    const void* src;        // what the transposed cast reads: h, or x without a residual
    int64_t rows;
    int64_t ld_x, ld_res, ld_h, ld_y, ld_s, ld_qt, ld_st, ld_src;
    int cols;
    float eps;
    bool x_bf16, h_bf16, src_bf16;
    NormOut out;
    int fmt, pow2;
    Drop drop;              // of x; only with a residual
    // set by the launcher:
    int64_t first_row;      // of this launch
    double inv_cols;        // 1 / cols
    bool past;              // read past the caches
};
hipError_t launch_layernorm_fwd(const LayerNormFwdArgs& a, hipStream_t stream);

struct LayerNormBwdArgs {
    const void* dy;         // [rows][ld_dy] bf16 or fp32
    const void* h;          // [rows][ld_h] bf16 or fp32
    const float* mean;      // [rows]
    const float* rstd;      // [rows]
    const uint16_t* gamma;  // [cols] bf16
    const void* dres;       // [rows][ld_dres], h's type, or null
    void* dh;               // [rows][ld_dh], h's type
    void* dx;               // [rows][ld_dx] bf16 or fp32, or null
    float* dgamma;          // [cols] or null
    float* dbeta;           // [cols] or null
    float* partial;         // [blocks][2][ld_partial], or null: neither sum wanted
    int64_t rows, blocks;
    int64_t ld_dy, ld_h, ld_dres, ld_dh, ld_dx, ld_partial;
    int cols;
    bool dy_bf16, h_bf16, dx_bf16;
    Drop drop;
    float inv_cols;         // 1 / cols, set by the launcher
};
int64_t layernorm_bwd_blocks(int64_t rows, int64_t cols);
hipError_t launch_layernorm_bwd(const LayerNormBwdArgs& a, hipStream_t stream);

// ------------------------------------------------------------ gated feed-forward
enum class Act : int { Silu = 1, Gelu = 2 };

// The GEMM's arguments (a, b, scales, M, N = 2 H of the forward and H of the data gradient, one group), with
//   forward:  out (y, plain), q_out / q_scales / qt_out / qt_scales (y, fp8), aux (z, or null)
//   dgrad:    out (dz, plain), q_out ... (dz, fp8), preact (z)
// and flags = the activation.
// Most rows of the kernel for few tokens, whose sums are exact but for fp32 roundings in any batch of up to so many.  It is
// not always the faster one (us by it and by the parts of gated.hip, K -> H, at 16, 32, 64
// and 128 rows): 7168 -> 2048 12.2, 29.0; 14.5, 29.5; 20.5, 31.4; 21.3, 30.9.  2048 -> 1024 4.5, 10.3; 5.7, 10.4; 8.4, 10.5; 8.7,
// 10.6.  4096 -> 7168 16.6, 20.1; 19.8, 20.5; 28.4, 21.7; 37.4, 21.7.  4096 -> 14336 27.3, 31.8; 33.4, 30.7; 41.6, 30.8; 62.9, 39.1.
constexpr int64_t kFewRows = 128;
// Whether the row-wise cast of y reads fp32 rows that the large products' kernels left in the workspace.
bool gated_fwd_through_f32(int64_t M, int64_t H);
hipError_t launch_gated_fwd(const GemmArgs& a, hipStream_t stream);
hipError_t launch_gated_dgrad(const GemmArgs& a, hipStream_t stream);
// The forward of up to kFewRows rows; fp8 outputs have the sums in the workspace.
int64_t gated_few_workspace_bytes(int64_t M, int64_t N, bool fp8);
hipError_t launch_gated_few(const GemmArgs& a, int64_t K, void* workspace, hipStream_t stream);
// The per-token cast of fp32 rows; cols a multiple of 128.
hipError_t launch_cast_f32_rows(const float* x, int64_t rows, int64_t cols, int64_t ld_x, int fmt, bool pow2, uint8_t* q,
                                int64_t ld_q, float* scales, int64_t ld_s, hipStream_t stream);

}  // namespace tefp8
