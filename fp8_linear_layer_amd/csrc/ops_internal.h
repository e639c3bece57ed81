// Internal interface between the C-ABI front end of the operators around the GEMMs (api_ops.cpp)
// and their gfx950 kernels (norm.hip, router.hip, grad_clip.hip).  Not installed; not part of the ABI.
#pragma once

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "te_fp8.h"

namespace tefp8 {

// The calling thread's error text (api.cpp): report() stores a failure and returns its status,
// report_ok() clears it.
te_status_t report(te_status_t status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
te_status_t report_ok();
bool log_calls();

// ------------------------------------------------------------ root-mean-square norm
constexpr int kNormMaxCols = 32768;   // a row fits the registers of one workgroup (forward)
enum class NormOut : int { Bf16, F32, Fp8 };

struct NormFwdArgs {
    const void* x;          // [rows][ld_x] bf16 or fp32
    const void* res;        // [rows][ld_res] bf16 or fp32, or null
    const uint16_t* gamma;  // [cols] bf16
    void* h;                // [rows][ld_h], the residual's type; null without a residual
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
    // set by the launcher:
    int64_t first_row;      // of this launch
    bool past;              // read past the caches
    NormOut out;
    int fmt, pow2;
};
hipError_t launch_rmsnorm_fwd(const NormFwdArgs& a, hipStream_t stream);

struct NormBwdArgs {
    const void* dy;         // [rows][ld_dy] bf16 or fp32
    const void* h;          // [rows][ld_h] bf16 or fp32
    const float* rstd;      // [rows]
    const uint16_t* gamma;  // [cols] bf16
    const void* dres;       // [rows][ld_dres], h's type, or null
    void* dh;               // [rows][ld_dh], h's type
    float* dgamma;          // [cols]
    float* partial;         // [blocks][ld_partial]
    int64_t rows, blocks;
    int64_t ld_dy, ld_h, ld_dres, ld_dh, ld_partial;
    int cols;
    bool dy_bf16, h_bf16;
};
int64_t rmsnorm_bwd_blocks(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, hipStream_t stream);

// ------------------------------------------------------------ top-k router
constexpr int kRouterMaxExperts = 2048;
constexpr int kRouterMaxTopK = 16;

struct RouterArgs {
    const void* logits;      // [tokens][ld] bf16 or fp32
    const uint8_t* mask;     // [tokens] or null
    int64_t tokens, ld;
    int experts, top_k;
    bool bf16, renorm;
    int32_t* index;          // [tokens][top_k]
    float* weight;           // [tokens][top_k]
    float* lse;              // [tokens] or null
    int32_t* counts;         // [experts]; null: no counts and no loss
    int32_t* routed;         // [1]
    float* loss;             // [1]
    void* workspace;         // null: one workgroup
    int64_t blocks;
};
int64_t router_fwd_blocks(int64_t tokens, int64_t experts, bool loss);
int64_t router_fwd_workspace_bytes(int64_t tokens, int64_t experts);
hipError_t launch_router_fwd(const RouterArgs& a, hipStream_t stream);

struct RouterBwdArgs {
    const void* logits;      // [tokens][ld] bf16 or fp32
    int64_t tokens, ld;
    int experts, top_k;
    bool bf16, renorm;
    const int32_t* index;    // [tokens][top_k]
    const float* lse;        // [tokens]
    const float* d_weight;   // [tokens][top_k] or null
    const int32_t* counts;   // [experts], with d_loss
    const int32_t* routed;   // [1], with d_loss
    const float* d_loss;     // [1] or null
    void* d_logits;          // [tokens][ld_d], the logits' type
    int64_t ld_d;
};
hipError_t launch_router_bwd(const RouterBwdArgs& a, hipStream_t stream);

// ------------------------------------------------------------ gradient norm and clipping
// Tensors of one launch: their descriptors travel in the kernel's arguments (at most 4 KiB).
constexpr int kClipBatch = 96;
// Gradients of this many bytes in a call go past the caches: twice the last cache's size.  Both passes, gradients just
// written by another kernel, ordinarily and past the caches: fp32 into bf16 256 MiB 116.7 and 131.9 us, 512 MiB
// 296.2 and 270.1; bf16 into bf16 256 MiB 150.4 and 167.1, 512 MiB 345.4 and 326.2 (bf16 into fp32, whose stores are
// half lines, 498.3 and 516.6).  Gradients that nothing has touched gain 3 to 6 % from 256 MiB on.
constexpr int64_t kClipPast = (int64_t)1 << 29;
constexpr int kClipBlocks = 1024;   // most workgroups of a launch; each has a slot for its sum, shared by the launches

struct ClipTensor {
    const void* grad;
    void* out;
    int64_t n;
};
struct ClipBatch {
    ClipTensor t[kClipBatch];
    int32_t first[kClipBatch];   // first chunk of each tensor
    uint8_t types[kClipBatch];   // bit 0: bf16 gradient, bit 1: bf16 output
    int32_t n, chunks;
};
int64_t clip_chunks(int64_t n);
int64_t clip_blocks(const ClipBatch& b);
int64_t clip_workspace_bytes();
// `have` sums are there from earlier launches; `past`: read and written past the caches.
hipError_t launch_grad_sumsq(const ClipBatch& b, double* partial, int64_t have, bool past, hipStream_t stream);
hipError_t launch_grad_scale(const ClipBatch& b, const double* partial, int64_t slots, float max_norm, float* norm,
                             bool past, hipStream_t stream);

}  // namespace tefp8
