// The norm before the head, its gradient, and 8-bit checkpoints of activations
// (see "the norm before the head" in grpo.h): what norm_fwd.cu, norm_bwd.cu,
// norm_ckpt.cu, norm_plan.cu and norm_abi.cu share.
#pragma once
#include "internal.h"

namespace grpo {

constexpr int kNormMaxD = 16384;       // widest row of the norm (a row stays in one block)
constexpr int kSmCount = 152;          // of a GB300: what the gradient's workspace is sized for
constexpr int kClusterMax = 8;
constexpr int kUnit = 16;              // elements of a thread's load: a 32-byte sector of a 16-bit matrix
constexpr int kWarpThreads = 128;      // block whose warps, or parts of them, take a row each
constexpr int kBlockMax = 512;         // widest block that takes a row as a whole
constexpr int kCkptBlock = GRPO_CKPT_BLOCK;
constexpr float kLeastScale = 1.17549435e-38f;   // 2^-126: its reciprocal is finite, and neither is subnormal

// s comes from x (+ residual), or from a checkpoint (codes, scales).
struct NormParams {
    const uint16_t* x;
    const uint16_t* residual;
    const int8_t* codes;
    const uint16_t* scales;      // bf16, one for each kCkptBlock columns of a row
    const void* weight;
    const uint8_t* mask;         // nullable
    int64_t N;
    int d;
    float eps;
    int weight_f32;
    float plus;                  // added to the weight: 0 or 1
    int width;                   // threads of a row
    int y_type;                  // grpo_dtype of y
    float y_inv;                 // 1 / the given scale, 0: a scale per row
    // outputs of the forward pass, null where not wanted
    void* y;
    float* row_scale;
    uint16_t* sum;
    int8_t* codes_out;
    uint16_t* scales_out;
    // the gradient
    const uint16_t* dy;
    const uint16_t* dsum;        // nullable
    uint16_t* dx;
    void* dweight;               // nullable
    float* part;                 // [parts x d]
    int* bad;                    // [parts] whether a part met a gradient that is not finite (1), or a wait ran out (2)
    int parts;
    bool joined;                 // the blocks are one cluster and join their sums themselves
    int stages;                  // of the ring that rows are copied into
    int* found_inf;
};

struct CkptParams {
    const uint16_t* x;           // pack: the source; unpack: unused
    uint16_t* x_out;
    const int8_t* codes;
    const uint16_t* scales;
    int8_t* codes_out;
    uint16_t* scales_out;
    const uint8_t* mask;
    int64_t N;
    int d;
    uint64_t per_row;            // ceil(2^64 / (d / 16)): the row of a unit by a product
};

// How a row is dealt to threads, and rows to blocks.
struct NormPlan {
    int width, upt;              // threads of a row, and units of 16 elements that each has
    int threads, grid, per_sm;   // of a block; blocks, and how many of them an SM is to have
    bool wide;                   // a row takes whole warps (else some lanes of one)
    bool joined = false;         // the blocks are one cluster (a power of two of them) and join their sums
};
NormPlan norm_fwd_plan(int64_t N, int d, int sm_count);
NormPlan norm_bwd_plan(int64_t N, int d, int sm_count, bool ckpt, bool dsum);
int norm_parts(int64_t N, int d);    // most blocks of norm_bwd_plan on kSmCount SMs

cudaError_t launch_norm_fwd(const NormParams& p, const NormPlan& o, bool bf16, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormParams& p, const NormPlan& o, bool bf16, cudaStream_t st);
cudaError_t launch_norm_join(const NormParams& p, bool bf16, cudaStream_t st);
cudaError_t launch_ckpt_pack(const CkptParams& p, bool bf16, cudaStream_t st);
cudaError_t launch_ckpt_unpack(const CkptParams& p, bool bf16, cudaStream_t st);

}  // namespace grpo
