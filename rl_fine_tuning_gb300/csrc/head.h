// Declarations of the head operators: log-probs of given tokens, the clipped
// policy loss and the preference loss, all from hidden states and W.
//
// One call runs, per chunk of masked-in rows (at most R of them):
//   gather     compact (and transposed) copies of the rows; the given token's
//              logit of each row by itself
//   logits     z = h . W^T, streaming (max, sum exp, sum z exp); with a
//              backward the exponentials stay in the chunk buffer
//   merge      per row: logsumexp, q, entropy; the operator's d loss / d q
//   dlogits, dH, dW
// A chunk's bounds, like every count, are device data (k_plan).
#pragma once
#include "internal.h"

namespace grpo {

enum HeadMode {
    HEAD_LOGP = 0,    // q and entropy out
    HEAD_GRAD = 1,    // d loss / d q is an input
    HEAD_CLIP = 2,    // clipped policy loss
    HEAD_PAIR = 3     // preference loss: d loss / d q follows from sums over pairs of completions
};

constexpr int kPieceK = 1024;       // K elements the tensor cores add up before the sum moves to registers
constexpr int kHeadThreads = 384;   // a warpgroup with the producer and MMA warps, two of epilogue warps
constexpr int kHeadSplitsMax = 512;    // vocabulary splits of the logits kernel
constexpr int kHeadChunkTiles = 76;    // default rows per chunk, in tiles of 128
// SM pairs of a GB300, for what the host lays out before it asks the device: the size of
// the workspace and dH's unit width.  The launches and k_plan go by the device's own
// count; on another count these would only be less well tuned.
constexpr int kSmPairs = 76;
constexpr int kDhSlotsMax = 4 * kSmPairs;   // 256 x 256 partial tiles of dH (80 MB)
constexpr int kDhWideSlotsMax = 256;  // 256 x 512 ones
constexpr int kFewRows = 32;        // rows of the few-row kernel
constexpr int kFewCtas = 256;          // most CTAs of the few-row kernel
constexpr int kFewVocab = 128;      // vocabulary rows per tile of the few-row kernel
// what stands for a logit that does not count (the given token's own, columns
// past V): finite, so no inf - inf can form, far below every logit, and a
// power of two, so its product with log2 e is that constant's rounding, exactly
constexpr float kNoLogit = -1267650600228229401496703205376.f;   // -2^100
constexpr float kNoLogit2 = kNoLogit * 1.4426950408889634f;
// Correction of the tensor cores' rounding towards zero, for the logits: n additions
// of terms of one size make a sum too small by kAddLoss n of itself (see head_tc.cu)
constexpr double kAddLoss = 1.45e-8;
// A chunk with a row whose q is below this takes dlogits relative to the running
// maximum instead of to the given token (see k_head_scale): bf16 would hold
// p_v / p_tok up to e^88, but g p_tok h has to stay a normal number as well, and with
// p_tok >= e^-40 it does for every |g h| above 3e-21.
constexpr float kLeastQ = -40.f;

struct PlanParams {
    const uint8_t* mask;    // nullptr: every row counts
    int64_t N;
    int L, n_seq, R;
    int by_pair;            // chunks of whole pairs of completions
    int pairs_of_g2;        // completions 2i and 2i + 1 are a pair: count pairs, not completions, with a valid row
    int max_chunks;
    int n_nt, ks, n_pairs, slots_max;   // dH: d tiles, K-stages, SM pairs, partial tiles
    int backward;
    int n_w;                // dW units in dH's launch (0: dW has its own)
    int* counts;
    int* off;               // [n_seq + 1] valid rows before completion i
    int* cb;                // [max_chunks + 1] first valid row of chunk c
    int* pb;                // [max_chunks + 1] first pair of chunk c (by_pair)
    int2* dh_plan;          // [max_chunks] (units in one piece, K pieces of the rest)
    int2* lg_plan;          // [max_chunks] (vocabulary splits, tiles per split) of the logits kernel
    int n_ntiles, s_max;    // vocabulary tiles, most splits
    unsigned* gmax;         // [max_chunks] largest |d loss / d q| (float bits), zeroed
    int* far;               // [max_chunks], zeroed
    int* rows;              // [N] valid rows, ascending
    int* found_inf;         // nullable, zeroed
    float* loss;            // nullable, zeroed: what it is when no row counts
    int* status;            // zeroed
};

struct GatherParams {
    const int* counts;
    const int* cb;
    const int* rows;
    const int* tokens;
    const uint8_t* mask;
    const uint16_t* h;
    const uint16_t* W;
    uint16_t* hc;           // [R x d]
    uint16_t* hct;          // [d x R], nullable
    double* zt;             // [N] logit of the given token
    uint16_t* dH;           // nullable: rows of masked rows are zeroed with chunk 0
    void* dW;               // nullable: zeroed with chunk 0 when no row counts
    int64_t dw_bytes;
    float* out0;            // nullable per-row outputs, zeroed on masked rows with chunk 0
    float* out1;
    float* stats;           // [N x 3]
    float zscale;
    int64_t N;
    int d, V, R, chunk;
    int* status;
};

// What the logits kernel keeps
enum LogitsMode {
    LG_STATS = 0,      // (m, s) per row
    LG_ENTROPY = 1,    // (m, s, u)
    LG_KEEP_MAX = 2,   // (m, s) and the exponentials relative to the running maximum, fp16
    LG_KEEP_TOKEN = 3  // s and the exponentials relative to the given token's logit, bf16
};

struct LogitsParams {
    const int* counts;
    const int* cb;
    const int* rows;
    const int* tokens;
    const double* zt;       // [N] logit of the given token (LG_KEEP_TOKEN)
    const int* only_if;     // nullable: nothing to do unless *only_if
    float4* part;           // [R x 2S] (m, s, u, -) of each half split, m in base 2
    uint16_t* E;            // [R x V_pad] exponentials; nullptr (LG_KEEP_TOKEN): not stored
    float* mx;              // [R x nc32] running max per 32 columns, base 2
    float zscale;           // logit = zscale * accumulator: 1 / temperature and the rounding's correction
    float zscale2;          // zscale log2 e
    int64_t N;
    const int2* plan;       // [max_chunks] (S, nps)
    int chunk, V, d, n_ntiles, V_pad, nc32, R;
    int* status;
};

struct FewParams {
    const int* tokens;
    const uint8_t* mask;    // nullable
    const double* zt;       // [N] logit of the given token
    float4* part;           // [N x grid]
    int* counter;
    float* logp;
    float* entropy;         // nullable
    float inv_t;            // 1 / temperature
    float zscale, zscale2;  // as in LogitsParams
    int N, V, d, n_tiles;
    int* status;
};

struct HeadMergeParams {
    const float4* part;
    const int2* plan;       // [max_chunks] (S, nps): 2 S partials a row
    int relative;           // the partials are relative to the given token's logit (LG_KEEP_TOKEN)
    const int* only_if;     // nullable: nothing to do unless *only_if
    int* far;               // nullable: [max_chunks] <- 1 if a row of the chunk has q < kLeastQ
    const int* counts;
    const int* cb;
    const int* off;
    const int* rows;
    const int* tokens;
    const double* zt;
    float2* lse2;           // [N] logsumexp in base 2, as the sum of two numbers
    float* gco;
    float* ell;
    unsigned* gmax;
    float* logp;            // nullable [N]
    float* entropy;         // nullable [N]
    const float* dlogp;     // HEAD_GRAD
    const float* adv;       // HEAD_CLIP ...
    const float* logp_old;
    const float* logp_ref;  // nullable
    float* stats;           // nullable [N x 3]
    float beta, clip_lo, clip_hi, inv_t;
    int mode, loss_mode, chunk, L, V, R;
    int64_t N;
    int* status;
};

struct PairParams {
    const int* counts;
    const int* off;
    const int* pb;          // nullptr: every pair
    const int* rows;
    const int* tokens;
    const float* logp;
    const float* logp_ref;
    float* gco;
    unsigned* gmax;         // of this chunk
    double* pair_ell;       // [n_pairs]
    float* pair_stats;      // nullable [n_pairs x 4]
    float beta, smoothing;
    int kind, length_mean, n_pairs, chunk, V;
    int64_t N;
    int* status;
};

struct LossParams {
    const float* ell;        // weighted objective per valid row, or nullptr
    const double* pair_ell;  // per pair, or nullptr
    int n_pairs;
    float* loss;             // nullptr: nothing to do
};

// ChunkParams of the head operators' GEMMs
struct HeadChunkParams : ChunkParams {
    CUtensorMap mHct;       // hct, dW's B operand
    LossParams loss;        // written with the last chunk that has rows
    float* dw_acc;          // fp32 dW (the caller's, or the workspace's when dw16 is given and there are several chunks)
    uint16_t* dw16;         // 16-bit dW, nullable
    float* dh_part;         // [slots][256 x dh_cols] fp32
    int dh_cols;            // columns of a dH unit: 256 or 512
    const int2* dh_plan;
    const float* logp;      // [N] q
    const float2* lse2;     // [N] logsumexp in base 2, as the sum of two numbers
    const double* zt;       // [N] logit of the given token
    float* rowf;            // nullable: [R] factor of a dlogits row (relative dlogits)
    uint16_t* hct;          // [d x R]
    const uint16_t* hc;     // [R x d]
    const int* far;         // nullable: [max_chunks]
    const unsigned* gmax;
    int gmax_chunk;         // which entry of gmax holds this chunk's
    float loss_scale;
};

// dH's share of the same rounding.  A dH row is almost the given token's own term,
// g (1 - p_tok) W[tok]: the other tokens' terms mostly cancel.  So the running sum
// has its final size from that token's place on, and each addition after it takes
// kTokenLoss of it: measured 3.2e-8 to 3.4e-8 with tokens at the start, the quarters
// and near the end of a vocabulary of 100352 (1.9e-4 of dH at the start, nothing at
// the end, which fp16 outputs would show).  piece: vocabulary rows of a K piece, V where
// the sum is whole.  What another likely token's term loses is not covered.  Up to
// kEvenVocab tokens the whole correction is below 1.7e-5, a thirtieth of fp16's half
// step, and the epilogue goes without the load of the token.
constexpr float kTokenLoss = 3.2e-8f;
constexpr int kEvenVocab = 8192;

__device__ __forceinline__ float dh_gain(int tok, int V, int piece) {
    const int t = min(max(tok, 0), V - 1);   // a bad token's row is 0
    return 1.f + kTokenLoss * static_cast<float>(min(piece - t % piece, V - t) / 16);
}

cudaError_t launch_plan(const PlanParams& p, cudaStream_t st);
cudaError_t launch_head_gather(const GatherParams& p, bool bf16, int sm_count, cudaStream_t st);
cudaError_t launch_head_logits(const LogitsParams& p, const CUtensorMap& mH, const CUtensorMap& mW, int n_sm, bool bf16,
                               int mode, cudaStream_t st);
cudaError_t launch_head_merge(const HeadMergeParams& p, cudaStream_t st);
cudaError_t launch_pair_coef(const PairParams& p, cudaStream_t st);
cudaError_t launch_head_dlogits(const HeadChunkParams& p, float* oscale, bool bf16, int sm_count, cudaStream_t st);
cudaError_t launch_merge_dlogits(const HeadMergeParams& m, const HeadChunkParams& p, float* oscale, int sm_count,
                                 cudaStream_t st);
cudaError_t launch_head_scale(const HeadChunkParams& p, float* oscale, int sm_count, cudaStream_t st);
cudaError_t launch_head_grads(const HeadChunkParams& p, const CUtensorMap& mDS, const CUtensorMap& mDSmn,
                              const CUtensorMap& mWmn, int n_sm, bool bf16, cudaStream_t st);
cudaError_t launch_head_dh(const HeadChunkParams& p, const CUtensorMap& mDS, const CUtensorMap& mWmn, int n_sm, bool bf16,
                           cudaStream_t st);
cudaError_t launch_head_dw(const HeadChunkParams& p, const CUtensorMap& mDSmn, int n_sm, bool bf16, cudaStream_t st);
cudaError_t launch_head_dh_join(const HeadChunkParams& p, bool bf16, int sm_count, cudaStream_t st);
cudaError_t launch_loss(const LossParams& l, const int* counts, cudaStream_t st);
cudaError_t launch_few_prep(const FewParams& p, const uint16_t* h, const uint16_t* W, bool bf16, double* zt, cudaStream_t st);
cudaError_t launch_few(const FewParams& p, const CUtensorMap& mH, const CUtensorMap& mW, int grid, bool bf16, int nc,
                       cudaStream_t st);

}  // namespace grpo
