// 8-bit checkpoints of activations (see norm_abi.cu for the entry points), and
// how the norm's rows are dealt to threads.
#include "norm_device.cuh"

namespace grpo {

namespace {

constexpr int kCkptThreads = 256;
constexpr int kCkptUpt = 2;            // units of a thread at once

// The row of unit i, i / (d / 16), is a product with ceil(2^64 / (d / 16)): exact while i * (d / 16) < 2^64.
__device__ __forceinline__ bool unit_counts(const CkptParams& p, int64_t i) {
    return !p.mask || p.mask[__umul64hi(static_cast<uint64_t>(i), p.per_row)];
}

template <bool kBf16>
__global__ void __launch_bounds__(kCkptThreads) k_ckpt_pack(const CkptParams p) {
    const int64_t n = p.N * (p.d / kUnit);     // a multiple of 4: the 4 lanes of a block of columns go together
    const int64_t i0 = blockIdx.x * static_cast<int64_t>(kCkptThreads * kCkptUpt) + threadIdx.x;
    chain_next();
    chain_wait();
    Unit x[kCkptUpt];
#pragma unroll
    for (int k = 0; k < kCkptUpt; ++k) {
        const int64_t i = i0 + k * kCkptThreads;
        x[k] = load_unit(p.x + i * kUnit, i < n && unit_counts(p, i));
    }
#pragma unroll
    for (int k = 0; k < kCkptUpt; ++k) {
        const int64_t i = i0 + k * kCkptThreads;
        uint16_t scale;
        const uint4 c = encode<kBf16>(x[k], &scale);
        if (i < n) {
            *reinterpret_cast<uint4*>(p.codes_out + i * kUnit) = c;
            if ((i & 3) == 0) p.scales_out[i / (kCkptBlock / kUnit)] = scale;
        }
    }
}

template <bool kBf16>
__global__ void __launch_bounds__(kCkptThreads) k_ckpt_unpack(const CkptParams p) {
    const int64_t n = p.N * (p.d / kUnit);
    const int64_t i0 = blockIdx.x * static_cast<int64_t>(kCkptThreads * kCkptUpt) + threadIdx.x;
    chain_next();
    chain_wait();
    uint4 c[kCkptUpt];
    uint32_t scale[kCkptUpt];
#pragma unroll
    for (int k = 0; k < kCkptUpt; ++k) {
        const int64_t i = i0 + k * kCkptThreads;
        const bool on = i < n && unit_counts(p, i);
        c[k] = load_codes(p.codes + i * kUnit, on);
        scale[k] = load_scale(p.scales + i / (kCkptBlock / kUnit), on);
    }
#pragma unroll
    for (int k = 0; k < kCkptUpt; ++k) {
        const int64_t i = i0 + k * kCkptThreads;
        if (i < n) store_unit(p.x_out + i * kUnit, decode<kBf16>(c[k], bf16_value(scale[k])));
    }
}

// a block for each 8192 elements: at most 2^31 blocks for 2^31 rows of 8192 columns; the caller refuses more
int64_t ckpt_blocks(const CkptParams& p) {
    const int64_t each = kCkptThreads * kCkptUpt;
    return (p.N * (p.d / kUnit) + each - 1) / each;
}

}  // namespace

namespace {

// the row's threads, and their units
NormPlan row_plan(int d, bool two) {
    NormPlan o;
    const int n_unit = d / kUnit;
    o.wide = n_unit > 64;
    if (!o.wide) {
        o.width = n_unit <= 8 ? 4 : n_unit <= 32 ? 16 : 32;
        o.upt = (n_unit + o.width - 1) / o.width;
        o.threads = kWarpThreads;
    } else {
        o.upt = n_unit > kBlockMax || two ? 2 : 1;
        o.threads = o.width = (n_unit + 32 * o.upt - 1) / (32 * o.upt) * 32;
    }
    return o;
}

}  // namespace

NormPlan norm_fwd_plan(int64_t N, int d, int sm_count) {
    NormPlan o = row_plan(d, false);
    const int64_t rows = o.threads / o.width, turns = (N + rows - 1) / rows;
    o.per_sm = (o.upt == 1 ? 1024 : 512) / o.threads;
    const int64_t once = static_cast<int64_t>(o.per_sm) * sm_count, waves = turns / 8 / once;
    o.grid = static_cast<int>(turns < once ? turns : waves > 1 ? waves * once : once);
    return o;
}

NormPlan norm_bwd_plan(int64_t N, int d, int sm_count, bool ckpt, bool dsum) {
    const bool two = ckpt && !dsum && N >= 64LL * sm_count;
    NormPlan o = row_plan(d, two);
    const int64_t rows = o.threads / o.width, turns = (N + rows - 1) / rows;
    const int resident = !o.wide ? 512 : o.upt == 2 ? 384 : dsum ? 512 : 768;
    o.per_sm = resident < o.threads ? 1 : resident / o.threads;
    const int64_t most = static_cast<int64_t>(o.per_sm) * sm_count;
    o.grid = static_cast<int>(turns < most ? turns : most);
    return o;
}

cudaError_t launch_ckpt_pack(const CkptParams& p, bool bf16, cudaStream_t st) {
    return launch_chained(bf16 ? k_ckpt_pack<true> : k_ckpt_pack<false>, ckpt_blocks(p), kCkptThreads, 0, p, st);
}

cudaError_t launch_ckpt_unpack(const CkptParams& p, bool bf16, cudaStream_t st) {
    return launch_chained(bf16 ? k_ckpt_unpack<true> : k_ckpt_unpack<false>, ckpt_blocks(p), kCkptThreads, 0, p, st);
}

}  // namespace grpo
