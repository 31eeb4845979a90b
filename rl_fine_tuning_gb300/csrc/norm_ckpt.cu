// 8-bit checkpoints of activations: packing and unpacking (norm_abi.cu has the entry
// points; the norm's kernels write and read them too).
//
// Per element 2 bytes on one side and 1 + 1/32 on the other, and nothing but HBM to
// bound them: 655M elements take 275 us to pack (7.2 TB/s) and 281 to unpack (7.1),
// where a copy reaches 6.8.  A block works on 8192 elements, 16 a thread at a time, and ends.
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

// at most 2^30: see kMostElements
int64_t ckpt_blocks(const CkptParams& p) {
    const int64_t each = kCkptThreads * kCkptUpt;
    return (p.N * (p.d / kUnit) + each - 1) / each;
}

}  // namespace

cudaError_t launch_ckpt_pack(const CkptParams& p, bool bf16, cudaStream_t st) {
    return launch_chained(bf16 ? k_ckpt_pack<true> : k_ckpt_pack<false>, ckpt_blocks(p), kCkptThreads, 0, p, st);
}

cudaError_t launch_ckpt_unpack(const CkptParams& p, bool bf16, cudaStream_t st) {
    return launch_chained(bf16 ? k_ckpt_unpack<true> : k_ckpt_unpack<false>, ckpt_blocks(p), kCkptThreads, 0, p, st);
}

}  // namespace grpo
