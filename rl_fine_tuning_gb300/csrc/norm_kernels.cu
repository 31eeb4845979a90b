// The norm before the head, its gradient, and 8-bit checkpoints of activations.
//
// All of them move bytes: a handful of operations per element against 3 to 8
// bytes, so HBM bounds them.  A row is read once; what is needed of it twice
// (after its sum of squares is known) stays on chip.
#include <cfloat>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "norm.h"

namespace grpo {

namespace {

constexpr int kThreads = 256;
constexpr int kV = 8;                  // elements of a thread's load: 16 bytes of a 16-bit matrix

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

template <bool kBf16>
__device__ __forceinline__ float value16(uint16_t bits) {
    return kBf16 ? bf16_value(bits) : __half2float(__ushort_as_half(bits));
}
template <bool kBf16>
__device__ __forceinline__ uint16_t bits16(float v) {
    return kBf16 ? bf16_bits(v) : __half_as_ushort(__float2half_rn(v));
}

// the largest finite scale of a checkpoint: 2^121 (bf16), 2^9 (fp16)
template <bool kBf16>
constexpr float kMostScale = kBf16 ? 2.658455992e36f : 512.f;

struct alignas(16) Vec {
    uint16_t v[kV];
};

template <bool kBf16>
__device__ __forceinline__ void load8(const uint16_t* a, float (&v)[kV]) {
    const Vec x = *reinterpret_cast<const Vec*>(a);
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = value16<kBf16>(x.v[i]);
}

template <bool kBf16>
__device__ __forceinline__ void store8(uint16_t* a, const float (&v)[kV]) {
    Vec x;
#pragma unroll
    for (int i = 0; i < kV; ++i) x.v[i] = bits16<kBf16>(v[i]);
    *reinterpret_cast<Vec*>(a) = x;
}

// 8 values of s = rounded x + residual, or of a checkpoint, at element `at`
template <bool kBf16>
__device__ __forceinline__ void load_stream(const NormParams& p, int64_t at, float (&v)[kV]) {
    if (p.codes) {
        const float scale = bf16_value(p.scales[at / kCkptBlock]);
        const uint2 c = *reinterpret_cast<const uint2*>(p.codes + at);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int8_t code = static_cast<int8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
            v[i] = value16<kBf16>(bits16<kBf16>(static_cast<float>(code) * scale));
        }
        return;
    }
    load8<kBf16>(p.x + at, v);
    if (p.residual) {
        float r[kV];
        load8<kBf16>(p.residual + at, r);
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = value16<kBf16>(bits16<kBf16>(v[i] + r[i]));
    }
}

__device__ __forceinline__ void load_weight(const NormParams& p, bool bf16, int j, float (&w)[kV]) {
    if (p.weight_f32) {
        const float4* a = reinterpret_cast<const float4*>(static_cast<const float*>(p.weight) + j);
        const float4 b = a[0], c = a[1];
        w[0] = b.x, w[1] = b.y, w[2] = b.z, w[3] = b.w, w[4] = c.x, w[5] = c.y, w[6] = c.z, w[7] = c.w;
    } else if (bf16) {
        load8<true>(static_cast<const uint16_t*>(p.weight) + j, w);
    } else {
        load8<false>(static_cast<const uint16_t*>(p.weight) + j, w);
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) w[i] += p.plus;
}

// One scale per kCkptBlock columns, which 8 neighbouring lanes hold: max |x| / 127
// in bf16, at least 2^-126.  Values are compared as bit patterns, so that a NaN
// is the largest and makes its whole block NaN.  A scale rounded down puts the
// largest value at up to 127.5 steps: it still is within half a step of code 127.
// Scales end where 127 of them still are finite in the 16-bit type; of a block
// beyond that, the values near the type's largest take code 127 too.
template <bool kBf16>
__device__ __forceinline__ void encode8(const float (&v)[kV], int8_t* codes, uint16_t* scale_out) {
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffu << (threadIdx.x & 24), top, o, 8));
    float s = __fmul_rn(__uint_as_float(top), 1.f / 127);
    s = s < kLeastScale ? kLeastScale : s;
    if (s > kMostScale<kBf16> && s <= FLT_MAX) s = kMostScale<kBf16>;
    const uint16_t bits = bf16_bits(s);
    const float inv = __fdiv_rn(1.f, bf16_value(bits));
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int q = max(-127, min(127, __float2int_rn(__fmul_rn(v[i], inv))));
        c[i / 4] |= static_cast<uint32_t>(q & 255) << (8 * (i & 3));
    }
    *reinterpret_cast<uint2*>(codes) = make_uint2(c[0], c[1]);
    if ((threadIdx.x & 7) == 0) *scale_out = bits;
}

__device__ __forceinline__ uint2 codes8(const float (&v)[kV], bool e5m2) {
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __nv_fp8_interpretation_t t = e5m2 ? __NV_E5M2 : __NV_E4M3;
        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, t);
        const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, t);
        c[i] = a | b << 16;
    }
    return make_uint2(c[0], c[1]);
}

// Sum and maximum over the block, in a fixed order; every thread gets them.
__device__ __forceinline__ float block_sum(float v, float* s) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) v += s[i];
    return v;
}

__device__ __forceinline__ float block_max(float v, float* s) {
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) v = fmaxf(v, s[i]);
    return v;
}

__device__ __forceinline__ float row_largest(int y_type) { return y_type == GRPO_E4M3 ? 448.f : 57344.f; }

// ---------------------------------------------------------------- forward

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) k_norm_fwd(const NormParams p) {
    extern __shared__ Vec row[];
    __shared__ float s_red[kThreads / 32];
    const int n_vec = p.d / kV;
    const bool y16 = p.y_type == GRPO_BF16 || p.y_type == GRPO_FP16;
    for (int64_t t = blockIdx.x; t < p.N; t += gridDim.x) {
        const bool counts = !p.mask || p.mask[t];
        float sq = 0.f;
        for (int i = threadIdx.x; i < n_vec; i += kThreads) {
            float v[kV] = {};
            const int64_t at = t * p.d + i * kV;
            if (counts) load_stream<kBf16>(p, at, v);
#pragma unroll
            for (int k = 0; k < kV; ++k) sq += v[k] * v[k];
            if (p.sum) store8<kBf16>(p.sum + at, v);
            if (p.codes_out) encode8<kBf16>(v, p.codes_out + at, p.scales_out + at / kCkptBlock);
            store8<kBf16>(row[i].v, v);
        }
        const float rstd = 1.f / sqrtf(block_sum(sq, s_red) / p.d + p.eps);
        auto normed = [&](int i, float (&v)[kV]) {
            float w[kV];
            load8<kBf16>(row[i].v, v);
            load_weight(p, kBf16, i * kV, w);
#pragma unroll
            for (int k = 0; k < kV; ++k) v[k] = v[k] * rstd * w[k];
        };
        float inv = p.y_inv;
        if (!y16 && (p.row_scale || inv == 0.f)) {
            float top = 0.f;
            for (int i = threadIdx.x; i < n_vec; i += kThreads) {
                float v[kV];
                normed(i, v);
#pragma unroll
                for (int k = 0; k < kV; ++k) top = fmaxf(top, fabsf(v[k]));
            }
            const float scale = fmaxf(__fmul_rn(block_max(top, s_red), 1.f / row_largest(p.y_type)), kLeastScale);
            if (threadIdx.x == 0) p.row_scale[t] = counts ? scale : kLeastScale;
            if (inv == 0.f) inv = __fdiv_rn(1.f, scale);
        }
        for (int i = threadIdx.x; i < n_vec; i += kThreads) {
            float v[kV];
            normed(i, v);
            if (!counts)
                for (int k = 0; k < kV; ++k) v[k] = 0.f;
            const int64_t at = t * p.d + i * kV;
            if (y16) {
                store8<kBf16>(static_cast<uint16_t*>(p.y) + at, v);
            } else {
#pragma unroll
                for (int k = 0; k < kV; ++k) v[k] *= inv;
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + at) = codes8(v, p.y_type == GRPO_E5M2);
            }
        }
    }
}

// ---------------------------------------------------------------- gradient

// dx = rstd (g - s rstd^2 mean(g s)) + dsum with g = dy w.  Block b takes rows
// b, b + gridDim.x, ... and leaves its sum of dy s rstd, for every column, in part[b].
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) k_norm_bwd(const NormParams p) {
    extern __shared__ Vec row[];
    __shared__ float s_red[kThreads / 32];
    const int n_vec = p.d / kV;
    Vec* row_dy = row + n_vec;
    float* acc = reinterpret_cast<float*>(row_dy + n_vec);
    for (int j = threadIdx.x; j < p.d; j += kThreads) acc[j] = 0.f;
    __syncthreads();
    bool bad = false;
    for (int64_t t = blockIdx.x; t < p.N; t += gridDim.x) {
        if (p.mask && !p.mask[t]) {
            const float zero[kV] = {};
            for (int i = threadIdx.x; i < n_vec; i += kThreads) store8<kBf16>(p.dx + t * p.d + i * kV, zero);
            continue;
        }
        float sq = 0.f, gs = 0.f;
        for (int i = threadIdx.x; i < n_vec; i += kThreads) {
            float v[kV], dy[kV], w[kV];
            const int64_t at = t * p.d + i * kV;
            load_stream<kBf16>(p, at, v);
            load8<kBf16>(p.dy + at, dy);
            load_weight(p, kBf16, i * kV, w);
#pragma unroll
            for (int k = 0; k < kV; ++k) {
                sq += v[k] * v[k];
                gs += v[k] * (dy[k] * w[k]);
            }
            store8<kBf16>(row[i].v, v);
            store8<kBf16>(row_dy[i].v, dy);
        }
        sq = block_sum(sq, s_red);
        gs = block_sum(gs, s_red);
        const float rstd = 1.f / sqrtf(sq / p.d + p.eps);
        const float c = rstd * rstd * (gs / p.d);
        for (int i = threadIdx.x; i < n_vec; i += kThreads) {
            float v[kV], dy[kV], w[kV], more[kV] = {};
            const int64_t at = t * p.d + i * kV;
            load8<kBf16>(row[i].v, v);
            load8<kBf16>(row_dy[i].v, dy);
            load_weight(p, kBf16, i * kV, w);
            if (p.dsum) load8<kBf16>(p.dsum + at, more);
#pragma unroll
            for (int k = 0; k < kV; ++k) {
                acc[i * kV + k] += dy[k] * (v[k] * rstd);
                v[k] = rstd * (dy[k] * w[k] - v[k] * c) + more[k];
                v[k] = value16<kBf16>(bits16<kBf16>(v[k]));
                bad |= !(fabsf(v[k]) <= FLT_MAX);
            }
            store8<kBf16>(p.dx + at, v);
        }
    }
    if (p.dweight)
        for (int i = threadIdx.x; i < n_vec; i += kThreads)
            for (int k = 0; k < kV; ++k) p.part[static_cast<int64_t>(blockIdx.x) * p.d + i * kV + k] = acc[i * kV + k];
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) p.bad[blockIdx.x] = any;
}

// dw and found_inf from the parts, in the order of the parts; one block
template <bool kBf16>
__global__ void __launch_bounds__(1024) k_norm_join(const NormParams p) {
    bool bad = false;
    for (int b = threadIdx.x; b < p.parts; b += blockDim.x) bad |= p.bad[b] != 0;
    if (p.dweight)
        for (int j = threadIdx.x; j < p.d; j += blockDim.x) {
            float v = 0.f;
            for (int b = 0; b < p.parts; ++b) v += p.part[static_cast<int64_t>(b) * p.d + j];
            if (p.weight_f32) {
                static_cast<float*>(p.dweight)[j] = v;
            } else {
                const uint16_t r = bits16<kBf16>(v);
                static_cast<uint16_t*>(p.dweight)[j] = r;
                v = value16<kBf16>(r);
            }
            bad |= !(fabsf(v) <= FLT_MAX);
        }
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.found_inf = any ? 1 : 0;
}

// ---------------------------------------------------------------- checkpoints

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) k_ckpt_pack(const CkptParams p) {
    const int64_t n = p.N * (p.d / kV);    // a multiple of 8: the 8 lanes of a block of columns go together
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        float v[kV] = {};
        if (!p.mask || p.mask[i * kV / p.d]) load8<kBf16>(p.x + i * kV, v);
        encode8<kBf16>(v, p.codes_out + i * kV, p.scales_out + i * kV / kCkptBlock);
    }
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) k_ckpt_unpack(const CkptParams p) {
    const int64_t n = p.N * (p.d / kV);
    NormParams q = {};
    q.codes = p.codes;
    q.scales = p.scales;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        float v[kV] = {};
        if (!p.mask || p.mask[i * kV / p.d]) load_stream<kBf16>(q, i * kV, v);
        store8<kBf16>(p.x_out + i * kV, v);
    }
}

int stream_blocks(const CkptParams& p, int sm_count) {
    const int64_t want = (p.N * (p.d / kV) + kThreads - 1) / kThreads, most = 8LL * sm_count;
    return static_cast<int>(want < most ? want : most);
}

}  // namespace

int norm_parts(int64_t N, int d, int sm_count) {
    (void)d;
    int most = sm_count < kNormParts ? sm_count : kNormParts;
    return static_cast<int>(N < most ? N : most);
}

cudaError_t launch_norm_fwd(const NormParams& p, bool bf16, int sm_count, cudaStream_t st) {
    const int64_t most = 4LL * sm_count;
    const int grid = static_cast<int>(p.N < most ? p.N : most);
    if (bf16)
        k_norm_fwd<true><<<grid, kThreads, p.d * 2, st>>>(p);
    else
        k_norm_fwd<false><<<grid, kThreads, p.d * 2, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormParams& p, bool bf16, int sm_count, cudaStream_t st) {
    (void)sm_count;
    const auto f = bf16 ? k_norm_bwd<true> : k_norm_bwd<false>;
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxD * 8);
    if (e != cudaSuccess) return e;
    f<<<p.parts, kThreads, p.d * 8, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_norm_join(const NormParams& p, bool bf16, cudaStream_t st) {
    if (bf16)
        k_norm_join<true><<<1, 1024, 0, st>>>(p);
    else
        k_norm_join<false><<<1, 1024, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_ckpt_pack(const CkptParams& p, bool bf16, int sm_count, cudaStream_t st) {
    const int grid = stream_blocks(p, sm_count);
    if (bf16)
        k_ckpt_pack<true><<<grid, kThreads, 0, st>>>(p);
    else
        k_ckpt_pack<false><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_ckpt_unpack(const CkptParams& p, bool bf16, int sm_count, cudaStream_t st) {
    const int grid = stream_blocks(p, sm_count);
    if (bf16)
        k_ckpt_unpack<true><<<grid, kThreads, 0, st>>>(p);
    else
        k_ckpt_unpack<false><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace grpo
