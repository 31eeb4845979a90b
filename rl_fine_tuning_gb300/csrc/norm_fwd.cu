// The norm before the head: forward pass (norm_abi.cu has the entry point, norm_plan.cu
// deals the rows).
//   s = x + residual, or a checkpoint's values;  y = s / sqrt(mean s^2 + eps) w
// 5 operations an element against 3 to 8 bytes: HBM bounds it.  A row is read
// once and stays in registers, 16-bit values in pairs, between its sum of squares
// and its outputs (s, its checkpoint, y), and while it is worked on, the next row's
// loads are under way.  A thread has 16 elements of a row, a whole sector to load and to store, or twice
// that in the widest rows.  Rows that do not count cost the stores of their zeros.
// Measured: 160,000 x 4096 with the residual, 54% of the rows: 579 us, 7.0 TB/s (a copy reaches 6.8);
// 10,000 x 4096 to E4M3 and a checkpoint: 39 us, 6.3 TB/s.  Copies of the rows to come
// into shared memory by each thread for itself (cp.async) were slower: 764 us against 626 at the time.
#include "norm_device.cuh"

namespace grpo {

namespace {

// of a thread with one or two units: 1024 or 512 threads an SM; 8-bit y of a sum in rows of a warp spills 8 bytes a thread
constexpr int kFwdRegs = 64, kFwdRegsTwo = 128;

template <bool kMax>
__device__ __forceinline__ float both(float a, float b) { return kMax ? fmaxf(a, b) : a + b; }

// Sum (or maximum) over a row's threads, in a fixed order; every thread gets it.
// A block's: the warps' values lie in s, of which the next call takes another
// part, so that one barrier is enough; entries of warps that are not there hold 0.
template <bool kWide, bool kMax>
__device__ __forceinline__ float row_join(float v, int width, float* s) {
    for (int o = kWide ? 16 : width / 2; o > 0; o >>= 1) v = both<kMax>(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (!kWide) return v;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (unsigned i = 0; i < blockDim.x; i += 128) {
        const float4 x = *reinterpret_cast<const float4*>(s + i / 32);
        v = both<kMax>(v, both<kMax>(both<kMax>(x.x, x.y), both<kMax>(x.z, x.w)));
    }
    return v;
}

// kUpt units a thread.  kWide: a block takes one row at a time; else 4 to 32 lanes of its warps take one each.
template <bool kBf16, int kSrc, int kUpt, bool kWide, bool kOut8>
__global__ void __maxnreg__(kUpt == 1 ? kFwdRegs : kFwdRegsTwo) k_norm_fwd(const NormParams p) {
    __shared__ alignas(16) float s_join[4][kBlockMax / 32];
    extern __shared__ float4 s_weight[];
    const int n_unit = p.d / kUnit;
    const int width = kWide ? static_cast<int>(blockDim.x) : p.width;
    const int pad = width * kUpt;
    const int lane = kWide ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) & (width - 1);
    const int rows = kWide ? 1 : kWarpThreads / width;            // rows that a block works on at once
    const uint32_t step = gridDim.x * rows, first = blockIdx.x * rows, N = static_cast<uint32_t>(p.N);   // N < 2^31
    const uint32_t mine = kWide ? 0 : threadIdx.x / width;
    const bool want_scale = kOut8 && (p.row_scale || p.y_inv == 0.f);
    const float inv_d = 1.f / p.d;
    const float inv_largest = p.y_type == GRPO_E4M3 ? 1.f / 448 : 1.f / 57344;
    chain_next();
    chain_wait();
    Raw<kSrc, kUpt> raw = {};
    uint32_t t = first + mine;
    int64_t at = static_cast<int64_t>(t) * p.d + lane * kUnit;         // the thread's first element of row t
    const int64_t at_step = static_cast<int64_t>(step) * p.d;
    Ahead ahead;
    ahead.begin(p, t, step, kWide ? 32 : width);
    uint32_t alive = ahead.bits(kWide ? 32 : width);       // bit q: row t + q step counts
    load_row<kSrc, kUpt, kWide>(p, at, alive & 1, lane, width, n_unit, &raw);
    stage_weight<kBf16>(p, s_weight, pad);
    for (unsigned i = threadIdx.x; i < 4 * kBlockMax / 32; i += blockDim.x) s_join[0][i] = 0.f;
    __syncthreads();
    int turn = 0;
    for (uint32_t base = first; base < N; base += step, t += step, at += at_step) {   // whole blocks go round together
        const bool live = alive & 1, next = alive >> 1 & 1, here = t < N;
        ahead.advance(p, t, step, kWide ? 32 : width);
        alive = ahead.bits(kWide ? 32 : width);
        Unit s[kUpt];
#pragma unroll
        for (int k = 0; k < kUpt; ++k) s[k] = stream_of<kBf16>(raw, k);
        load_row<kSrc, kUpt, kWide>(p, at + at_step, next, lane, width, n_unit, &raw);
        if (kWide && !live) {                 // the whole block's row
#pragma unroll
            for (int k = 0; k < kUpt; ++k) {
                const int i = lane + k * width;
                if (i >= n_unit) break;
                if (kOut8)
                    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + at + k * width * kUnit) = make_uint4(0, 0, 0, 0);
                else
                    store_unit(static_cast<uint16_t*>(p.y) + at + k * width * kUnit, Unit{});
                if (p.sum) store_unit(p.sum + at + k * width * kUnit, Unit{});
                if (p.codes_out) {
                    *reinterpret_cast<uint4*>(p.codes_out + at + k * width * kUnit) = make_uint4(0, 0, 0, 0);
                    if ((i & 3) == 0) p.scales_out[(at + k * width * kUnit) / kCkptBlock] = bf16_bits(kLeastScale);
                }
            }
            if (p.row_scale && lane == 0) p.row_scale[t] = kLeastScale;
            continue;
        }
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kUpt; ++k) {
            const Unit32 v = values<kBf16>(s[k]);
            F2 sq = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sq = f2_fma(v.p[i], v.p[i], sq);
            if (!kWide || lane + k * width < n_unit) sum += sum_of(sq);
        }
        if (p.sum) {
#pragma unroll
            for (int k = 0; k < kUpt; ++k)
                if (here && lane + k * width < n_unit) store_unit(p.sum + at + k * width * kUnit, s[k]);
        }
        if (p.codes_out) {
#pragma unroll
            for (int k = 0; k < kUpt; ++k) {
                const int i = lane + k * width;
                uint16_t scale;
                const uint4 c = encode<kBf16>(s[k], &scale);
                if (here && i < n_unit) {
                    *reinterpret_cast<uint4*>(p.codes_out + at + k * width * kUnit) = c;
                    if ((i & 3) == 0) p.scales_out[(at + k * width * kUnit) / kCkptBlock] = scale;
                }
            }
        }
        const float sq = row_join<kWide, false>(sum, width, s_join[turn]);
        const float rstd = rsqrtf(sq * inv_d + p.eps);
        const F2 rstd2 = f2(rstd, rstd);
        Unit32 y[kUpt];
#pragma unroll
        for (int k = 0; k < kUpt; ++k) {
            const Unit32 w = staged_weight(s_weight, pad, lane + k * width);
            y[k] = values<kBf16>(s[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[k].p[i] = f2_mul(f2_mul(y[k].p[i], rstd2), w.p[i]);
        }
        if (!kOut8) {
#pragma unroll
            for (int k = 0; k < kUpt; ++k) {
                const int i = lane + k * width;
                Unit u = rounded<kBf16>(y[k]);
                if (!kWide && !live) u = Unit{};            // not 0 times a weight that is not finite
                if (here && i < n_unit) store_unit(static_cast<uint16_t*>(p.y) + at + k * width * kUnit, u);
            }
        } else {
            float inv = p.y_inv;
            if (want_scale) {
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < kUpt; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = f2_values(y[k].p[i]);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                top = row_join<kWide, true>(kWide || live ? top : 0.f, width, s_join[2 + turn]);
                const float scale = fmaxf(__fmul_rn(top, inv_largest), kLeastScale);
                if (p.row_scale && here && lane == 0) p.row_scale[t] = scale;
                if (inv == 0.f) inv = __frcp_rn(scale);
            }
            const F2 inv2 = f2(inv, inv);
#pragma unroll
            for (int k = 0; k < kUpt; ++k) {
                const int i = lane + k * width;
#pragma unroll
                for (int j = 0; j < 8; ++j) y[k].p[j] = f2_mul(y[k].p[j], inv2);
                uint4 c = p.y_type == GRPO_E5M2 ? codes8<true>(y[k]) : codes8<false>(y[k]);
                if (!kWide && !live) c = make_uint4(0, 0, 0, 0);
                if (here && i < n_unit) *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + at + k * width * kUnit) = c;
            }
        }
        turn ^= 1;
    }
}

template <bool kBf16, int kSrc, bool kOut8>
cudaError_t fwd_of(const NormParams& p, const NormPlan& o, cudaStream_t st) {
    auto f = o.wide ? o.upt == 1 ? k_norm_fwd<kBf16, kSrc, 1, true, kOut8> : k_norm_fwd<kBf16, kSrc, 2, true, kOut8>
                    : o.upt == 1 ? k_norm_fwd<kBf16, kSrc, 1, false, kOut8> : k_norm_fwd<kBf16, kSrc, 2, false, kOut8>;
    const size_t smem = static_cast<size_t>(o.width) * o.upt * kUnit * 4;
    if (smem > 40 * 1024) {                    // only the widest rows, two units a thread; 48 KB need no permission
        static MostSmem most;
        const cudaError_t e = most.allow(f, kNormMaxD * 4);
        if (e != cudaSuccess) return e;
    }
    return launch_chained(f, o.grid, o.threads, smem, p, st);
}

template <bool kBf16, int kSrc>
cudaError_t fwd_as(const NormParams& p, const NormPlan& o, cudaStream_t st) {
    const bool out8 = p.y_type == GRPO_E4M3 || p.y_type == GRPO_E5M2;
    return out8 ? fwd_of<kBf16, kSrc, true>(p, o, st) : fwd_of<kBf16, kSrc, false>(p, o, st);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormParams& p, const NormPlan& o, bool bf16, cudaStream_t st) {
    if (p.codes) return bf16 ? fwd_as<true, kCkpt>(p, o, st) : fwd_as<false, kCkpt>(p, o, st);
    if (p.residual) return bf16 ? fwd_as<true, kXResidual>(p, o, st) : fwd_as<false, kXResidual>(p, o, st);
    return bf16 ? fwd_as<true, kX>(p, o, st) : fwd_as<false, kX>(p, o, st);
}

}  // namespace grpo
