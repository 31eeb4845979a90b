// The join of a row's partial sums, used by the merge and by the few-row kernel.
#pragma once
#include "head.h"

namespace grpo {

// A row's partials (m, s, u) joined with its given token, whose column the
// logits kernels left out.  With M = max m and everything relative to 2^M,
//   lse = ln 2 (M + log2 s),   q = z_tok - lse,   H = -sum p log p = lse - u / s.
// The last additions are in fp64: q is a difference of two numbers of about 10.
struct RowSum {
    double lse, q;
    float ent;
};

__device__ __forceinline__ RowSum join_row(const float4* part, int S2, int lane, double zt) {
    constexpr double kLog2eD = 1.4426950408889634074, kLn2D = 0.69314718055994530942;
    float m = kNoLogit2;
    for (int k = lane; k < S2; k += 32) m = fmaxf(m, __ldcg(part + k).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = fmaxf(m, static_cast<float>(zt * kLog2eD));
    float s = 0.f, u = 0.f;
    for (int k = lane; k < S2; k += 32) {
        const float4 ps = __ldcg(part + k);
        const float f = exp2f(ps.x - m);   // 0 for a part that held the token's column alone
        s = fmaf(ps.y, f, s);
        u = fmaf(ps.z, f, u);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        u += __shfl_xor_sync(0xffffffffu, u, o);
    }
    const double et = exp2(zt * kLog2eD - static_cast<double>(m));
    const double sd = static_cast<double>(s) + et;
    RowSum r;
    r.lse = (static_cast<double>(m) + log2(sd)) * kLn2D;
    r.q = zt - r.lse;
    const float ent = static_cast<float>(r.lse - (static_cast<double>(u) + et * zt) / sd);
    r.ent = ent < 0.f ? 0.f : ent;
    return r;
}

// The same from sums relative to the given token's logit, part.x the fp32 value
// of z_tok log2 e that was the base: s = sum e^(z - z_tok) over the other
// columns, q = -log(1 + s).  s overflows when another logit is far above the
// token's; q is then -inf and the caller takes another way.
__device__ __forceinline__ RowSum join_row_relative(const float4* part, int S2, int lane, double zt) {
    float s = 0.f;
    for (int k = lane; k < S2; k += 32) s += __ldcg(part + k).y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const double base = static_cast<double>(__ldcg(part).x);
    RowSum r;
    r.q = -log1p(static_cast<double>(s) * exp2(base - zt * 1.4426950408889634074));
    r.lse = zt - r.q;
    r.ent = 0.f;
    return r;
}

}  // namespace grpo
