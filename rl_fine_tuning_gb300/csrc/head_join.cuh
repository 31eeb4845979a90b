// The join of a row's partial sums, used by the merge and by the few-row kernel.
#pragma once
#include "head.h"

namespace grpo {

// A row's partials (m, s, u) joined with its given token, whose column the
// logits kernels left out.  With M = max m, everything relative to 2^M, and
// x = s 2^M / e^z_tok (the other tokens' weight against the given one's),
//   q = -log(1 + x),   lse = z_tok - q,   H = -sum p log p = lse - E[z].
// log1p keeps q's relative precision however near the token's probability is
// to 1.  The differences of numbers of about 10 are in fp64, the functions in
// fp32 (fp64 ones cost microseconds).  lse2, for the dlogits: lse in base 2 as
// M + log2(s + e^z_tok / 2^M), two numbers: rounded to one it would be 4 off for
// logits of 1e7, and a probability of 1 would be 8.
struct RowSum {
    double lse, q;
    float ent;
    float2 lse2;
};

__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

__device__ __forceinline__ RowSum finish_row(float m, float s, float u, double zt) {
    constexpr double kLog2eD = 1.4426950408889634074, kLn2D = 0.69314718055994530942;
    RowSum r;
    float mean;   // E[z]
    const double dm = static_cast<double>(m) - zt * kLog2eD;
    if (dm < 80.0) {
        const float f = exp2f(static_cast<float>(dm));   // 0 when there is no other token: m is about -2^100
        const float x = s * f;
        r.q = -static_cast<double>(log1pf(x));
        r.lse = zt - r.q;
        const float up = -static_cast<float>(dm);
        r.lse2 = make_float2(m, up > 100.f ? up : log2f(s + exp2f(up)));   // s is below 2^50
        mean = (fmaf(u, f, static_cast<float>(zt))) / (1.f + x);
    } else {   // p below 2^-80: the given token adds nothing
        int ex;
        const float mant = frexpf(s, &ex);
        r.lse = (static_cast<double>(m) + ex + static_cast<double>(log2f(mant))) * kLn2D;
        r.lse2 = make_float2(m, log2f(s));
        r.q = zt - r.lse;
        mean = u / s;
    }
    const float ent = static_cast<float>(r.lse - static_cast<double>(mean));
    r.ent = ent < 0.f ? 0.f : ent;
    return r;
}

__device__ __forceinline__ RowSum join_row(const float4* part, int S2, int lane, double zt) {
    float m = kNoLogit2;
    for (int k = lane; k < S2; k += 32) m = fmaxf(m, __ldcg(part + k).x);
    m = warp_max(m);
    float s = 0.f, u = 0.f;
    for (int k = lane; k < S2; k += 32) {
        const float4 ps = __ldcg(part + k);
        const float f = exp2f(ps.x - m);
        s = fmaf(ps.y, f, s);
        u = fmaf(ps.z, f, u);
    }
    return finish_row(m, warp_sum(s), warp_sum(u), zt);
}

// The same for at most 32 kPer partials, read once: all loads in flight together
template <int kPer>
__device__ __forceinline__ RowSum join_row_once(const float4* part, int S2, int lane, double zt) {
    float4 v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        v[j] = lane + 32 * j < S2 ? __ldcg(part + lane + 32 * j) : make_float4(kNoLogit2, 0.f, 0.f, 0.f);
    float m = kNoLogit2;
#pragma unroll
    for (int j = 0; j < kPer; ++j) m = fmaxf(m, v[j].x);
    m = warp_max(m);
    float s = 0.f, u = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const float f = exp2f(v[j].x - m);
        s = fmaf(v[j].y, f, s);
        u = fmaf(v[j].z, f, u);
    }
    return finish_row(m, warp_sum(s), warp_sum(u), zt);
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
    r.q = -static_cast<double>(log1pf(s * exp2f(static_cast<float>(base - zt * 1.4426950408889634074))));
    r.lse = zt - r.q;
    r.ent = 0.f;
    r.lse2 = make_float2(0.f, 0.f);   // not used: the dlogits are relative to the token
    return r;
}

// The loss from the rows' (or pairs') weighted objectives, by one warp: fp64 sums in
// a fixed order.
__device__ __forceinline__ void write_loss(const LossParams& l, const int* counts, int lane) {
    if (!l.loss) return;
    double acc = 0.0;
    if (l.pair_ell) {
        for (int i = lane; i < l.n_pairs; i += 32) acc += __ldcg(l.pair_ell + i);
    } else {
        const int nv = counts[C_NVALID];
#pragma unroll 8
        for (int i = lane; i < nv; i += 32) acc += static_cast<double>(__ldcg(l.ell + i));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) {
        const int n = l.pair_ell ? counts[C_NACT] : 1;   // rows carry their weight in the mean already
        *l.loss = n > 0 ? static_cast<float>(acc / n) : 0.f;
    }
}

}  // namespace grpo
