// The steps of the head operators that are not GEMMs: the plan (valid rows,
// completion offsets, chunk bounds), the gather with the given token's logit,
// the per-row merge with the operators' d loss / d q, the preference loss over
// pairs, the dlogits pass, the join of split dH tiles, and the loss sums.
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "head_join.cuh"
#include "ptx.cuh"

namespace grpo {

namespace {

constexpr int kPlanItems = 16;
constexpr int kTilesPerSplit = 8;

// exclusive sum over the block; *total gets the block's sum
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[w] = x;
    __syncthreads();
    if (w == 0) {
        int y = lane < nw ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        if (lane < nw) s_warp[lane] = y;
    }
    __syncthreads();
    const int off = w > 0 ? s_warp[w - 1] : 0;
    *total = s_warp[nw - 1];
    __syncthreads();
    return off + x - v;
}

// sum over the block in a fixed tree; every thread gets it.  sh: blockDim.x doubles
__device__ __forceinline__ double block_sum(double v, double* sh) {
    sh[threadIdx.x] = v;
    __syncthreads();
    for (int s = blockDim.x >> 1; s > 0; s >>= 1) {
        if (threadIdx.x < s) sh[threadIdx.x] += sh[threadIdx.x + s];
        __syncthreads();
    }
    const double r = sh[0];
    __syncthreads();
    return r;
}

// the choice of the lane with the lowest cost (ties: the smaller choice)
__device__ __forceinline__ int warp_best(float cost, int choice) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float oc = __shfl_xor_sync(0xffffffffu, cost, o);
        const int ob = __shfl_xor_sync(0xffffffffu, choice, o);
        if (oc < cost || (oc == cost && ob < choice)) {
            cost = oc;
            choice = ob;
        }
    }
    return choice;
}

// (first valid row, valid rows) of a chunk; 0 rows past the last one
__device__ __forceinline__ int2 chunk_bounds(const int* counts, const int* cb, int chunk) {
    if (chunk >= counts[C_NCHUNKS]) return make_int2(0, 0);
    const int c0 = cb[chunk];
    return make_int2(c0, cb[chunk + 1] - c0);
}

template <bool kBf16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    const __half2_raw r{static_cast<unsigned short>(w & 0xFFFFu), static_cast<unsigned short>(w >> 16)};
    return __half22float2(__half2(r));
}

template <bool kBf16>
__device__ __forceinline__ uint16_t round16(float x) {
    return kBf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

// exponent all ones
template <bool kBf16>
__device__ __forceinline__ bool nonfinite16(uint16_t h) {
    constexpr uint16_t e = kBf16 ? 0x7F80 : 0x7C00;
    return (h & e) == e;
}

// h . W[tok] by one warp; every lane gets it
template <bool kBf16>
__device__ __forceinline__ double token_logit(const uint4* a, const uint4* b, int vpr, int lane) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = lane; i < vpr; i += 32) {
        const uint4 x = a[i], y = b[i];
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = unpack16<kBf16>(xw[j]), g = unpack16<kBf16>(yw[j]);
            acc[j] = fmaf(f.x, g.x, acc[j]);
            acc[j] = fmaf(f.y, g.y, acc[j]);
        }
    }
    double z = (static_cast<double>(acc[0]) + acc[1]) + (static_cast<double>(acc[2]) + acc[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    return z;
}

}  // namespace

// ------------------------------------------------------------ plan
// One block: 6 us up to 16,384 rows (latency), about 2 for each 16,384 more.
// It walks the mask in segments of 16 rows a thread and writes the valid
// rows in order, the number of valid rows before each completion, the chunk
// bounds and, for each chunk, how the logits' and dH's units are split.
//
// Logits split: a unit is (256 rows, nps vocabulary tiles of 256); nps is the one
// for which the units, one per SM pair at a time, take the fewest tile times,
// with 0.002 of a tile time for each split's partials.  At most kTilesPerSplit
// tiles: with long units all row tiles of the chunk are in flight at once, and h
// no longer stays in L2 (9728 rows, d = 4096, V = 32768: 64 tiles a unit read 3.9 GB
// from memory and took 1.45 ms, 8 read 0.9 GB and took 1.35).
//
// Chunks hold R rows, or (by_pair) as many whole pairs of completions as fit R
// rows: a pair's d loss / d q needs the sums over both completions, so a chunk
// of whole pairs can go from its logits to its gradients without computing the
// logits twice.
//
// dH split: dH's units (256 x 256 tiles, each a sum over the whole vocabulary)
// run in rounds of one per SM pair.  The units of the last round are cut into
// K pieces, which k_dh_join adds, so that all SM pairs share it; with dW's units
// in the same launch (head_grads_kernel) those share it first.  The cost model counts
// K-stages per SM pair: 12 and 4 for a dH and a dW unit's own cost, 0.3 for each
// partial tile's trip through memory.
template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) k_plan(const PlanParams p) {
    __shared__ int s_warp[32];
    __shared__ int s_act;
    const int tid = threadIdx.x;
    if (tid == 0) {
        *p.status = 0;
        if (p.found_inf) *p.found_inf = 0;
        if (p.loss) *p.loss = 0.f;
        s_act = 0;
    }
    const bool vec = p.mask && (reinterpret_cast<uintptr_t>(p.mask) & 15u) == 0;
    int carry = 0;
    for (int64_t base = 0; base < p.N; base += kPlanThreads * kPlanItems) {
        const int64_t t0 = base + tid * kPlanItems;
        uint32_t bits = 0;
        if (!p.mask) {
            const int64_t left = p.N - t0;
            bits = left >= kPlanItems ? 0xFFFFu : left > 0 ? (1u << left) - 1u : 0u;
        } else if (vec && t0 + kPlanItems <= p.N) {
            const uint4 u = *reinterpret_cast<const uint4*>(p.mask + t0);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < kPlanItems; ++k)
                if ((w[k >> 2] >> (8 * (k & 3))) & 0xFFu) bits |= 1u << k;
        } else {
#pragma unroll
            for (int k = 0; k < kPlanItems; ++k)
                if (t0 + k < p.N && p.mask[t0 + k] != 0) bits |= 1u << k;
        }
        int total;
        int vi = carry + block_scan(__popc(bits), s_warp, &total);
        for (int64_t b = (t0 + p.L - 1) / p.L * p.L; b < t0 + kPlanItems && b < p.N; b += p.L)
            p.off[b / p.L] = vi + __popc(bits & ((1u << (b - t0)) - 1u));
#pragma unroll
        for (int k = 0; k < kPlanItems; ++k)
            if ((bits >> k) & 1u) {
                if (GRPO_DCHECK(vi < p.N, p.status)) p.rows[vi] = static_cast<int>(t0 + k);
                ++vi;
            }
        carry += total;
    }
    const int nv = carry;
    if (tid == 0) p.off[p.n_seq] = nv;
    for (int c = tid; c < p.max_chunks; c += kPlanThreads) {
        p.gmax[c] = 0u;
        p.far[c] = 0;
    }
    __syncthreads();   // off is complete
    if (p.by_pair) {
        const int n_pr = p.n_seq / 2;
        if (tid == 0) {
            int c = 0, pr = 0;
            p.pb[0] = 0;
            p.cb[0] = 0;
            while (nv > 0 && pr < n_pr && GRPO_DCHECK(c < p.max_chunks, p.status)) {
                // the most pairs from pr on whose rows fit: off is monotonic, and one pair always fits
                const int first = p.off[2 * pr];
                int lo = pr + 1, hi = n_pr;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (p.off[2 * mid] - first <= p.R) lo = mid;
                    else hi = mid - 1;
                }
                pr = lo;
                ++c;
                p.pb[c] = pr;
                p.cb[c] = p.off[2 * pr];
            }
            p.counts[C_NCHUNKS] = c;
            for (int i = c + 1; i <= p.max_chunks; ++i) p.pb[i] = n_pr;
            if (c == 0) p.pb[1] = n_pr;   // no valid row: chunk 0 holds every (empty) pair
        }
    } else {
        const int n_chunks = (nv + p.R - 1) / p.R;
        for (int c = tid; c <= n_chunks; c += kPlanThreads)
            p.cb[c] = static_cast<int>(min(static_cast<int64_t>(c) * p.R, static_cast<int64_t>(nv)));
        if (tid == 0) p.counts[C_NCHUNKS] = n_chunks;
    }
    // completions, or pairs of them, with a valid row
    const int step = p.pairs_of_g2 ? 2 : 1;
    int act = 0;
    for (int i = tid * step; i < p.n_seq; i += kPlanThreads * step) act += p.off[i + step] > p.off[i];
    if (act) atomicAdd(&s_act, act);
    __syncthreads();
    if (tid == 0) {
        p.counts[C_NVALID] = nv;
        p.counts[C_NACT] = s_act;
    }
    // one warp per chunk; a lane weighs two numbers of splits or pieces
    const int n_chunks = p.counts[C_NCHUNKS];
    const int lane = tid & 31;
    for (int c = tid >> 5; c < n_chunks; c += kPlanThreads / 32) {
        const int row_pairs = (p.cb[c + 1] - p.cb[c] + 2 * kBM - 1) / (2 * kBM);
        float best_cost = 3e38f;
        int best = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = lane + 1 + 32 * h;   // tiles per split
            const int s = (p.n_ntiles + k - 1) / k;
            if (k > p.n_ntiles || s > p.s_max || (k > kTilesPerSplit && p.n_ntiles <= kTilesPerSplit * p.s_max)) continue;
            const float cost = static_cast<float>((row_pairs * s + p.n_pairs - 1) / p.n_pairs) * k + 0.002f * s;
            if (cost < best_cost) {
                best_cost = cost;
                best = k;
            }
        }
        best = warp_best(best_cost, best);
        if (lane == 0) p.lg_plan[c] = make_int2((p.n_ntiles + best - 1) / best, best);
        if (!p.backward) continue;
        const int units = row_pairs * p.n_nt;
        const int full = units / p.n_pairs * p.n_pairs, rem = units - full;
        const int ks_w = (p.cb[c + 1] - p.cb[c] + kBK - 1) / kBK;
        best_cost = 3e38f;
        best = 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int s = lane + 1 + 32 * h;
            if (rem == 0 || s > p.ks || (s > 1 && rem * s > p.slots_max)) continue;
            const int kper = (p.ks + s - 1) / s;
            if ((s - 1) * kper >= p.ks) continue;   // the last piece would be empty
            const float whole = static_cast<float>(full / p.n_pairs) * (p.ks + 12);
            const float last = static_cast<float>((rem * s + p.n_pairs - 1) / p.n_pairs) * (kper + 12);
            const float all = whole + (static_cast<float>(rem * s) * (kper + 12) + static_cast<float>(p.n_w) * (ks_w + 4)) / p.n_pairs;
            const float cost = fmaxf(whole + last, all) + (s > 1 ? 0.3f * rem * s : 0.f);
            if (cost < best_cost) {
                best_cost = cost;
                best = s;
            }
        }
        best = warp_best(best_cost, best);
        if (lane == 0) p.dh_plan[c] = make_int2(best > 1 ? full : units, best);
    }
}

cudaError_t launch_plan(const PlanParams& p, cudaStream_t st) {
    // few rows: fewer warps to synchronise
    if (p.N <= 256 * kPlanItems) k_plan<256><<<1, 256, 0, st>>>(p);
    else k_plan<1024><<<1, 1024, 0, st>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------ gather
// Blocks take work items in this order:
//   64 x 64 tiles of the chunk's rows: compact copy, and its transpose through
//     shared memory for dW's K-major operand; slots past the last row, up to
//     the next multiple of 128, become zeros
//   8 rows, one per warp: the given token's logit h . W[tok].  The tensor
//     cores round towards zero while they accumulate, so their logits are a
//     few 1e-6 of their size too small, always in one direction; a token that
//     the model finds likely would carry that into q and into sums of q over
//     thousands of tokens.  This dot product is summed in fp32 per lane and in
//     fp64 across lanes.
//   (chunk 0) 8 masked rows: zeros in dH and the per-row outputs
// Bound by HBM (9728 rows at d = 4096: 76 us for 320 MB), by latency for few rows.
constexpr int kGTile = 64;

template <bool kBf16>
__global__ void __launch_bounds__(256) k_head_gather(const GatherParams p) {
    __shared__ uint32_t tile[kGTile][kGTile / 2 + 1];
    const int2 cbn = chunk_bounds(p.counts, p.cb, p.chunk);
    const int c0 = cbn.x, n_c = cbn.y;
    if (n_c == 0 && p.chunk > 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_fill = min(p.R, (n_c + kBM - 1) / kBM * kBM);   // a multiple of 128
    const int nt_d = p.d / kGTile;
    const int64_t n_tiles = static_cast<int64_t>(n_fill / kGTile) * nt_d;
    const int64_t n_dots = (n_c + 7) / 8;
    const int64_t n_zero = p.chunk == 0 && p.mask ? (p.N + 7) / 8 : 0;
    const int vpr = p.d / 8;   // 16-byte vectors per row
    const uint4* h = reinterpret_cast<const uint4*>(p.h);
    for (int64_t it = blockIdx.x; it < n_tiles + n_dots + n_zero; it += gridDim.x) {
        if (it < n_tiles) {
            const int r0 = static_cast<int>(it / nt_d) * kGTile;
            const int d0 = static_cast<int>(it % nt_d) * kGTile;
            for (int i = threadIdx.x; i < kGTile * 8; i += blockDim.x) {
                const int r = i >> 3, v = i & 7;
                const int slot = r0 + r;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (slot < n_c) {
                    const int t = p.rows[c0 + slot];
                    if (GRPO_DCHECK(t >= 0 && t < p.N, p.status)) x = h[static_cast<int64_t>(t) * vpr + (d0 >> 3) + v];
                }
                reinterpret_cast<uint4*>(p.hc)[static_cast<int64_t>(slot) * vpr + (d0 >> 3) + v] = x;
                tile[r][4 * v] = x.x;
                tile[r][4 * v + 1] = x.y;
                tile[r][4 * v + 2] = x.z;
                tile[r][4 * v + 3] = x.w;
            }
            if (!p.hct) continue;   // uniform over the grid
            __syncthreads();
            for (int i = threadIdx.x; i < kGTile * 8; i += blockDim.x) {
                const int k = i >> 3, v = i & 7;   // output row d0 + k, slots r0 + 8v .. r0 + 8v + 7
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w0 = tile[8 * v + 2 * j][k >> 1], w1 = tile[8 * v + 2 * j + 1][k >> 1];
                    const uint32_t e0 = (k & 1) ? (w0 >> 16) : (w0 & 0xFFFFu);
                    const uint32_t e1 = (k & 1) ? (w1 >> 16) : (w1 & 0xFFFFu);
                    o[j] = e0 | (e1 << 16);
                }
                *reinterpret_cast<uint4*>(p.hct + static_cast<int64_t>(d0 + k) * p.R + r0 + 8 * v) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
            __syncthreads();
        } else if (it < n_tiles + n_dots) {
            const int slot = static_cast<int>(it - n_tiles) * 8 + warp;
            if (slot >= n_c) continue;
            const int t = p.rows[c0 + slot];
            if (!GRPO_DCHECK(t >= 0 && t < p.N, p.status)) continue;
            const int tok = p.tokens[t];
            double z = 0.0;
            if (tok >= 0 && tok < p.V)   // else the merge reports it
                z = token_logit<kBf16>(h + static_cast<int64_t>(t) * vpr,
                                       reinterpret_cast<const uint4*>(p.W) + static_cast<int64_t>(tok) * vpr, vpr, lane) *
                    static_cast<double>(p.zscale);
            if (lane == 0) p.zt[t] = z;
        } else {
            const int64_t t = (it - n_tiles - n_dots) * 8 + warp;
            if (t >= p.N || p.mask[t]) continue;
            if (p.dH) {
                uint4* o = reinterpret_cast<uint4*>(p.dH) + t * vpr;
                for (int i = lane; i < vpr; i += 32) o[i] = make_uint4(0, 0, 0, 0);
            }
            if (lane == 0) {
                if (p.out0) p.out0[t] = 0.f;
                if (p.out1) p.out1[t] = 0.f;
                if (p.stats)
                    for (int j = 0; j < 3; ++j) p.stats[3 * t + j] = 0.f;
            }
        }
    }
    if (p.dW && p.chunk == 0 && p.counts[C_NVALID] == 0) {
        const int64_t n16 = p.dw_bytes / 16;
        for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < n16; i += gridDim.x * 256LL)
            static_cast<uint4*>(p.dW)[i] = make_uint4(0, 0, 0, 0);
    }
}

cudaError_t launch_head_gather(const GatherParams& p, bool bf16, int sm_count, cudaStream_t st) {
    const int64_t tiles = static_cast<int64_t>(p.R / kGTile) * (p.d / kGTile) + (p.R + 7) / 8 +
                          (p.chunk == 0 ? (p.N + 7) / 8 : 0);
    const int blocks = static_cast<int>(tiles < sm_count * 8 ? tiles : sm_count * 8);
    if (bf16) k_head_gather<true><<<blocks, 256, 0, st>>>(p);
    else k_head_gather<false><<<blocks, 256, 0, st>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------ few rows: the given tokens' logits
// One block per row; block 0 also resets the status word and the counter of
// finished CTAs that head_few_kernel's last CTA is found by.
template <bool kBf16>
__global__ void __launch_bounds__(32) k_few_prep(const FewParams p, const uint4* __restrict__ h,
                                                 const uint4* __restrict__ W, double* __restrict__ zt) {
    chain_next();
    const int n = blockIdx.x, lane = threadIdx.x, vpr = p.d / 8;
    if (n == 0 && lane == 0) {
        *p.status = 0;
        *p.counter = 0;
    }
    const int tok = p.tokens[n];
    if ((p.mask && !p.mask[n]) || tok < 0 || tok >= p.V) return;
    const double z = token_logit<kBf16>(h + static_cast<int64_t>(n) * vpr, W + static_cast<int64_t>(tok) * vpr, vpr, lane);
    if (lane == 0) zt[n] = z * static_cast<double>(p.inv_t);
}

cudaError_t launch_few_prep(const FewParams& p, const uint16_t* h, const uint16_t* W, bool bf16, double* zt,
                            cudaStream_t st) {
    const uint4 *hv = reinterpret_cast<const uint4*>(h), *wv = reinterpret_cast<const uint4*>(W);
    if (bf16) k_few_prep<true><<<p.N, 32, 0, st>>>(p, hv, wv, zt);
    else k_few_prep<false><<<p.N, 32, 0, st>>>(p, hv, wv, zt);
    return cudaGetLastError();
}

// ------------------------------------------------------------ merge
// One warp per row of the chunk, reading its 2 S partials (at most 16 KB): 27 us for
// 4.9K rows of a 152K vocabulary.  HEAD_CLIP, with r = exp(q - q_old), x = p - q:
//   ell = -min(r A, clip(r) A) + beta (e^x - x - 1)
//   d ell / d q = -A r where the minimum is r A and moves with r, else 0;  + beta (1 - e^x)
// (r exactly at a border counts as not clipped.)  gco is d loss / d (h . W), the
// row's weight in the mean and 1 / temperature included; ell carries the weight too.
constexpr int kHeadMergeThreads = 256;

// One row's merge by one warp; lane 0 writes and returns what its dlogits need.
struct RowGrad {
    float2 lse2;
    float g, q;
    int tok;   // -1: nothing (a bad token id, reported here)
};

__device__ __forceinline__ RowGrad merge_row(const HeadMergeParams& p, int slot, int c0, int lane) {
    RowGrad out{make_float2(0.f, 0.f), 0.f, 0.f, -1};
    const int S2 = 2 * p.plan[p.chunk].x;
    const int t = p.rows[c0 + slot];
    if (!GRPO_DCHECK(t >= 0 && t < p.N, p.status)) return out;
    const int tok = p.tokens[t];
    const bool ok = tok >= 0 && tok < p.V;
    // a bad token's row has no sum; an infinite one makes its probabilities 0, whatever its logits
    RowSum r{0.0, 0.0, 0.f, make_float2(INFINITY, 0.f)};
    if (ok) r = p.relative ? join_row_relative(p.part + static_cast<int64_t>(slot) * S2, S2, lane, p.zt[t])
                           : join_row(p.part + static_cast<int64_t>(slot) * S2, S2, lane, p.zt[t]);
    if (lane != 0) return out;
    if (!ok) atomicCAS(p.status, 0, GRPO_ERR_SHAPE);
    const float q = static_cast<float>(r.q);
    if (p.far && !(q >= kLeastQ)) atomicOr(p.far + p.chunk, 1);
    float g = 0.f, ell = 0.f, ratio = 0.f, pen = 0.f;
    if (ok && p.mode == HEAD_GRAD) g = p.dlogp[t];
    if (ok && p.mode == HEAD_CLIP) {
        const int i = t / p.L;
        const float A = p.adv[i];
        ratio = expf(static_cast<float>(r.q - p.logp_old[t]));
        const bool cut = A >= 0.f ? ratio > p.clip_hi : ratio < p.clip_lo;
        ell = -A * (cut ? (A >= 0.f ? p.clip_hi : p.clip_lo) : ratio);
        g = cut ? 0.f : -A * ratio;
        if (p.logp_ref) {
            const float x = static_cast<float>(p.logp_ref[t] - r.q);
            const float em1 = expm1f(x);
            pen = em1 - x;
            ell = fmaf(p.beta, pen, ell);
            g = fmaf(-p.beta, em1, g);
        }
        const float w = p.loss_mode == GRPO_SEQUENCE_MEAN
                            ? 1.f / (static_cast<float>(p.off[i + 1] - p.off[i]) * p.counts[C_NACT])
                            : 1.f / p.counts[C_NVALID];
        ell *= w;
        g *= w;
    }
    g *= p.inv_t;
    p.lse2[t] = r.lse2;
    if (p.logp) p.logp[t] = q;
    if (p.entropy) p.entropy[t] = r.ent;
    if (p.stats) {
        p.stats[3 * static_cast<int64_t>(t)] = q;
        p.stats[3 * static_cast<int64_t>(t) + 1] = ratio;
        p.stats[3 * static_cast<int64_t>(t) + 2] = pen;
    }
    if (p.mode == HEAD_GRAD || p.mode == HEAD_CLIP) p.gco[t] = g;
    if (p.ell) p.ell[c0 + slot] = ell;
    out.lse2 = r.lse2;
    out.g = g;
    out.q = q;
    out.tok = ok ? tok : -1;
    return out;
}

__global__ void __launch_bounds__(kHeadMergeThreads) k_head_merge(const HeadMergeParams p) {
    __shared__ unsigned s_max;
    if (p.only_if && *p.only_if == 0) return;
    const int2 cbn = chunk_bounds(p.counts, p.cb, p.chunk);
    const int c0 = cbn.x, n_c = cbn.y;
    const int lane = threadIdx.x & 31;
    const int slot = blockIdx.x * (kHeadMergeThreads / 32) + (threadIdx.x >> 5);
    if (blockIdx.x * (kHeadMergeThreads / 32) >= n_c) return;
    if (threadIdx.x == 0) s_max = 0u;
    __syncthreads();
    if (slot < n_c && GRPO_DCHECK(slot < p.R, p.status)) {
        const RowGrad r = merge_row(p, slot, c0, lane);
        if (p.gmax && lane == 0) atomicMax(&s_max, __float_as_uint(fabsf(r.g)));
    }
    if (!p.gmax) return;
    __syncthreads();
    if (threadIdx.x == 0 && s_max) atomicMax(p.gmax + p.chunk, s_max);
}

cudaError_t launch_head_merge(const HeadMergeParams& p, cudaStream_t st) {
    constexpr int kRows = kHeadMergeThreads / 32;
    k_head_merge<<<(p.R + kRows - 1) / kRows, kHeadMergeThreads, 0, st>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------ preference loss
// One block per pair of completions (2i preferred, 2i + 1 not):
//   S = sum (or mean) over a completion's rows of q - p,   m = beta (S_2i - S_2i+1)
// and d loss / d q of their rows.  Sums in fp64 in a fixed order.  Pairs
// without a row are left out of the mean.  A row whose token is out of range adds
// 0 to S (its dlogits are zeros whatever its d loss / d q).  8 us (latency).
__global__ void __launch_bounds__(256) k_pair_coef(const PairParams p) {
    __shared__ double sh[256];
    __shared__ float s_g[2];
    const int pr = blockIdx.x;
    if (p.pb && (pr < p.pb[p.chunk] || pr >= p.pb[p.chunk + 1])) return;
    const int b[3] = {p.off[2 * pr], p.off[2 * pr + 1], p.off[2 * pr + 2]};
    double S[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        double acc = 0.0;
        for (int i = b[c] + threadIdx.x; i < b[c + 1]; i += 256) {
            const int t = p.rows[i];
            if (!GRPO_DCHECK(t >= 0 && t < p.N, p.status)) continue;
            // the three loads before the branch, so that their latencies overlap
            const int tok = p.tokens[t];
            const float q = p.logp[t], ref = p.logp_ref[t];
            if (tok >= 0 && tok < p.V) acc += static_cast<double>(q) - static_cast<double>(ref);
        }
        S[c] = block_sum(acc, sh);
        if (p.length_mean && b[c + 1] > b[c]) S[c] /= b[c + 1] - b[c];
    }
    if (threadIdx.x == 0) {
        const double beta = p.beta, e = p.smoothing;
        const double m = beta * (S[0] - S[1]);
        double ell = 0.0, dm = 0.0;
        if (b[2] > b[0]) {
            if (p.kind == GRPO_PAIR_HINGE) {
                ell = m < 1.0 ? 1.0 - m : 0.0;
                dm = m < 1.0 ? -1.0 : 0.0;
            } else if (p.kind == GRPO_PAIR_SQUARE) {
                const double x = (S[0] - S[1]) - 0.5 / beta;
                ell = x * x;
                dm = 2.0 * x / beta;
            } else {
                const float mf = static_cast<float>(m);
                const double up = log1pf(expf(-fabsf(mf))) + (m < 0.0 ? -m : 0.0);   // -log sigmoid(m)
                ell = up + e * m;                                                  // -log sigmoid(-m) = up + m
                dm = e - 1.f / (1.f + expf(mf));
            }
            if (m != m) ell = dm = m;   // a NaN stays one
        }
        const int n_act = p.counts[C_NACT];
        const double c = n_act > 0 ? beta * dm / n_act : 0.0;
        const int n0 = b[1] - b[0], n1 = b[2] - b[1];
        s_g[0] = static_cast<float>(p.length_mean && n0 > 0 ? c / n0 : c);
        s_g[1] = static_cast<float>(p.length_mean && n1 > 0 ? -c / n1 : -c);
        p.pair_ell[pr] = ell;
        if (p.pair_stats) {
            float* o = p.pair_stats + 4 * static_cast<int64_t>(pr);
            o[0] = static_cast<float>(beta * S[0]);
            o[1] = static_cast<float>(beta * S[1]);
            o[2] = static_cast<float>(m);
            o[3] = static_cast<float>(ell);
        }
        if (p.gmax && n0 > 0) atomicMax(p.gmax, __float_as_uint(fabsf(s_g[0])));
        if (p.gmax && n1 > 0) atomicMax(p.gmax, __float_as_uint(fabsf(s_g[1])));
    }
    if (!p.gco) return;
    __syncthreads();
    for (int i = b[0] + threadIdx.x; i < b[2]; i += 256) {
        const int t = p.rows[i];
        if (GRPO_DCHECK(t >= 0 && t < p.N, p.status)) p.gco[t] = i < b[1] ? s_g[0] : s_g[1];
    }
}

cudaError_t launch_pair_coef(const PairParams& p, cudaStream_t st) {
    k_pair_coef<<<p.n_pairs, 256, 0, st>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------ loss
// Without a backward; with one, an idle warp of the last chunk's dH kernel (or of the
// one for dH and dW) does the same.
__global__ void __launch_bounds__(32) k_loss(const LossParams l, const int* __restrict__ counts) {
    write_loss(l, counts, threadIdx.x);
}

cudaError_t launch_loss(const LossParams& l, const int* counts, cudaStream_t st) {
    k_loss<<<1, 32, 0, st>>>(l, counts);
    return cudaGetLastError();
}

// ------------------------------------------------------------ dlogits
// In place: the kept exponentials E = 2^(z log2 e - m) (fp16) of a row become
//   dS = g (onehot(tok) - E 2^(m - lse log2 e)),   m the base of the column's group of 32
// (lse log2 e as two fp32 numbers, see RowSum),
// rounded to the input type, which the two GEMMs need.  E is fp16 for both types: the
// chunk buffer has 16 bits an entry, and it is overwritten in place.  Beside bf16's
// rounding E's is small; fp16 dlogits have two roundings of one size (3.0e-4 of dH and
// dW together against 64 bits, fp32 exponentials 2.1e-4).  fp16 has no exponent range
// to spare: there g is multiplied by the power of two 2^e that takes the chunk's
// largest |g| to 2^13 .. 2^14, and the GEMMs' epilogues undo it (oscale), whatever
// the caller's loss scale is.  e reaches 162 (a saturated preference pair's g is
// 1e-36, fp32 goes down to 2^-149), where 2^e is no fp32 number: ldexpf applies it.
// Reads and writes the chunk once: bound by HBM.
// One row by one block; true if a value is not finite.
template <bool kBf16>
__device__ __forceinline__ bool dlogits_row(const HeadChunkParams& p, int slot, int tok, float2 lse2, float q, float coef) {
    uint4* row = reinterpret_cast<uint4*>(p.dS + static_cast<int64_t>(slot) * p.V_pad);
    const int nvec = p.V_pad / 8;
    const float dtok = -coef * expm1f(q);   // g (1 - p_tok)
    const float* mrow = p.mx + static_cast<int64_t>(slot) * p.nc32;
    bool bad = false;
    for (int i = threadIdx.x; i < nvec; i += kTransformThreads) {
        const int v0 = i * 8;
        const float c = coef * exp2f((mrow[v0 >> 5] - lse2.x) - lse2.y);
        const uint4 u = row[i];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int va = v0 + 2 * j, vb = va + 1;
            const float2 e = unpack16<false>(w[j]);
            float d0 = -c * e.x, d1 = -c * e.y;
            if (va == tok) d0 = dtok;
            if (vb == tok) d1 = dtok;
            if (va >= p.V) d0 = 0.f;
            if (vb >= p.V) d1 = 0.f;
            const uint16_t h0 = round16<kBf16>(d0), h1 = round16<kBf16>(d1);
            bad |= nonfinite16<kBf16>(h0) || nonfinite16<kBf16>(h1);
            o[j] = static_cast<uint32_t>(h0) | (static_cast<uint32_t>(h1) << 16);
        }
        row[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    return bad;
}

__device__ __forceinline__ void zero_row(const HeadChunkParams& p, int slot) {
    uint4* row = reinterpret_cast<uint4*>(p.dS + static_cast<int64_t>(slot) * p.V_pad);
    for (int i = threadIdx.x; i < p.V_pad / 8; i += kTransformThreads) row[i] = make_uint4(0, 0, 0, 0);
}

template <bool kBf16>
__global__ void __launch_bounds__(kTransformThreads) k_head_dlogits(const HeadChunkParams p, float* oscale) {
    const int2 cbn = chunk_bounds(p.counts, p.cb, p.chunk);
    const int c0 = cbn.x, n_c = cbn.y;
    if (n_c == 0 || (p.far && p.far[p.chunk] == 0)) return;
    int e = 0;
    if (!kBf16) {
        const float gm = __uint_as_float(p.gmax[p.gmax_chunk]);
        if (gm > 0.f && isfinite(gm)) e = 13 - ilogbf(gm);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) oscale[p.chunk] = kBf16 ? p.loss_scale : ldexpf(p.loss_scale, -e);
    const int n_fill = min(p.R, (n_c + kBM - 1) / kBM * kBM);
    bool bad = false;
    for (int slot = blockIdx.x; slot < n_fill; slot += gridDim.x) {
        if (slot >= n_c) {
            zero_row(p, slot);
            continue;
        }
        const int t = p.rows[c0 + slot];
        if (!GRPO_DCHECK(t >= 0 && t < p.N, p.status)) continue;
        const int tok = p.tokens[t];
        const float coef = tok >= 0 && tok < p.V ? (kBf16 ? p.gco[t] : ldexpf(p.gco[t], e)) : 0.f;
        bad |= dlogits_row<kBf16>(p, slot, tok, p.lse2[t], p.logp[t], coef);
    }
    if (__syncthreads_or(bad) && threadIdx.x == 0) atomicOr(p.found_inf, 1);
}

// Merge and dlogits of a bf16 chunk in one launch, one block per row: for chunks
// so small that the launches are what counts, where no step lies between the two
// (the preference loss sums over rows first; fp16 needs the chunk's largest g).
__global__ void __launch_bounds__(kTransformThreads) k_merge_dlogits(const HeadMergeParams m, const HeadChunkParams p,
                                                                     float* oscale) {
    __shared__ RowGrad s_row;
    const int2 cbn = chunk_bounds(p.counts, p.cb, p.chunk);
    const int c0 = cbn.x, n_c = cbn.y;
    if (n_c == 0) return;
    if (blockIdx.x == 0 && threadIdx.x == 0) oscale[p.chunk] = p.loss_scale;
    const int n_fill = min(p.R, (n_c + kBM - 1) / kBM * kBM);
    bool bad = false;
    for (int slot = blockIdx.x; slot < n_fill; slot += gridDim.x) {
        if (slot >= n_c) {
            zero_row(p, slot);
            continue;
        }
        if (threadIdx.x < 32) {
            const RowGrad r = merge_row(m, slot, c0, threadIdx.x);
            if (threadIdx.x == 0) s_row = r;
        }
        __syncthreads();
        const RowGrad r = s_row;
        bad |= dlogits_row<true>(p, slot, r.tok, r.lse2, r.q, r.tok >= 0 ? r.g : 0.f);
        __syncthreads();   // s_row is read
    }
    if (__syncthreads_or(bad) && threadIdx.x == 0) atomicOr(p.found_inf, 1);
}

cudaError_t launch_merge_dlogits(const HeadMergeParams& m, const HeadChunkParams& p, float* oscale, int sm_count,
                                 cudaStream_t st) {
    const int blocks = p.R < sm_count * 8 ? p.R : sm_count * 8;
    k_merge_dlogits<<<blocks, kTransformThreads, 0, st>>>(m, p, oscale);
    return cudaGetLastError();
}

cudaError_t launch_head_dlogits(const HeadChunkParams& p, float* oscale, bool bf16, int sm_count, cudaStream_t st) {
    const int blocks = p.R < sm_count * 8 ? p.R : sm_count * 8;
    if (bf16) k_head_dlogits<true><<<blocks, kTransformThreads, 0, st>>>(p, oscale);
    else k_head_dlogits<false><<<blocks, kTransformThreads, 0, st>>>(p, oscale);
    return cudaGetLastError();
}

// ------------------------------------------------------------ relative dlogits
// Without a pass over the dlogits.  The logits kernel knows the given token's
// logit beforehand and keeps A_v = e^(z_v - z_tok) = p_v / p_tok, so with
// s = sum of A over the other columns, p_tok = 1 / (1 + s) and
//   dS_v = g (onehot - p_v) = f A_v  with  f = -g p_tok  and  A_tok = -s.
// f is a factor of the row: dH's epilogue applies it, and for dW, where rows are
// summed, the rows of h carry it.  Roundings to bf16: A, which has to be a tensor
// core operand beside bf16 W and h, and f h, likewise, for dW.  The row's largest entry
// is the token's: f is taken as -g (1 - p_tok) / A_tok with A_tok as rounded, so that
// entry is exact in dH; the others carry A_tok's rounding (in f) beside their own,
// which is the better trade: half of a row's sum of absolute products is the token's
// (dH's error on 4.9K rows 1.7e-3 instead of 2.4e-3).  On 4.9K rows of a 152K vocabulary
// at d = 1536 this kernel and the empty fallback take 0.02 ms where the pass took 0.53.
//
// This kernel writes A_tok, f, and f h transposed for dW's K-major operand.  In
// a chunk that holds a row with q < kLeastQ (far), the logits kernel ran again
// with running maxima and the pass made the dlogits; f is 1 there.
__global__ void __launch_bounds__(256) k_head_scale(const HeadChunkParams p, float* oscale) {
    __shared__ uint32_t tile[kGTile][kGTile / 2 + 1];
    __shared__ float s_f[kGTile];
    const int2 cbn = chunk_bounds(p.counts, p.cb, p.chunk);
    const int c0 = cbn.x, n_c = cbn.y;
    if (n_c == 0) return;
    const bool far = p.far[p.chunk] != 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) oscale[p.chunk] = p.loss_scale;
    const int n_fill = min(p.R, (n_c + kBM - 1) / kBM * kBM);   // a multiple of 128
    const int nt_d = p.d / kGTile, vpr = p.d / 8;
    const int64_t n_tiles = static_cast<int64_t>(n_fill / kGTile) * nt_d;
    for (int64_t it = blockIdx.x; it < n_tiles; it += gridDim.x) {
        const int r0 = static_cast<int>(it / nt_d) * kGTile;
        const int d0 = static_cast<int>(it % nt_d) * kGTile;
        if (threadIdx.x < kGTile) {
            const int slot = r0 + threadIdx.x;
            float f = 0.f;
            if (slot < n_c) {
                const int t = p.rows[c0 + slot];
                if (GRPO_DCHECK(t >= 0 && t < p.N, p.status)) {
                    const int tok = p.tokens[t];
                    const float q = p.logp[t];
                    f = 1.f;
                    if (!far) {
                        // the entries are relative to the fp32 number that z_tok log2 e was rounded to
                        const double zt2 = p.zt[t] * 1.4426950408889634074;
                        const float up = exp2f(static_cast<float>(static_cast<double>(static_cast<float>(zt2)) - zt2));
                        const float s = expm1f(-q) / up;
                        const uint16_t s16 = round16<true>(s);
                        const float sr = __uint_as_float(static_cast<uint32_t>(s16) << 16);
                        f = -p.gco[t] * (sr > 0.f ? -expm1f(q) / sr : expf(q) * up);
                        if (d0 == 0 && tok >= 0 && tok < p.V)
                            p.dS[static_cast<int64_t>(slot) * p.V_pad + tok] = s16 ^ 0x8000u;
                    }
                }
                if (d0 == 0) p.rowf[slot] = f;
            }
            s_f[threadIdx.x] = f;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kGTile * 8; i += blockDim.x) {
            const int r = i >> 3, v = i & 7;
            const uint4 x = reinterpret_cast<const uint4*>(p.hc)[static_cast<int64_t>(r0 + r) * vpr + (d0 >> 3) + v];
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            const float f = s_f[r];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 y = unpack16<true>(w[j]);
                tile[r][4 * v + j] = static_cast<uint32_t>(round16<true>(f * y.x)) |
                                     (static_cast<uint32_t>(round16<true>(f * y.y)) << 16);
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kGTile * 8; i += blockDim.x) {
            const int k = i >> 3, v = i & 7;   // output row d0 + k, slots r0 + 8v .. r0 + 8v + 7
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w0 = tile[8 * v + 2 * j][k >> 1], w1 = tile[8 * v + 2 * j + 1][k >> 1];
                const uint32_t e0 = (k & 1) ? (w0 >> 16) : (w0 & 0xFFFFu);
                const uint32_t e1 = (k & 1) ? (w1 >> 16) : (w1 & 0xFFFFu);
                o[j] = e0 | (e1 << 16);
            }
            *reinterpret_cast<uint4*>(p.hct + static_cast<int64_t>(d0 + k) * p.R + r0 + 8 * v) =
                make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncthreads();
    }
}

cudaError_t launch_head_scale(const HeadChunkParams& p, float* oscale, int sm_count, cudaStream_t st) {
    const int64_t tiles = static_cast<int64_t>(p.R / kGTile) * (p.d / kGTile);
    const int blocks = static_cast<int>(tiles < sm_count * 8 ? tiles : sm_count * 8);
    k_head_scale<<<blocks, 256, 0, st>>>(p, oscale);
    return cudaGetLastError();
}

// ------------------------------------------------------------ dH join
// One warp per row (and 256 columns) of a split dH tile: adds its K pieces in order, scales,
// rounds and stores it.
template <bool kBf16>
__global__ void __launch_bounds__(256) k_dh_join(const HeadChunkParams p) {
    const int2 cbn = chunk_bounds(p.counts, p.cb, p.chunk);
    const int c0 = cbn.x, n_c = cbn.y;
    if (n_c == 0) return;
    const int2 plan = p.dh_plan[p.chunk];
    const int cols = p.dh_cols, halves = cols / kBN;
    const int n_nt = (p.d + cols - 1) / cols;
    const int units = (n_c + 2 * kBM - 1) / (2 * kBM) * n_nt;
    const int rem = units - plan.x;
    const float scale = p.oscale[p.chunk];
    const int ks = (p.V + kBK - 1) / kBK, piece = (ks + plan.y - 1) / plan.y * kBK;   // vocabulary rows of a K piece
    const int lane = threadIdx.x & 31;
    bool bad = false;
    for (int it = blockIdx.x * 8 + (threadIdx.x >> 5); it < rem * 2 * kBM * halves; it += gridDim.x * 8) {
        const int r = it / (2 * kBM * halves), rest = it - r * 2 * kBM * halves;
        const int row = rest / halves, col0 = (rest - row * halves) * kBN + 8 * lane;
        const int unit = plan.x + r;
        const int slot = unit / n_nt * 2 * kBM + row;
        const int col = unit % n_nt * cols + col0;
        if (slot >= n_c || col >= p.d) continue;
        const int t = p.rows[c0 + slot];
        if (!GRPO_DCHECK(t >= 0 && t < p.N, p.status)) continue;
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const float* src = p.dh_part + (static_cast<int64_t>(r) * 2 * kBM + row) * cols + col0;
        for (int s = 0; s < plan.y; ++s, src += static_cast<int64_t>(rem) * 2 * kBM * cols) {
            const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
            acc[0] += a.x, acc[1] += a.y, acc[2] += a.z, acc[3] += a.w;
            acc[4] += b.x, acc[5] += b.y, acc[6] += b.z, acc[7] += b.w;
        }
        float f = scale;
        if (p.V > kEvenVocab) f *= dh_gain(p.tokens[t], p.V, piece);
        if (p.rowf) f *= p.rowf[slot];
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint16_t h0 = round16<kBf16>(acc[2 * j] * f), h1 = round16<kBf16>(acc[2 * j + 1] * f);
            bad |= nonfinite16<kBf16>(h0) || nonfinite16<kBf16>(h1);
            o[j] = static_cast<uint32_t>(h0) | (static_cast<uint32_t>(h1) << 16);
        }
        *reinterpret_cast<uint4*>(p.dH + static_cast<int64_t>(t) * p.d + col) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (bad) atomicOr(p.found_inf, 1);
}

cudaError_t launch_head_dh_join(const HeadChunkParams& p, bool bf16, int sm_count, cudaStream_t st) {
    if (bf16) k_dh_join<true><<<sm_count * 4, 256, 0, st>>>(p);
    else k_dh_join<false><<<sm_count * 4, 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace grpo
