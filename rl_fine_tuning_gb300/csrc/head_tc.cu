// Tensor-core kernels of the head operators (tcgen05 + TMEM, fed by TMA).
//
//   head_logits_kernel  z = h . W^T of a chunk on SM pairs (M = 256: two row
//       tiles), with a streaming (max, sum exp) per row; the logits are never
//       written.  With a backward it keeps the exponentials, relative to the
//       running maximum or to the given token's logit (enum LogitsMode).
//   head_few_kernel     the same for at most 32 rows, W as the M operand, so
//       that W streams through the SMs once
//   head_dh_kernel, head_dh_wide_kernel   dH = dlogits . W
//   head_dw_kernel      dW = dlogits^T . h, written in the type of W or in fp32
//   head_grads_kernel   both, for small chunks
//
// Bounds and rates.  The chunk kernels are bound by the tensor cores, and in a
// long step by the card's power limit (cuBLAS sustains 1765 TFLOP/s in bf16 then,
// 1967 in a burst).  7500 rows of the 8B head (d = 4096, V = 128256), inside a step:
// logits 4.9 ms = 1.61 PFLOP/s (12% of it for storing the exponentials), dH
// 4.5 ms = 1.75, dW 4.55 ms = 1.73.  The few-row kernel is bound by HBM: 160 to
// 169 us for one row of that head on different cards, 93 to 98% of a copy's rate.
//
// Sums over K.  tcgen05.mma adds to its fp32 accumulator with rounding towards
// zero: after d / 16 additions a logit of 11 was 4.6e-5 too small at d = 4096
// (measured), always in one direction, so it stays in log-probs, in ratios
// near 1 and in sums of log-probs over a completion.  Two remedies:
//   - the tensor cores add only kPieceK products at a time, and the pieces
//     are added in registers, rounding to nearest.  Eight epilogue warps
//     hold one 128 x 256 accumulator (128 registers a thread).  4.9K rows of a
//     152K vocabulary at d = 1536: 1.27 ms with whole sums, 1.31 with pieces of
//     1024, 1.35 of 512, 1.50 of 256.
//   - each of n additions loses about half a unit in the last place of the
//     partial sum, whose expected value grows linearly to the final one, so
//     the loss is proportional to the sum: kAddLoss n.  Measured per addition:
//     1.43e-8 of the sum for n = 64, 1.57e-8 for n = 256, within 8% on five kinds
//     of inputs (half as much again with outlier columns).  The forward
//     kernels multiply it back in with the scale of the logits; what is left is
//     below 1.3e-7 of a logit, with outlier columns 5.4e-7.
#include <atomic>
#include <cfloat>

#include "head_join.cuh"
#include "tc_pair.cuh"

namespace grpo {

namespace {

// K-stages per piece: the fewest pieces of at most kPieceK, all of one length but
// for the last (a short piece leaves the epilogue too little time for the one
// before it: d = 1536 as 768 + 768 takes 8% less than as 1024 + 512)
__device__ __forceinline__ int piece_stages(int ks) {
    const int n = (ks * kBK + kPieceK - 1) / kPieceK;
    return (ks + n - 1) / n;
}

// ====================================================================== logits of a chunk

constexpr int kLgStages = 7;
constexpr int kLgStageBytes = 16384 + 16384;   // A (128 rows x 64), B half (128 vocabulary rows x 64)
constexpr int kLgSmem = kLgStages * kLgStageBytes + 1024 + 512;

// units: (row-tile pair, vocabulary split), row-tile pairs fastest within
// groups of kFwdGroup so that a W tile is shared in L2
struct LgSched {
    int n_units, ks, per, n_pc, n_mp, c0, n_c, S, nps;
};

__device__ __forceinline__ bool lg_setup(const LogitsParams& p, LgSched& sc) {
    if (p.chunk >= p.counts[C_NCHUNKS]) return false;
    sc.c0 = p.cb[p.chunk];
    sc.n_c = p.cb[p.chunk + 1] - sc.c0;
    sc.n_mp = (sc.n_c + 2 * kBM - 1) / (2 * kBM);
    sc.S = p.plan[p.chunk].x;
    sc.nps = p.plan[p.chunk].y;
    sc.n_units = sc.n_mp * sc.S;
    sc.ks = p.d / kBK;
    sc.per = piece_stages(sc.ks);
    sc.n_pc = (sc.ks + sc.per - 1) / sc.per;
    return sc.n_units > 0;
}

__device__ __forceinline__ int lg_items(const LogitsParams& p, const LgSched& sc, int split) {
    return min(split * sc.nps + sc.nps, p.n_ntiles) - split * sc.nps;
}

// One row's running statistics over the columns a thread sees: with m = max of
// z log2 e - kUp rounded up, s = sum 2^(z log2 e - m) and u = sum z 2^(z log2 e - m).
// In base 2 the rounding of m cancels; e^(z - m) with m log2 e rounded would not.
// Rounded up, because a step of logits of 1e7 is 1: an m too small by that would
// take the largest exponential out of fp16's range.  kUp lifts the exponentials to
// at most 2^14, so that fp16 keeps 11 bits of those down to 2^-28 of the largest.
constexpr float kUp = 14.f;

struct RowStat {
    float m, s, u;
};

template <bool kBf16, int kMode>
__device__ __forceinline__ void lg_body(const LogitsParams& p, const CUtensorMap& mA, const CUtensorMap& mB) {
    constexpr bool kKeep = kMode >= LG_KEEP_MAX, kEnt = kMode == LG_ENTROPY, kToken = kMode == LG_KEEP_TOKEN;
    extern __shared__ uint8_t smem_raw[];
    LgSched sc;
    if (p.only_if && *p.only_if == 0) return;
    if (!lg_setup(p, sc)) return;
    const int cid = static_cast<int>(blockIdx.x) >> 1;
    const int n_pairs = static_cast<int>(gridDim.x) >> 1;
    if (cid >= sc.n_units) return;   // uniform across the pair
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    Smem sm = carve_smem<kLgStages, kLgStageBytes>(smem_raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    int* status = p.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kLgStages; ++s) {
            mbar_init(&sm.full[s], 1);    // leader: its producer's expect_tx + both CTAs' bytes
            mbar_init(&sm.empty[s], 1);   // the leader's MMA commit, multicast to both CTAs
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.acc_full[b], 1);     // the leader's commit, multicast
            mbar_init(&sm.acc_empty[b], 16);   // leader: the eight epilogue warps of both CTAs
        }
        mbar_init(sm.drain, 1);
        *sm.abort_flag = 0;
        sm.ld_count[0] = sm.ld_count[1] = sm.ld_count[2] = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&mA);
        tma_prefetch_desc(&mB);
    }
    if (warp == 1) {
        tmem_alloc_pair(sm.tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *sm.tmem_slot;
    const uint32_t full0 = map_cluster(smem_u32(&sm.full[0]), 0);
    const uint32_t acc_empty0 = map_cluster(smem_u32(&sm.acc_empty[0]), 0);

    // 3 x 128 threads at 168 registers: the epilogue's two warpgroups take 216 each,
    // the first keeps 64 (216 + 216 + 64 <= 3 x 168)
    if (warp >= 4) {
        setmaxnreg_inc<216>();
        // ------------------------------------------------ epilogue: warp w holds lanes 32 (w % 4) .. + 31
        // and columns 128 half .. + 127 of the accumulator, one row per thread
        const int half = (warp - 4) >> 2;
        const int row = lane + 32 * (warp & 3);
        const uint32_t tq = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 128u * half;
        int it = 0;
        for (int unit = cid; unit < sc.n_units; unit += n_pairs) {
            int mp, split;
            decode_grouped(unit, sc.n_mp, sc.S, kFwdGroup, &mp, &split);
            const int n_items = lg_items(p, sc, split);
            const int slot = (2 * mp + rank) * kBM + row;
            bool valid = slot < sc.n_c && GRPO_DCHECK(slot < p.R, status);
            const int t = valid ? p.rows[sc.c0 + slot] : 0;
            if (valid && !GRPO_DCHECK(t >= 0 && t < p.N, status)) valid = false;
            const int tok = valid ? p.tokens[t] : -1;
            RowStat e{kNoLogit2, 0.f, 0.f};
            // rows past the chunk's last, up to the next multiple of 128: zeros with LG_KEEP_TOKEN (their
            // compact rows are zeros; with LG_KEEP_MAX the dlogits pass writes them)
            const bool stored = kToken ? p.E && slot < min(p.R, (sc.n_c + kBM - 1) / kBM * kBM) : valid;
            if (kToken) {
                const bool ok = valid && tok >= 0 && tok < p.V;
                e.m = ok ? static_cast<float>(p.zt[t] * 1.4426950408889634074) : INFINITY;
            }
            for (int item = 0; item < n_items; ++item) {
                float a[128];
                for (int pc = 0; pc < sc.n_pc; ++pc, ++it) {
                    const int b = it & 1;
                    if (!mbar_wait(&sm.acc_full[b], (it >> 1) & 1u, sm.abort_flag, status)) goto epi_done;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float v[32];
                        tmem_ld32(tq + b * 256 + c * 32, v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) a[32 * c + j] = pc == 0 ? v[j] : a[32 * c + j] + v[j];
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (leader) mbar_arrive(&sm.acc_empty[b]);
                        else mbar_arrive_peer(acc_empty0 + 8u * b);
                    }
                }
                const int n0 = (split * sc.nps + item) * kBN + 128 * half;
                float mv[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int col0 = n0 + 32 * c;
                    mv[c] = 0.f;
                    if (col0 >= p.V) continue;
                    float* v = a + 32 * c;
                    // columns past V and the row's own token do not count here
                    const int nvalid = p.V - col0;
                    if (nvalid < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j >= nvalid) v[j] = kNoLogit;
                    }
                    if (__any_sync(0xffffffffu, static_cast<unsigned>(tok - col0) < 32u)) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (tok == col0 + j) v[j] = kNoLogit;
                    }
                    float base = e.m;
                    if (!kToken) {
                        float cmax = v[0];
#pragma unroll
                        for (int j = 1; j < 32; ++j) cmax = fmaxf(cmax, v[j]);
                        base = fmaxf(e.m, __fmaf_ru(cmax, p.zscale2, -kUp));
                    }
                    float s0 = 0.f, s1 = 0.f, u0 = 0.f, u1 = 0.f;
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float x0 = fast_exp2(fmaf(v[j], p.zscale2, -base));
                        const float x1 = fast_exp2(fmaf(v[j + 1], p.zscale2, -base));
                        s0 += x0;
                        s1 += x1;
                        if (kEnt) {
                            u0 = fmaf(x0, v[j], u0);
                            u1 = fmaf(x1, v[j + 1], u1);
                        }
                        v[j] = x0;
                        v[j + 1] = x1;
                    }
                    if (kToken) {
                        e.s += s0 + s1;
                    } else {
                        const float f = fast_exp2(e.m - base);
                        e.s = fmaf(e.s, f, s0 + s1);
                        if (kEnt) e.u = fmaf(e.u, f, u0 + u1);
                        e.m = base;
                        mv[c] = base;
                    }
                    if (kKeep && stored && GRPO_DCHECK(col0 + 32 <= p.V_pad, status)) {
                        // 64 bytes of one row as two whole 32-byte sectors.  (Boxes through shared memory
                        // and TMA stores need a K-stage's room: 5% slower.)
                        uint16_t* e16 = p.E + static_cast<int64_t>(slot) * p.V_pad + col0;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float* w = v + 16 * h;
                            st_global_v8(e16 + 16 * h, pack2(w[0], w[1], kToken), pack2(w[2], w[3], kToken),
                                         pack2(w[4], w[5], kToken), pack2(w[6], w[7], kToken), pack2(w[8], w[9], kToken),
                                         pack2(w[10], w[11], kToken), pack2(w[12], w[13], kToken),
                                         pack2(w[14], w[15], kToken));
                        }
                    }
                }
                // nc32 is a multiple of 8 and n0 of 128: 16-byte aligned
                if (kMode == LG_KEEP_MAX && valid && GRPO_DCHECK((n0 >> 5) + 4 <= p.nc32, status))
                    *reinterpret_cast<float4*>(p.mx + static_cast<int64_t>(slot) * p.nc32 + (n0 >> 5)) =
                        make_float4(mv[0], mv[1], mv[2], mv[3]);
            }
            if (kEnt) e.u *= p.zscale;   // sum of z, not of the accumulator
            if (valid && GRPO_DCHECK(split >= 0 && split < sc.S, status))
                p.part[static_cast<int64_t>(slot) * (2 * sc.S) + 2 * split + half] = make_float4(e.m, e.s, e.u, 0.f);
        }
    epi_done:;
    } else {
        setmaxnreg_dec<64>();
        if (warp == 0) {
            // ------------------------------------------------ TMA producer (both CTAs)
            if (lane == 0) {
                int s = 0, n_issued = 0;
                uint32_t ph = 0;
                for (int unit = cid; unit < sc.n_units; unit += n_pairs) {
                    int mp, split;
                    decode_grouped(unit, sc.n_mp, sc.S, kFwdGroup, &mp, &split);
                    const int m0 = (2 * mp + rank) * kBM;
                    const int n_items = lg_items(p, sc, split);
                    for (int item = 0; item < n_items; ++item) {
                        const int n0 = (split * sc.nps + item) * kBN + rank * 128;
                        for (int k = 0; k < sc.ks; ++k) {
                            if (!mbar_wait(&sm.empty[s], ph ^ 1u, sm.abort_flag, status)) goto producer_done;
                            uint8_t* st = sm.stages + s * kLgStageBytes;
                            if (leader) mbar_arrive_expect_tx(&sm.full[s], 2 * kLgStageBytes);
                            tma_load_2d_pair(&mA, full0 + 8u * s, st, k * kBK, m0);
                            tma_load_2d_pair(&mB, full0 + 8u * s, st + 16384, k * kBK, n0);
                            ++n_issued;
                            if (++s == kLgStages) {
                                s = 0;
                                ph ^= 1u;
                            }
                        }
                    }
                }
            producer_done:
                sm.ld_count[0] = n_issued;
            }
        } else if (warp == 1) {
            // ------------------------------------------------ MMA issuer (leader only)
            if (lane == 0 && leader) {
                constexpr uint32_t idesc = make_idesc_f16(256, 256, kBf16, false, false);
                int s = 0, n_used = 0;
                uint32_t ph = 0;
                int it = 0;
                for (int unit = cid; unit < sc.n_units; unit += n_pairs) {
                    int mp, split;
                    decode_grouped(unit, sc.n_mp, sc.S, kFwdGroup, &mp, &split);
                    const int n_items = lg_items(p, sc, split);
                    for (int item = 0; item < n_items; ++item)
                        for (int k0 = 0; k0 < sc.ks; k0 += sc.per, ++it) {
                            const int b = it & 1;
                            if (!mbar_wait(&sm.acc_empty[b], ((it >> 1) & 1u) ^ 1u, sm.abort_flag, status)) goto mma_done;
                            tc_fence_after();
                            const uint32_t acc = tmem + b * 256;
                            const int k1 = min(k0 + sc.per, sc.ks);
                            for (int k = k0; k < k1; ++k) {
                                if (!mbar_wait(&sm.full[s], ph, sm.abort_flag, status)) goto mma_done;
                                ++n_used;
                                tc_fence_after();
                                const uint32_t st = smem_u32(sm.stages + s * kLgStageBytes);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    umma_pair_f16(acc, desc_kmajor(st + kk * 32), desc_kmajor(st + 16384 + kk * 32), idesc,
                                                  (k == k0 && kk == 0) ? 0u : 1u);
                                umma_pair_commit_both(&sm.empty[s]);
                                if (++s == kLgStages) {
                                    s = 0;
                                    ph ^= 1u;
                                }
                            }
                            umma_pair_commit_both(&sm.acc_full[b]);
                        }
                }
            mma_done:
                sm.ld_count[1] = n_used;
                umma_pair_commit(sm.drain);
                {
                    const uint32_t a = smem_u32(sm.drain);
                    const uint64_t t0 = globaltimer();
                    while (!mbar_try_wait(a, 0)) {
                        if (globaltimer() - t0 > kWaitTimeoutNs) {
                            atomicCAS(status, 0, GRPO_ERR_TIMEOUT);
                            break;
                        }
                    }
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // The end of tc_pair_body: after an abort in either CTA, the loads in
    // flight land before either CTA leaves; nobody leaves before both are done.
    cluster_sync();
    if (leader && threadIdx.x == 0) {
        const uint32_t peer_cnt = map_cluster(smem_u32(const_cast<int*>(sm.ld_count)), 1);
        const uint32_t peer_abort = map_cluster(smem_u32(const_cast<int*>(sm.abort_flag)), 1);
        const int peer_issued = static_cast<int>(ld_shared_cluster_u32(peer_cnt));
        const bool aborted = *sm.abort_flag || ld_shared_cluster_u32(peer_abort) != 0;
        int settled = 1;
        if (aborted) {
            const int issued = sm.ld_count[0], used = sm.ld_count[1];
            const int both = min(issued, peer_issued);
            settled = wait_inflight<kLgStages>(sm.full, used, both) && issued == peer_issued ? 1 : 0;
        }
        sm.ld_count[2] = settled;
        st_shared_cluster_u32(peer_cnt + 8u, static_cast<uint32_t>(settled));
    }
    cluster_sync();
    if (!sm.ld_count[2]) abort_grace(sm.abort_flag, true);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

template <bool kBf16, int kMode>
__global__ void __launch_bounds__(kHeadThreads, 1)
    head_logits_kernel(const __grid_constant__ LogitsParams p, const __grid_constant__ CUtensorMap mA,
                       const __grid_constant__ CUtensorMap mB) {
    lg_body<kBf16, kMode>(p, mA, mB);
}

// Shared memory limit and the number of clusters of two that fit on the device at
// once, set and asked once per kernel and device: both calls cost the host as
// much as a launch does.
constexpr int kDevices = 64;

template <auto kKern>
cudaError_t pairs_fit(int threads, int smem, int n_sm, int* clusters) {
    static std::atomic<int> known[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kDevices && (*clusters = known[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
    const void* fn = reinterpret_cast<const void*>(kKern);
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(n_sm / 2 * 2);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    *clusters = n_sm / 2;
    int active = 0;
    if (cudaOccupancyMaxActiveClusters(&active, fn, &cfg) == cudaSuccess && active > 0 && active < *clusters)
        *clusters = active;
    if (*clusters < 1) return cudaErrorInvalidConfiguration;
    if (dev < kDevices) known[dev].store(*clusters, std::memory_order_release);
    return cudaSuccess;
}

// Persistent launch of a kernel on SM pairs: one CTA per SM, capped by how many
// clusters fit on the device at once, so that every CTA runs concurrently.
template <auto kKern, class... A>
cudaError_t launch_pairs(int threads, int smem, int n_sm, cudaStream_t st, const A&... args) {
    int clusters = 0;
    const cudaError_t e = pairs_fit<kKern>(threads, smem, n_sm, &clusters);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(clusters * 2);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kKern, args...);
}

// ====================================================================== few rows
// z^T = W . h^T: a tile is 128 vocabulary rows (M) by kNC hidden rows (N), so
// W goes through shared memory once and nothing else of size does.  A thread
// owns one vocabulary row of the tile: its columns are the hidden rows, whose
// running (max, sum exp, sum z exp) it keeps over all of its CTA's tiles; the
// 128 threads are joined once at the end, and the last CTA to finish joins the
// CTAs' partials.  The bytes of W are the floor.
template <int kNC>
struct FewShape {
    static constexpr int kStageBytes = 16384 + kNC * 128;
    static constexpr int kStages = 200 * 1024 / kStageBytes;
    static constexpr int kSmem = kStages * kStageBytes + 1024 + 512;
};

template <bool kBf16, int kNC>
__global__ void __launch_bounds__(kThreads, 1)
    head_few_kernel(const __grid_constant__ FewParams p, const __grid_constant__ CUtensorMap mH,
                    const __grid_constant__ CUtensorMap mW) {
    using F = FewShape<kNC>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_tok[kNC];
    __shared__ float s_part[4][kNC][3];
    __shared__ int s_last;
    Smem sm = carve_smem<F::kStages, F::kStageBytes>(smem_raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    int* status = p.status;
    const int ks = p.d / kBK, per = piece_stages(ks);

    if (threadIdx.x == 0) {
        for (int s = 0; s < F::kStages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.acc_full[b], 1);
            mbar_init(&sm.acc_empty[b], 4);
        }
        mbar_init(sm.drain, 1);
        *sm.abort_flag = 0;
        sm.ld_count[0] = sm.ld_count[1] = sm.ld_count[2] = 0;
        fence_barrier_init();
    }
    if (threadIdx.x < kNC) s_tok[threadIdx.x] = static_cast<int>(threadIdx.x) < p.N ? p.tokens[threadIdx.x] : -1;
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&mH);
        tma_prefetch_desc(&mW);
    }
    if (warp == 1) {
        tmem_alloc(sm.tmem_slot, 2 * kNC);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sm.tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, n_issued = 0;
            uint32_t ph = 0;
            for (int tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x)
                for (int k = 0; k < ks; ++k) {
                    if (!mbar_wait(&sm.empty[s], ph ^ 1u, sm.abort_flag, status)) goto producer_done;
                    uint8_t* st = sm.stages + s * F::kStageBytes;
                    mbar_arrive_expect_tx(&sm.full[s], F::kStageBytes);
                    tma_load_2d(&mW, &sm.full[s], st, k * kBK, tile * kFewVocab);
                    tma_load_2d(&mH, &sm.full[s], st + 16384, k * kBK, 0);
                    ++n_issued;
                    if (++s == F::kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
        producer_done:
            sm.ld_count[0] = n_issued;
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = make_idesc_f16(128, kNC, kBf16, false, false);
            int s = 0, n_used = 0, it = 0;
            uint32_t ph = 0;
            for (int tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x)
                for (int k0 = 0; k0 < ks; k0 += per, ++it) {
                    const int b = it & 1;
                    if (!mbar_wait(&sm.acc_empty[b], ((it >> 1) & 1u) ^ 1u, sm.abort_flag, status)) goto mma_done;
                    tc_fence_after();
                    const int k1 = min(k0 + per, ks);
                    for (int k = k0; k < k1; ++k) {
                        if (!mbar_wait(&sm.full[s], ph, sm.abort_flag, status)) goto mma_done;
                        ++n_used;
                        tc_fence_after();
                        const uint32_t st = smem_u32(sm.stages + s * F::kStageBytes);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16(tmem + b * kNC, desc_kmajor(st + kk * 32), desc_kmajor(st + 16384 + kk * 32), idesc,
                                     (k == k0 && kk == 0) ? 0u : 1u);
                        umma_commit(&sm.empty[s]);
                        if (++s == F::kStages) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    umma_commit(&sm.acc_full[b]);
                }
        mma_done:
            sm.ld_count[1] = n_used;
            umma_commit(sm.drain);
            {
                const uint32_t a = smem_u32(sm.drain);
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(a, 0)) {
                    if (globaltimer() - t0 > kWaitTimeoutNs) {
                        atomicCAS(status, 0, GRPO_ERR_TIMEOUT);
                        break;
                    }
                }
            }
        }
    } else {
        const int quarter = warp & 3;
        const uint32_t tq = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        float m[kNC], s[kNC], u[kNC];
#pragma unroll
        for (int n = 0; n < kNC; ++n) {
            m[n] = kNoLogit2;
            s[n] = u[n] = 0.f;
        }
        int it = 0;
        for (int tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x) {
            float a[kNC];
            for (int k0 = 0; k0 < ks; k0 += per, ++it) {
                const int b = it & 1;
                if (!mbar_wait(&sm.acc_full[b], (it >> 1) & 1u, sm.abort_flag, status)) goto epi_done;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kNC / 16; ++c) {
                    float v[16];
                    tmem_ld16(tq + b * kNC + 16 * c, v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) a[16 * c + j] = k0 == 0 ? v[j] : a[16 * c + j] + v[j];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.acc_empty[b]);
            }
            const int vr = tile * kFewVocab + 32 * quarter + lane;
#pragma unroll
            for (int n = 0; n < kNC; ++n) {
                const float z = vr < p.V && vr != s_tok[n] ? a[n] : kNoLogit;
                const float mn = fmaxf(m[n], __fmul_ru(z, p.zscale2));
                const float f = fast_exp2(m[n] - mn), x = fast_exp2(fmaf(z, p.zscale2, -mn));
                s[n] = fmaf(s[n], f, x);
                u[n] = fmaf(u[n], f, x * z);
                m[n] = mn;
            }
        }
        // the 32 vocabulary rows of the warp, then the four warps through shared memory
#pragma unroll
        for (int n = 0; n < kNC; ++n) {
            float mw = m[n];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
            const float f = fast_exp2(m[n] - mw);
            float sw = s[n] * f, uw = u[n] * f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                sw += __shfl_xor_sync(0xffffffffu, sw, o);
                uw += __shfl_xor_sync(0xffffffffu, uw, o);
            }
            if (lane == 0) {
                s_part[quarter][n][0] = mw;
                s_part[quarter][n][1] = sw;
                s_part[quarter][n][2] = uw * p.zscale;
            }
        }
    epi_done:;
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*sm.abort_flag) {
        if (threadIdx.x == 0)
            sm.ld_count[2] = wait_inflight<F::kStages>(sm.full, sm.ld_count[1], sm.ld_count[0]) ? 1 : 0;
        __syncthreads();
        if (!sm.ld_count[2]) abort_grace(sm.abort_flag);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kNC);
    }
    // W, h and the tokens are the caller's and were there before k_few_prep began;
    // its own results (zt, the counter) are needed from here on
    chain_wait();
    // this CTA's partial of each row
    const int n_cta = static_cast<int>(gridDim.x);
    if (static_cast<int>(threadIdx.x) < min(kNC, p.N)) {
        const int n = threadIdx.x;
        float mm = s_part[0][n][0], ss = 0.f, uu = 0.f;
#pragma unroll
        for (int w = 1; w < 4; ++w) mm = fmaxf(mm, s_part[w][n][0]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = exp2f(s_part[w][n][0] - mm);
            ss = fmaf(s_part[w][n][1], f, ss);
            uu = fmaf(s_part[w][n][2], f, uu);
        }
        p.part[static_cast<int64_t>(n) * n_cta + blockIdx.x] = make_float4(mm, ss, uu, 0.f);
        __threadfence();
    }
    __syncthreads();
    if (threadIdx.x == 0) s_last = atomicAdd(p.counter, 1) == n_cta - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    for (int n = warp; n < p.N; n += kThreads / 32) {
        const int tok = s_tok[n];
        const bool on = !p.mask || p.mask[n] != 0;
        const bool ok = tok >= 0 && tok < p.V;
        RowSum r{0.0, 0.0, 0.f, make_float2(0.f, 0.f)};
        if (on && ok) r = join_row_once<kFewCtas / 32>(p.part + static_cast<int64_t>(n) * n_cta, n_cta, lane, p.zt[n]);
        if (lane == 0) {
            if (on && !ok) atomicCAS(status, 0, GRPO_ERR_SHAPE);
            p.logp[n] = static_cast<float>(r.q);
            if (p.entropy) p.entropy[n] = r.ent;
        }
    }
}

// Watches stored values for one that is not finite: 0 x is NaN for those alone, so
// a sum of them tells with one instruction per (packed pair of) value.
template <bool kBf16>
struct Finite {
    __nv_bfloat162 b = __floats2bfloat162_rn(0.f, 0.f);
    __half2 h = __floats2half2_rn(0.f, 0.f);
    float f = 0.f;
    __device__ __forceinline__ void see(uint32_t pk) {
        if (kBf16) b = __hfma2(reinterpret_cast<const __nv_bfloat162&>(pk), __floats2bfloat162_rn(0.f, 0.f), b);
        else h = __hfma2(reinterpret_cast<const __half2&>(pk), __floats2half2_rn(0.f, 0.f), h);
    }
    __device__ __forceinline__ void see_f32(float x) { f = fmaf(x, 0.f, f); }
    __device__ __forceinline__ bool bad() const {
        const float2 t = kBf16 ? __bfloat1622float2(b) : __half22float2(h);
        return !(t.x == 0.f && t.y == 0.f && f == 0.f);
    }
};

// ====================================================================== gradients
// dH's units are 256 x 256 tiles, sums over the vocabulary, some cut into K pieces;
// dW's are 256 x 256 tiles, sums over the chunk's rows.
//
// Eight epilogue warps, the second four for the upper half of the columns: a dW
// unit of 1000 rows has 8200 clocks of MMAs, and four warps took longer than that.
// A thread stores 32-byte pieces of its own row; boxes through shared memory and
// TMA stores were 10% faster for dW of a few rows, but they need a K-stage's room,
// which costs as much elsewhere.

// the loss, once all rows are merged (with the last chunk that has rows)
__device__ __forceinline__ void idle_loss(const HeadChunkParams& p, int lane) {
    if (blockIdx.x < 2 && p.chunk + 1 == p.counts[C_NCHUNKS]) write_loss(p.loss, p.counts, lane);
}

// Base: DhPairT (256 columns a unit) or DhPairWideT (512: the staged dlogits feed
// two MMAs, so they are read half as often, and half the shared memory traffic
// is theirs: 7% less time for dH of 7500 rows of the 8B head).
template <class Base, int kCols>
struct HeadDh : Base {
    static constexpr int kEpiWarps = 8;
    static constexpr bool kIdle = true;
    using Params = HeadChunkParams;
    using Epi = typename Base::Epi;
    using BaseCoord = typename Base::Coord;
    __device__ static void idle(const Params& p, int lane) { idle_loss(p, lane); }
    struct Sched : ChunkSched {
        int n_full, pieces, rem, kper;
    };
    struct Coord {
        int m0, n0, k0;
    };
    __device__ static bool setup(const Params& p, Sched& sc) {
        if (!Base::setup(p, sc)) return false;
        const int units = sc.n_units;
        const int2 plan = p.dh_plan[p.chunk];
        sc.n_full = plan.x;
        sc.pieces = plan.y;
        sc.rem = units - plan.x;
        sc.kper = (sc.ks + plan.y - 1) / plan.y;
        sc.n_units = sc.n_full + sc.rem * sc.pieces;
        return sc.n_units > 0;
    }
    // unit -> (tile unit, K piece; -1 for all of K).  Pieces are the slow index: the
    // tiles of one K range run together and share its W rows in L2.
    __device__ static int2 piece(const Sched& sc, int unit) {
        if (unit < sc.n_full) return make_int2(unit, -1);
        const int r = unit - sc.n_full;
        return make_int2(sc.n_full + r % sc.rem, r / sc.rem);
    }
    __device__ static int ksteps(const Params&, const Sched& sc, int unit) {
        const int2 u = piece(sc, unit);
        return u.y < 0 ? sc.ks : min(sc.kper, sc.ks - u.y * sc.kper);
    }
    __device__ static Coord coord(const Params&, const Sched& sc, int unit, int, int rank) {
        const int2 u = piece(sc, unit);
        return Coord{Base::mtile(sc, u.x, rank) * kBM, Base::dtile(sc, u.x) * kCols, u.y < 0 ? 0 : u.y * sc.kper};
    }
    __device__ static uint32_t tx_bytes(const Params& p, const Sched& sc, const Coord& c) {
        return Base::tx_bytes(p, sc, BaseCoord{c.m0, c.n0});
    }
    __device__ static void load(const Params& p, const Sched& sc, const Coord& c, int k, uint8_t* st, uint32_t bar,
                                const CUtensorMap* mA, const CUtensorMap* mA2, const CUtensorMap* mB, int rank) {
        Base::load(p, sc, BaseCoord{c.m0, c.n0}, c.k0 + k, st, bar, mA, mA2, mB, rank);
    }
    __device__ static void epi_begin(const Params&, const Sched&, int, int, int, Epi&) {}
    __device__ static void epi_end(const Params&, const Sched&, int, Epi&) {}
    template <bool kBf16>
    __device__ static void epi_item(const Params& p, const Sched& sc, int unit, int, int rank, uint32_t tacc, Epi&) {
        const int warp = threadIdx.x >> 5;
        const int row = (threadIdx.x & 31) + 32 * (warp & 3);
        const int c0 = ((warp - 2) >> 2) * (kCols / 64), c1 = c0 + kCols / 64;   // 32-column groups of this warp
        const int2 u = piece(sc, unit);
        const int slot = Base::mtile(sc, u.x, rank) * kBM + row;
        const int n0 = Base::dtile(sc, u.x) * kCols;
        bool valid = slot < sc.n_c;
        if (!__any_sync(0xffffffffu, valid)) return;
        if (u.y >= 0) {
            // partial tile: [piece][tile][256 rows][kCols] fp32
            const int64_t tile = static_cast<int64_t>(u.y) * sc.rem + (u.x - sc.n_full);
            float* out = p.dh_part + ((tile * 2 + rank) * kBM + row) * kCols;
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
                if (n0 + c * 32 >= p.d) break;
                float v[32];
                tmem_ld32(tacc + c * 32, v);
                if (valid) {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        st_global_v8(out + c * 32 + 8 * h, __float_as_uint(v[8 * h]), __float_as_uint(v[8 * h + 1]),
                                     __float_as_uint(v[8 * h + 2]), __float_as_uint(v[8 * h + 3]),
                                     __float_as_uint(v[8 * h + 4]), __float_as_uint(v[8 * h + 5]),
                                     __float_as_uint(v[8 * h + 6]), __float_as_uint(v[8 * h + 7]));
                }
            }
            return;
        }
        const int t = valid ? p.rows[sc.c0 + slot] : 0;
        if (valid && !GRPO_DCHECK(t >= 0 && t < p.N, p.status)) valid = false;
        float f = sc.winv;
        if (valid) {
            if (p.V > kEvenVocab) f *= dh_gain(p.tokens[t], p.V, p.V);
            if (p.rowf) f *= p.rowf[slot];
        }
        uint16_t* out = p.dH + static_cast<int64_t>(t) * p.d;
        Finite<kBf16> fin;
#pragma unroll 1
        for (int c = c0; c < c1; ++c) {
            const int col0 = n0 + c * 32;
            if (col0 >= p.d) break;
            float v[32];
            tmem_ld32(tacc + c * 32, v);
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                pk[j / 2] = pack2(v[j] * f, v[j + 1] * f, kBf16);
                fin.see(pk[j / 2]);
            }
            if (valid) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    st_global_v8(out + col0 + 16 * h, pk[8 * h], pk[8 * h + 1], pk[8 * h + 2], pk[8 * h + 3],
                                 pk[8 * h + 4], pk[8 * h + 5], pk[8 * h + 6], pk[8 * h + 7]);
            }
        }
        if (valid && fin.bad()) atomicOr(p.found_inf, 1);
    }
};
using HeadDhT = HeadDh<DhPairT, kBN>;
using HeadDhWideT = HeadDh<DhPairWideT, 2 * kBN>;

// DwPairT with the operators' output: chunks add up in fp32 (dw_acc), and with
// dw16 the last chunk (often the only one) rounds the sum to the type of W.
struct HeadDwT : DwPairT {
    static constexpr int kEpiWarps = 8;
    using Params = HeadChunkParams;
    struct Sched : ChunkSched {
        bool last;   // this chunk completes the 16-bit dW
    };
    __device__ static bool setup(const Params& p, Sched& sc) {
        sc.last = p.dw16 && p.chunk + 1 == p.counts[C_NCHUNKS];
        return DwPairT::setup(p, sc);
    }
    __device__ static void epi_begin(const Params&, const Sched&, int, int, int, Epi&) {}
    __device__ static void epi_end(const Params&, const Sched&, int, Epi&) {}
    template <bool kBf16>
    __device__ static void epi_item(const Params& p, const Sched& sc, int unit, int, int rank, uint32_t tacc, Epi&) {
        const int warp = threadIdx.x >> 5;
        const int row = (threadIdx.x & 31) + 32 * (warp & 3);
        const int c0 = ((warp - 2) >> 2) * (kBN / 64), c1 = c0 + kBN / 64;   // 32-column groups of this warp
        const int v = vtile(sc, unit, rank) * kBM + row;
        const int n0 = dtile(sc, unit) * kBN;
        const bool valid = v < p.V;
        if (!__any_sync(0xffffffffu, valid)) return;
        const bool first = p.chunk == 0;
        const int64_t at = static_cast<int64_t>(valid ? v : 0) * p.d;
        Finite<kBf16> fin;
#pragma unroll 1
        for (int c = c0; c < c1; ++c) {
            const int col0 = n0 + c * 32;
            if (col0 >= p.d) break;
            float x[32];
            tmem_ld32(tacc + c * 32, x);
            if (!valid) continue;
            float* acc = p.dw_acc + at + col0;
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] *= sc.winv;
            if (!first) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float prev[8];
                    ld_global_v8(acc + 8 * j, prev);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[8 * j + i] += prev[i];
                }
            }
            if (sc.last) {
                uint32_t pk[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    pk[j] = pack2(x[2 * j], x[2 * j + 1], kBf16);
                    fin.see(pk[j]);
                }
                uint16_t* out = p.dw16 + at + col0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    st_global_v8(out + 16 * h, pk[8 * h], pk[8 * h + 1], pk[8 * h + 2], pk[8 * h + 3], pk[8 * h + 4],
                                 pk[8 * h + 5], pk[8 * h + 6], pk[8 * h + 7]);
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) fin.see_f32(x[j]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    st_global_v8(acc + 8 * j, __float_as_uint(x[8 * j]), __float_as_uint(x[8 * j + 1]),
                                 __float_as_uint(x[8 * j + 2]), __float_as_uint(x[8 * j + 3]),
                                 __float_as_uint(x[8 * j + 4]), __float_as_uint(x[8 * j + 5]),
                                 __float_as_uint(x[8 * j + 6]), __float_as_uint(x[8 * j + 7]));
            }
        }
        if (valid && fin.bad()) atomicOr(p.found_inf, 1);
    }
};

// Both in one launch, for small chunks: dH's units come first, one per SM pair at
// a time; the pairs left over in dH's last round go on with dW's units, and all
// share the rest of those.
struct HeadGradsT {
    static constexpr int kStages = 7;
    static constexpr int kStageBytes = DhPairT::kStageBytes;
    static constexpr int kEpiWarps = 8;
    static constexpr bool kMixed = true, kIdle = true;
    static_assert(DhPairT::kStageBytes == DwPairT::kStageBytes, "one ring for both");
    using Params = HeadChunkParams;
    // Pair c of np does dH units c, c + np, ...: `full` rounds, and pairs below `r`
    // one more.  Meanwhile the others do `x` dW units each, as many as that round
    // takes; then all pairs share the dW units that are left.
    struct Sched {
        HeadDhT::Sched h;
        HeadDwT::Sched w;
        int n_units, np, full, r, x;
    };
    struct Coord {
        int w;                // 1: dW
        int a, b, k0;         // dH: m0, n0, first K-stage; dW: v0, n0
    };
    struct Epi {
        int unused;
    };
    __device__ static bool setup(const Params& p, Sched& sc) {
        if (!HeadDhT::setup(p, sc.h) || !HeadDwT::setup(p, sc.w)) return false;
        sc.np = static_cast<int>(gridDim.x) >> 1;
        sc.full = sc.h.n_units / sc.np;
        sc.r = sc.h.n_units - sc.full * sc.np;
        // K-stages of the last round's units, and 12 and 4 for the units' own cost (as in k_plan)
        const int kl = (sc.h.rem > 0 ? sc.h.kper : sc.h.ks) + 12;
        sc.x = sc.r > 0 ? min(kl / (sc.w.ks + 4), sc.w.n_units / (sc.np - sc.r)) : 0;
        const int rest = sc.w.n_units - (sc.np - sc.r) * sc.x;
        const int rounds = sc.full + max(sc.r > 0 ? 1 : 0, sc.x) + (rest + sc.np - 1) / sc.np;
        sc.n_units = rounds * sc.np;
        return true;
    }
    // unit = round * np + pair -> (kind: 0 dH, 1 dW, -1 nothing; index of that kind's unit)
    __device__ static int2 pick(const Sched& sc, int unit) {
        int j = unit / sc.np;
        const int c = unit - j * sc.np;
        if (j < sc.full) return make_int2(0, unit);
        j -= sc.full;
        const int others = sc.np - sc.r;
        if (c < sc.r) {
            if (j == 0) return make_int2(0, sc.full * sc.np + c);
            j -= 1;
        } else {
            if (j < sc.x) return make_int2(1, j * others + c - sc.r);
            j -= sc.x;
        }
        const int w = others * sc.x + j * sc.np + c;
        return w < sc.w.n_units ? make_int2(1, w) : make_int2(-1, 0);
    }
    __device__ static int items(const Params&, const Sched& sc, int unit) { return pick(sc, unit).x >= 0 ? 1 : 0; }
    __device__ static int ksteps(const Params& p, const Sched& sc, int unit) {
        const int2 u = pick(sc, unit);
        return u.x == 1 ? sc.w.ks : u.x == 0 ? HeadDhT::ksteps(p, sc.h, u.y) : 0;
    }
    __device__ static Coord coord(const Params& p, const Sched& sc, int unit, int item, int rank) {
        const int2 u = pick(sc, unit);
        if (u.x == 1) {
            const DwPairT::Coord c = DwPairT::coord(p, sc.w, u.y, item, rank);
            return Coord{1, c.v0, c.n0, 0};
        }
        const HeadDhT::Coord c = HeadDhT::coord(p, sc.h, u.y, item, rank);
        return Coord{0, c.m0, c.n0, c.k0};
    }
    __device__ static uint32_t tx_bytes(const Params& p, const Sched& sc, const Coord& c) {
        return c.w ? DwPairT::tx_bytes(p, sc.w, DwPairT::Coord{c.a, c.b}) : HeadDhT::tx_bytes(p, sc.h, HeadDhT::Coord{c.a, c.b, 0});
    }
    __device__ static void load(const Params& p, const Sched& sc, const Coord& c, int k, uint8_t* st, uint32_t bar,
                                const CUtensorMap* mA, const CUtensorMap* mA2, const CUtensorMap* mB, int rank) {
        if (c.w) DwPairT::load(p, sc.w, DwPairT::Coord{c.a, c.b}, k, st, bar, mA2, mA2, &p.mHct, rank);
        else HeadDhT::load(p, sc.h, HeadDhT::Coord{c.a, c.b, c.k0}, k, st, bar, mA, mA2, mB, rank);
    }
    __device__ static int kind(const Sched& sc, int unit) { return pick(sc, unit).x; }
    template <bool kBf16>
    __device__ static void mma_kind(int kind, uint32_t st, uint32_t acc, bool first) {
        if (kind == 1) DwPairT::mma<kBf16>(st, acc, first);
        else DhPairT::mma<kBf16>(st, acc, first);
    }
    __device__ static void idle(const Params& p, int lane) { idle_loss(p, lane); }
    __device__ static void epi_begin(const Params&, const Sched&, int, int, int, Epi&) {}
    __device__ static void epi_end(const Params&, const Sched&, int, Epi&) {}
    template <bool kBf16>
    __device__ static void epi_item(const Params& p, const Sched& sc, int unit, int item, int rank, uint32_t tacc, Epi&) {
        const int2 u = pick(sc, unit);
        HeadDhT::Epi eh;
        HeadDwT::Epi ew;
        if (u.x == 1) HeadDwT::epi_item<kBf16>(p, sc.w, u.y, item, rank, tacc, ew);
        else HeadDhT::epi_item<kBf16>(p, sc.h, u.y, item, rank, tacc, eh);
    }
};
constexpr int kGradThreads = 64 + 32 * HeadGradsT::kEpiWarps;

template <bool kBf16>
__global__ void __launch_bounds__(kGradThreads, 1)
    head_grads_kernel(const __grid_constant__ HeadChunkParams p, const __grid_constant__ CUtensorMap mA,
                      const __grid_constant__ CUtensorMap mA2, const __grid_constant__ CUtensorMap mB) {
    tc_pair_body<HeadGradsT, kBf16>(p, mA, mA2, mB);
}

template <bool kBf16>
__global__ void __launch_bounds__(kGradThreads, 1)
    head_dh_kernel(const __grid_constant__ HeadChunkParams p, const __grid_constant__ CUtensorMap mA,
                   const __grid_constant__ CUtensorMap mA2, const __grid_constant__ CUtensorMap mB) {
    tc_pair_body<HeadDhT, kBf16>(p, mA, mA2, mB);
}

template <bool kBf16>
__global__ void __launch_bounds__(kGradThreads, 1)
    head_dh_wide_kernel(const __grid_constant__ HeadChunkParams p, const __grid_constant__ CUtensorMap mA,
                        const __grid_constant__ CUtensorMap mA2, const __grid_constant__ CUtensorMap mB) {
    tc_pair_body<HeadDhWideT, kBf16>(p, mA, mA2, mB);
}

template <bool kBf16>
__global__ void __launch_bounds__(kGradThreads, 1)
    head_dw_kernel(const __grid_constant__ HeadChunkParams p, const __grid_constant__ CUtensorMap mA,
                   const __grid_constant__ CUtensorMap mA2, const __grid_constant__ CUtensorMap mB) {
    tc_pair_body<HeadDwT, kBf16>(p, mA, mA2, mB);
}

}  // namespace

cudaError_t launch_head_logits(const LogitsParams& p, const CUtensorMap& mH, const CUtensorMap& mW, int n_sm, bool bf16,
                               int mode, cudaStream_t st) {
    switch (mode) {
        case LG_KEEP_TOKEN: return launch_pairs<head_logits_kernel<true, LG_KEEP_TOKEN>>(kHeadThreads, kLgSmem, n_sm, st, p, mH, mW);
        case LG_KEEP_MAX:
            return bf16 ? launch_pairs<head_logits_kernel<true, LG_KEEP_MAX>>(kHeadThreads, kLgSmem, n_sm, st, p, mH, mW)
                        : launch_pairs<head_logits_kernel<false, LG_KEEP_MAX>>(kHeadThreads, kLgSmem, n_sm, st, p, mH, mW);
        case LG_ENTROPY:
            return bf16 ? launch_pairs<head_logits_kernel<true, LG_ENTROPY>>(kHeadThreads, kLgSmem, n_sm, st, p, mH, mW)
                        : launch_pairs<head_logits_kernel<false, LG_ENTROPY>>(kHeadThreads, kLgSmem, n_sm, st, p, mH, mW);
        default:
            return bf16 ? launch_pairs<head_logits_kernel<true, LG_STATS>>(kHeadThreads, kLgSmem, n_sm, st, p, mH, mW)
                        : launch_pairs<head_logits_kernel<false, LG_STATS>>(kHeadThreads, kLgSmem, n_sm, st, p, mH, mW);
    }
}

cudaError_t launch_head_grads(const HeadChunkParams& p, const CUtensorMap& mDS, const CUtensorMap& mDSmn,
                              const CUtensorMap& mWmn, int n_sm, bool bf16, cudaStream_t st) {
    constexpr int smem = smem_bytes<HeadGradsT>();
    return bf16 ? launch_pairs<head_grads_kernel<true>>(kGradThreads, smem, n_sm, st, p, mDS, mDSmn, mWmn)
                : launch_pairs<head_grads_kernel<false>>(kGradThreads, smem, n_sm, st, p, mDS, mDSmn, mWmn);
}

cudaError_t launch_head_dh(const HeadChunkParams& p, const CUtensorMap& mDS, const CUtensorMap& mWmn, int n_sm, bool bf16,
                           cudaStream_t st) {
    if (p.dh_cols == 2 * kBN) {
        constexpr int smem = smem_bytes<HeadDhWideT>();
        return bf16 ? launch_pairs<head_dh_wide_kernel<true>>(kGradThreads, smem, n_sm, st, p, mDS, mDS, mWmn)
                    : launch_pairs<head_dh_wide_kernel<false>>(kGradThreads, smem, n_sm, st, p, mDS, mDS, mWmn);
    }
    constexpr int smem = smem_bytes<HeadDhT>();
    return bf16 ? launch_pairs<head_dh_kernel<true>>(kGradThreads, smem, n_sm, st, p, mDS, mDS, mWmn)
                : launch_pairs<head_dh_kernel<false>>(kGradThreads, smem, n_sm, st, p, mDS, mDS, mWmn);
}

cudaError_t launch_head_dw(const HeadChunkParams& p, const CUtensorMap& mDSmn, int n_sm, bool bf16, cudaStream_t st) {
    constexpr int smem = smem_bytes<HeadDwT>();
    return bf16 ? launch_pairs<head_dw_kernel<true>>(kGradThreads, smem, n_sm, st, p, mDSmn, mDSmn, p.mHct)
                : launch_pairs<head_dw_kernel<false>>(kGradThreads, smem, n_sm, st, p, mDSmn, mDSmn, p.mHct);
}

template <bool kBf16, int kNC>
static cudaError_t launch_few_t(const FewParams& p, const CUtensorMap& mH, const CUtensorMap& mW, int grid, cudaStream_t st) {
    static std::atomic<int> known[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices || !known[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(head_few_kernel<kBf16, kNC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 FewShape<kNC>::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < kDevices) known[dev].store(1, std::memory_order_release);
    }
    // starts while k_few_prep runs (see chain_wait in the kernel): 2 us of 88 at 8 rows of a 152K vocabulary.
    // The chunked operators' kernels are not chained this way: their waiting blocks cost more
    // than the launches they hide (88 us instead of 53 for the smallest clipped-loss step).
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = FewShape<kNC>::kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, head_few_kernel<kBf16, kNC>, p, mH, mW);
}

cudaError_t launch_few(const FewParams& p, const CUtensorMap& mH, const CUtensorMap& mW, int grid, bool bf16, int nc,
                       cudaStream_t st) {
    if (nc <= 16)
        return bf16 ? launch_few_t<true, 16>(p, mH, mW, grid, st) : launch_few_t<false, 16>(p, mH, mW, grid, st);
    return bf16 ? launch_few_t<true, 32>(p, mH, mW, grid, st) : launch_few_t<false, 32>(p, mH, mW, grid, st);
}

}  // namespace grpo
