// The gradient of the norm before the head (norm_abi.cu has the entry point, norm_plan.cu
// deals the rows).  With rstd = 1 / sqrt(mean s^2 + eps):
//   dx = rstd dy w - s rstd^3 mean(dy w s) + dsum;  dw = the sum over the rows of dy s rstd
// Both means come from one pass over the row, so nothing of the forward pass has to be
// kept but s.  12 operations an element against 5 to 8 bytes: HBM bounds it, with
// instructions close behind (the codes of a checkpoint take 5 an element).  dw is
// summed in registers from row to row, then over the blocks in a fixed order.
// Measured: 160,000 x 4096 from a checkpoint, 54% of the rows: 372 us, 6.4 TB/s (a copy reaches 6.8);
// 40,000 x 4096 from 16 bits 149 us, with dsum 191 us (6.6 and 6.9 TB/s); 8192 x 1536, 60% of the rows,
// with dsum: 18 us, or 14.9 where the inputs stay in L2, and there 12.6 without dw (its parts and their sum).
#include "norm_device.cuh"

namespace grpo {

namespace {

constexpr int kBwdRegs = 80, kBwdRegsTwo = 128;      // of a thread with one or two units: 768 or 512 threads an SM
constexpr int kRowsRegs = 96;          // 640 threads an SM; with dsum 48 to 72 bytes a thread are spilled for it
constexpr int kStagesMax = 2;          // more gain nothing: what is under way is limited by the number of blocks
constexpr int kSmemSm = 226 * 1024;    // of an SM's 228 KB
constexpr int kSmemBlock = 2048;       // what a block takes of it beside the ring and the weight, and more

// Both sums over a row's threads, in a fixed order; every thread gets them.
__device__ __forceinline__ float2 warp_sums(float a, float b, int width) {
    for (int o = width / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return make_float2(a, b);
}

// Here the lower lanes of a warp join a, the upper ones b.  The warps leave theirs in s, of which the next row takes
// the other half, so that one barrier is enough; entries of warps that are not there hold 0.
// From a checkpoint without dsum (kEither) a row may have two units a thread or one, as the number of rows has it.  Its
// gradient is not to depend on that, so both add the same numbers in the same order:
//   two:  units half a row apart in the thread; lanes 16, 1, 2, 4 and 8 apart; the warps in turn
//   one:  those are lanes 16 apart, and 16 units lanes 8 (see one_as_two); lanes 1, 2 and 4 apart; two warps, 8 units
//         apart; these pairs in turn
template <int kUpt, bool kEither>
__device__ __forceinline__ float2 block_sums(float a, float b, float* s) {
    const bool upper = threadIdx.x & 16;
    float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v += __shfl_xor_sync(0xffffffffu, v, !kEither ? 8 >> i : kUpt == 2 ? 1 << i : i == 0 ? 8 : 1 << (i - 1));
    if ((threadIdx.x & 15) == 0) s[threadIdx.x >> 4] = v;
    __syncthreads();
    F2 sum = 0;
    for (unsigned i = 0; i < blockDim.x; i += 64) {
        const float4 x = *reinterpret_cast<const float4*>(s + i / 16);
        if (kEither && kUpt == 1)
            sum = f2_add(sum, f2_add(f2(x.x, x.y), f2(x.z, x.w)));
        else
            sum = f2_add(f2_add(sum, f2(x.x, x.y)), f2(x.z, x.w));
    }
    return f2_values(sum);
}

// The unit of a thread that has one, dealt as above: 8 lanes have 8 units that lie together.
__device__ __forceinline__ int one_as_two(int lane, int n_unit) {
    return (lane >> 6) * 32 + (lane >> 3 & 1) * 16 + (lane >> 5 & 1) * 8 + (lane & 7) + (lane >> 4 & 1) * (n_unit / 2);
}

// A unit's part of both sums: s^2, and s (dy w).
template <bool kBf16>
__device__ __forceinline__ float2 unit_sums(const Unit& s, const Unit& dy, const Unit32& w) {
    const Unit32 v = values<kBf16>(s), g = values<kBf16>(dy);
    F2 a = 0, b = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        a = f2_fma(v.p[j], v.p[j], a);
        b = f2_fma(v.p[j], f2_mul(g.p[j], w.p[j]), b);
    }
    return make_float2(sum_of(a), sum_of(b));
}

// dx = rstd dy w - s rstd^3 mean(dy w s) + dsum of a unit, and its dy s rstd added to acc.  c2: the factor of s.
template <bool kBf16, bool kDsum>
__device__ __forceinline__ Unit unit_grad(Unit s, Unit dy, const Unit& ds, const Unit32& w, F2 rstd2, F2 c2, F2 (&acc)[8]) {
    forget_values(&s);
    forget_values(&dy);
    const Unit32 v = values<kBf16>(s);
    Unit32 g = values<kBf16>(dy), x = {};
    if (kDsum) x = values<kBf16>(ds);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        g.p[j] = f2_mul(g.p[j], rstd2);
        acc[j] = f2_fma(g.p[j], v.p[j], acc[j]);
        x.p[j] = kDsum ? f2_fma(g.p[j], w.p[j], x.p[j]) : f2_mul(g.p[j], w.p[j]);
        x.p[j] = f2_fma(v.p[j], c2, x.p[j]);
    }
    return rounded<kBf16>(x);
}

// What found_inf says; the larger one, where it could say both.
constexpr int kNotFiniteValue = 1, kWaitRanOut = 2;

// A pair that turns NaN with the first value that is not finite.
template <bool kBf16>
__device__ __forceinline__ uint32_t mark_bad(uint32_t bad, const Unit& x) {
#pragma unroll
    for (int j = 0; j < 8; ++j) bad = pair_fma<kBf16>(x.w[j], 0u, bad);
    return bad;
}
template <bool kBf16>
__device__ __forceinline__ bool is_bad(uint32_t bad) {
    const float2 v = pair_values<kBf16>(bad);
    return !(v.x == 0.f && v.y == 0.f);
}

// Writes dw of column j; true if it is not finite.
template <bool kBf16>
__device__ __forceinline__ bool store_dweight(const NormParams& p, int j, float v) {
    if (p.weight_f32) {
        static_cast<float*>(p.dweight)[j] = v;
    } else {
        const uint32_t r = pair_bits<kBf16>(v, 0.f);
        static_cast<uint16_t*>(p.dweight)[j] = static_cast<uint16_t>(r);
        v = pair_values<kBf16>(r).x;
    }
    return !(fabsf(v) <= FLT_MAX);
}

// dw and found_inf from the parts of one cluster's blocks, which is the whole grid.
template <bool kBf16>
__device__ __forceinline__ void join_cluster(const NormParams& p) {
    cluster_sync();
    int bad = 0;
    if (blockIdx.x == 0 && threadIdx.x < gridDim.x) bad = p.bad[threadIdx.x];
    if (p.dweight)
        for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < p.d; j += gridDim.x * blockDim.x) {
            float v = 0.f;
            for (unsigned b = 0; b < gridDim.x; ++b) v += p.part[static_cast<int64_t>(b) * p.d + j];
            if (store_dweight<kBf16>(p, j, v)) bad = max(bad, kNotFiniteValue);
        }
    if (bad) atomicMax(p.found_inf, bad);  // 0 before, in block 0
}

__device__ __forceinline__ void bulk_load(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(to)),
                 "l"(from), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Rows of more than 512 columns: a block takes a row at a time, and copies the rows to
// come into a ring of p.stages stages in shared memory, one bulk copy a matrix: loads
// into registers took 16 to 24 of them, and so fewer rows an SM (475 us with two rows of 4096, 408 with three).
// Block b leaves its sum of dy s rstd of every column in part[b].
// A wait that runs out of time leaves garbage in its row; the block goes on, and found_inf says so (2).
template <bool kBf16, int kSrc, int kUpt, bool kDsum>
__global__ void __maxnreg__(kUpt == 1 ? kBwdRegs : kBwdRegsTwo) k_norm_bwd_wide(const NormParams p) {
    __shared__ alignas(16) float s_join[2][kBlockMax / 16];
    __shared__ uint64_t s_full[kStagesMax];
    __shared__ int s_abort;
    extern __shared__ float4 s_weight[];
    const int n_unit = p.d / kUnit, width = static_cast<int>(blockDim.x), pad = width * kUpt;
    constexpr bool kEither = kSrc == kCkpt && !kDsum;
    const int lane = static_cast<int>(threadIdx.x);
    const int unit0 = kUpt == 1 && kEither && n_unit % 64 == 0 ? one_as_two(lane, n_unit) : lane;      // the thread's first unit
    const uint32_t N = static_cast<uint32_t>(p.N), step = gridDim.x;      // N < 2^31
    const float inv_d = 1.f / p.d;
    chain_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.found_inf = 0;

    // a stage: dy, x or the codes, dsum
    constexpr int kSrcBytes = kSrc == kCkpt ? 1 : 2;
    const uint32_t matrix = pad * kUnit * 2, stage = matrix / 2 * (2 + kSrcBytes + (kDsum ? 2 : 0));
    char* ring = reinterpret_cast<char*>(s_weight + 4 * pad);
    auto copy_row = [&](int64_t at, int q) {                              // one thread
        char* to = ring + q * stage;
        mbar_arrive_expect_tx(&s_full[q], p.d * (2 + kSrcBytes + (kDsum ? 2 : 0)));
        bulk_load(to, p.dy + at, p.d * 2, &s_full[q]);
        if (kSrc == kCkpt)
            bulk_load(to + matrix, p.codes + at, p.d, &s_full[q]);
        else
            bulk_load(to + matrix, p.x + at, p.d * 2, &s_full[q]);
        if (kDsum) bulk_load(to + matrix + matrix / 2 * kSrcBytes, p.dsum + at, p.d * 2, &s_full[q]);
    };
    uint32_t t = blockIdx.x;
    int64_t at = static_cast<int64_t>(t) * p.d;
    const int64_t at_step = static_cast<int64_t>(step) * p.d;
    Ahead ahead;
    ahead.begin(p, t, step, 32);
    uint32_t alive = ahead.bits(32);           // bit q: row t + q step counts
    if (threadIdx.x == 0) {
        for (int q = 0; q < p.stages; ++q) mbar_init(&s_full[q], 1);
        s_abort = 0;
        fence_barrier_init();
        for (int q = 0; q < p.stages; ++q)
            if (alive >> q & 1) copy_row(at + q * at_step, q);
    }
    uint32_t scale[kUpt] = {};                 // (checkpoint) of the next row
    auto load_scales = [&](int64_t at, bool on) {
#pragma unroll
        for (int k = 0; k < (kSrc == kCkpt ? kUpt : 0); ++k) {
            const int i = unit0 + k * width;
            scale[k] = load_scale(p.scales + at / kCkptBlock + i / (kCkptBlock / kUnit), on && i < n_unit);
        }
    };
    load_scales(at, alive & 1);
    F2 acc[kUpt][8];
#pragma unroll
    for (int k = 0; k < kUpt; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[k][j] = 0;
    uint32_t bad = 0, phase = 0;
    stage_weight<kBf16>(p, s_weight, pad);
    for (int i = lane; i < 2 * kBlockMax / 16; i += width) s_join[0][i] = 0.f;     // a block may be one warp
    __syncthreads();
    int q = 0, turn = 0;
    for (; t < N; t += step, at += at_step) {
        const bool live = alive & 1, far = alive >> p.stages & 1;
        ahead.advance(p, t, step, 32);
        alive = ahead.bits(32);
        Unit s[kUpt], dy[kUpt], ds[kDsum ? kUpt : 1];
        float2 sums = make_float2(0.f, 0.f);
        if (live) {
            mbar_wait(&s_full[q], phase >> q & 1, &s_abort, nullptr);
            phase ^= 1u << q;
            const uint32_t from = smem_u32(ring) + q * stage;
#pragma unroll
            for (int k = 0; k < kUpt; ++k) {
                const uint32_t i = unit0 + k * width;
                dy[k] = read_unit(from + i * (kUnit * 2));
                if (kSrc == kCkpt)
                    s[k] = decode<kBf16>(read16(from + matrix + i * kUnit), bf16_value(scale[k]));
                else
                    s[k] = read_unit(from + matrix + i * (kUnit * 2));
                if (kDsum) ds[k] = read_unit(from + matrix + matrix / 2 * kSrcBytes + i * (kUnit * 2));
            }
        }
        load_scales(at + at_step, alive & 1);
        if (live) {
#pragma unroll
            for (int k = 0; k < kUpt; ++k) {
                const float2 u = unit_sums<kBf16>(s[k], dy[k], staged_weight(s_weight, pad, unit0 + k * width));
                if (unit0 + k * width < n_unit) sums = make_float2(sums.x + u.x, sums.y + u.y);
            }
            sums = block_sums<kUpt, kEither>(sums.x, sums.y, s_join[turn]);
            turn ^= 1;
        }
        // the whole block has read stage q: of this row above, or of the last one that was in it
        if (threadIdx.x == 0 && far && !s_abort) copy_row(at + p.stages * at_step, q);
        q = q + 1 == p.stages ? 0 : q + 1;
        const float rstd = rsqrtf(sums.x * inv_d + p.eps);
        const float c = -(rstd * rstd) * (sums.y * inv_d) * rstd;
        const F2 rstd2 = f2(rstd, rstd), c2 = f2(c, c);
#pragma unroll
        for (int k = 0; k < kUpt; ++k) {
            const int i = unit0 + k * width;
            Unit out = {};
            if (live)
                out = unit_grad<kBf16, kDsum>(s[k], dy[k], ds[kDsum ? k : 0], staged_weight(s_weight, pad, i), rstd2, c2, acc[k]);
            if (i < n_unit) {
                bad = mark_bad<kBf16>(bad, out);
                store_unit(p.dx + at + i * kUnit, out);
            }
        }
    }

    chain_next();
    const int any = __syncthreads_or(is_bad<kBf16>(bad));
    abort_grace(&s_abort);
    if (threadIdx.x == 0) p.bad[blockIdx.x] = s_abort ? kWaitRanOut : any ? kNotFiniteValue : 0;
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.d;
#pragma unroll
    for (int k = 0; k < kUpt; ++k) {
        const int i = unit0 + k * width;
        if (i >= n_unit || !p.dweight) break;
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 v = f2_values(acc[k][j]);
            w[2 * j] = __float_as_uint(v.x);
            w[2 * j + 1] = __float_as_uint(v.y);
        }
        st_global_v8(part + i * kUnit, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
        st_global_v8(part + i * kUnit + 8, w[8], w[9], w[10], w[11], w[12], w[13], w[14], w[15]);
    }
    if (p.joined) join_cluster<kBf16>(p);
}

// Rows of up to 512 columns: 4, 8, 16 or 32 lanes of a warp take a row at a time, a unit each; the next
// row's loads are under way while one is worked on.
template <bool kBf16, int kSrc, bool kDsum>
__global__ void __maxnreg__(kRowsRegs) k_norm_bwd_rows(const NormParams p) {
    extern __shared__ float4 s_weight[];       // and at the end the warps' sums of dw
    const int n_unit = p.d / kUnit, width = p.width, pad = width;
    const int lane = static_cast<int>(threadIdx.x) & (width - 1);
    const uint32_t rows = kWarpThreads / width, mine = threadIdx.x / width;        // rows that a block works on at once
    const uint32_t step = gridDim.x * rows, N = static_cast<uint32_t>(p.N);
    const float inv_d = 1.f / p.d;
    chain_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.found_inf = 0;

    F2 acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0;
    uint32_t bad = 0;
    Raw<kSrc, 1> raw;
    Unit raw_dy, raw_ds;
    uint32_t t = blockIdx.x * rows + mine;
    int64_t at = static_cast<int64_t>(t) * p.d + lane * kUnit;         // the thread's first element of row t
    const int64_t at_step = static_cast<int64_t>(step) * p.d;
    auto load = [&](int64_t at, bool on) {
        load_row<kSrc, 1, false>(p, at, on, lane, width, n_unit, &raw);
        raw_dy = load_unit(p.dy + at, on && lane < n_unit);
        if (kDsum) raw_ds = load_unit(p.dsum + at, on && lane < n_unit);
    };
    Ahead ahead;
    ahead.begin(p, t, step, width);
    uint32_t alive = ahead.bits(width);        // bit q: row t + q step counts
    load(at, alive & 1);
    stage_weight<kBf16>(p, s_weight, pad);
    __syncthreads();
    for (uint32_t base = blockIdx.x * rows; base < N; base += step, t += step, at += at_step) {   // whole blocks go round together
        const bool live = alive & 1, next = alive >> 1 & 1;
        ahead.advance(p, t, step, width);
        alive = ahead.bits(width);
        const Unit s = stream_of<kBf16>(raw, 0), dy = raw_dy;
        Unit ds;
        if (kDsum) ds = raw_ds;
        load(at + at_step, next);
        float2 sums = unit_sums<kBf16>(s, dy, staged_weight(s_weight, pad, lane));
        sums = warp_sums(sums.x, sums.y, width);
        const float rstd = rsqrtf(sums.x * inv_d + p.eps);
        const float c = -(rstd * rstd) * (sums.y * inv_d) * rstd;
        const F2 rstd2 = f2(rstd, rstd), c2 = f2(c, c);
        Unit out = unit_grad<kBf16, kDsum>(s, dy, ds, staged_weight(s_weight, pad, lane), rstd2, c2, acc);
        if (!live) out = Unit{};                         // not 0 times a weight that is not finite
        if (t < N && lane < n_unit) {
            bad = mark_bad<kBf16>(bad, out);
            store_unit(p.dx + at, out);
        }
    }

    chain_next();
    const int any = __syncthreads_or(is_bad<kBf16>(bad));
    if (threadIdx.x == 0) p.bad[blockIdx.x] = any ? kNotFiniteValue : 0;
    // the rows of a warp, then the warps of the block, in this order; in the weight's place
    float* s_dw = reinterpret_cast<float*>(s_weight);
    const int warp = threadIdx.x >> 5, wide = pad * kUnit;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float2 v = f2_values(acc[j]);
        for (int o = width; o < 32; o <<= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        // the pairs of a unit lie pad pairs apart: neighbouring lanes write neighbouring pairs
        if ((threadIdx.x & 31) < width) *reinterpret_cast<float2*>(s_dw + warp * wide + (j * pad + lane) * 2) = v;
    }
    __syncthreads();
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.d;
    for (int j = threadIdx.x; j < p.d / 2 && p.dweight; j += kWarpThreads) {       // pair j % 8 of unit j / 8
        F2 v = 0;
        for (int w = 0; w < kWarpThreads / 32; ++w)
            v = f2_add(v, *reinterpret_cast<const F2*>(s_dw + w * wide + ((j & 7) * pad + (j >> 3)) * 2));
        *reinterpret_cast<F2*>(part + 2 * j) = v;
    }
    if (p.joined) join_cluster<kBf16>(p);
}

// dw and found_inf from the parts.  A block takes 16 columns, and every thread each `slots`-th part of one.
constexpr int kJoinCols = 16, kJoinThreads = 1024;

template <bool kBf16>
__global__ void __launch_bounds__(kJoinThreads) k_norm_join(const NormParams p) {
    __shared__ float s_part[kJoinThreads / kJoinCols][kJoinCols + 1];
    const int slots = static_cast<int>(blockDim.x) / kJoinCols, lane = threadIdx.x & 31;
    const int slot = threadIdx.x / kJoinCols, col = threadIdx.x % kJoinCols;
    int bad = 0;
    chain_wait();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.parts; b += blockDim.x) bad = max(bad, p.bad[b]);
    if (p.dweight) {
        const float* part = p.part + blockIdx.x * kJoinCols + col;
        float v = 0.f;
#pragma unroll 8
        for (int b = slot; b < p.parts; b += slots) v += part[static_cast<int64_t>(b) * p.d];
        s_part[slot][col] = v;
        __syncthreads();
        const int j = threadIdx.x >> 5;            // a warp for each column
        if (j < kJoinCols) {
            v = 0.f;
            for (int i = lane; i < slots; i += 32) v += s_part[i][j];
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0 && store_dweight<kBf16>(p, blockIdx.x * kJoinCols + j, v)) bad = max(bad, kNotFiniteValue);
        }
    }
    if (bad) atomicMax(p.found_inf, bad);  // 0 before: the kernel that left the parts
}

template <bool kBf16, int kSrc, bool kDsum>
cudaError_t bwd_of(const NormParams& p, const NormPlan& o, cudaStream_t st) {
    const size_t weight = static_cast<size_t>(o.width) * o.upt * kUnit * 4;
    if (!o.wide)                               // 8 KB at most: d <= 512
        return launch_chained(k_norm_bwd_rows<kBf16, kSrc, kDsum>, o.grid, o.threads, weight * (kWarpThreads / 32), p, st,
                              o.joined ? o.grid : 1);
    const auto f = o.upt == 1 ? k_norm_bwd_wide<kBf16, kSrc, 1, kDsum> : k_norm_bwd_wide<kBf16, kSrc, 2, kDsum>;
    const size_t stage = weight / 4 * (2 + (kSrc == kCkpt ? 1 : 2) + (kDsum ? 2 : 0));
    NormParams r = p;
    const size_t room = static_cast<size_t>(kSmemSm) / o.per_sm - kSmemBlock;
    if (room < weight + stage) return cudaErrorInvalidConfiguration;
    r.stages = static_cast<int>((room - weight) / stage);
    if (r.stages > kStagesMax) r.stages = kStagesMax;
    const size_t smem = weight + r.stages * stage;
    static MostSmem most[2];
    const cudaError_t e = most[o.upt - 1].allow(f, kSmemSm - kSmemBlock);
    if (e != cudaSuccess) return e;
    return launch_chained(f, o.grid, o.threads, smem, r, st, o.joined ? o.grid : 1);
}

template <bool kBf16, int kSrc>
cudaError_t bwd_as(const NormParams& p, const NormPlan& o, cudaStream_t st) {
    return p.dsum ? bwd_of<kBf16, kSrc, true>(p, o, st) : bwd_of<kBf16, kSrc, false>(p, o, st);
}

}  // namespace

cudaError_t launch_norm_bwd(const NormParams& p, const NormPlan& o, bool bf16, cudaStream_t st) {
    if (p.codes) return bf16 ? bwd_as<true, kCkpt>(p, o, st) : bwd_as<false, kCkpt>(p, o, st);
    return bf16 ? bwd_as<true, kX>(p, o, st) : bwd_as<false, kX>(p, o, st);
}

cudaError_t launch_norm_join(const NormParams& p, bool bf16, cudaStream_t st) {
    // 32 or 64 slots, us of the whole gradient: 456 parts of 4096 columns (2000 rows) 14.4 and 14.3, 304 of 5120 15.9 and
    // 18.1, 608 of 2048 9.9 and 9.4, 1216 of 1024 9.7 and 8.2.  Parts are not all of it: up to 4864 columns the blocks of 64
    // slots are on the SMs at once, and few parts of few columns would gain as well (200 of 1024 6.0 and 5.3)
    const int threads = p.parts > 512 ? kJoinThreads : kJoinThreads / 2;
    return launch_chained(bf16 ? k_norm_join<true> : k_norm_join<false>, p.dweight ? p.d / kJoinCols : 1, threads, 0, p, st);
}

}  // namespace grpo
