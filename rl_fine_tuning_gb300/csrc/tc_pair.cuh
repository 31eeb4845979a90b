// The parts that the tensor-core translation units share: shared-memory and
// barrier layout, packing, the CTA-pair engine (tcgen05.mma.cta_group::2, fed
// by TMA) and its 16-bit dH and dW traits, and the persistent launch.
#pragma once
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace grpo {

constexpr int kThreads = 192;
constexpr int kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

// Operand layouts in shared memory (all 128-byte swizzled, as TMA writes them
// with CU_TENSOR_MAP_SWIZZLE_128B):
//   K-major  [rows][64 K-elements]: row r at r*128 B; 8-row groups 1024 B apart
//            (SBO = 1024).  K sub-step kk (16 elements) = +32 B.
//   MN-major [64 K-rows][64 MN-elements] boxes of 8 KB; box j holds MN
//            elements 64j..64j+63 (LBO = 8192); 8-K-row groups 1024 B apart
//            (SBO = 1024).  K sub-step kk = +2048 B.
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t a) { return make_sdesc_sw128(a, 16, 1024); }
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t a) { return make_sdesc_sw128(a, 8192, 1024); }

constexpr int kUnitSlots = 4;   // work units published ahead by the producer

struct Smem {
    uint8_t* stages;
    uint64_t* full;
    uint64_t* empty;
    uint64_t* acc_full;
    uint64_t* acc_empty;
    uint64_t* drain;
    uint64_t* unit_full;
    uint64_t* unit_empty;
    uint32_t* tmem_slot;
    volatile int* abort_flag;
    volatile int* unit_id;
    // [0] K-stages whose TMA loads this CTA's producer issued, [1] K-stages the
    // MMA lane consumed, [2] 1 once every issued load is known to have landed
    volatile int* ld_count;
};

template <int kStages, int kStageBytes>
__device__ __forceinline__ Smem carve_smem(uint8_t* raw) {
    Smem s;
    const uint32_t a = smem_u32(raw);
    uint8_t* base = raw + ((1024u - (a & 1023u)) & 1023u);
    s.stages = base;
    s.full = reinterpret_cast<uint64_t*>(base + kStages * kStageBytes);
    s.empty = s.full + kStages;
    s.acc_full = s.empty + kStages;
    s.acc_empty = s.acc_full + 2;
    s.drain = s.acc_empty + 2;
    s.unit_full = s.drain + 1;
    s.unit_empty = s.unit_full + kUnitSlots;
    s.tmem_slot = reinterpret_cast<uint32_t*>(s.unit_empty + kUnitSlots);
    s.abort_flag = reinterpret_cast<volatile int*>(s.tmem_slot + 1);
    s.unit_id = s.abort_flag + 1;
    s.ld_count = s.unit_id + kUnitSlots;
    return s;
}

template <class T>
constexpr int smem_bytes() {
    return T::kStages * T::kStageBytes + 1024 + 512;
}

// After an abort, wait (at most kInflightNs in all) for the K-stages whose loads
// were issued but not consumed, phases used .. issued-1 of the full barriers,
// to complete.  Returns true when all of them did.
constexpr unsigned long long kInflightNs = 2ull * 1000ull * 1000ull;   // 2 ms

template <int kStages>
__device__ __forceinline__ bool wait_inflight(uint64_t* full, int used, int issued) {
    const uint64_t t0 = globaltimer();
    for (int i = used; i < issued; ++i) {
        const uint32_t a = smem_u32(&full[i % kStages]);
        const uint32_t parity = static_cast<uint32_t>(i / kStages) & 1u;
        while (!mbar_try_wait(a, parity))
            if (globaltimer() - t0 > kInflightNs) return false;
    }
    return true;
}

__device__ __forceinline__ uint16_t f32_to_16(float x, bool bf16) {
    if (bf16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    return __half_as_ushort(__float2half_rn(x));
}

__device__ __forceinline__ uint32_t pack2(float a, float b, bool bf16) {
    return static_cast<uint32_t>(f32_to_16(a, bf16)) | (static_cast<uint32_t>(f32_to_16(b, bf16)) << 16);
}

// non-finite check of a packed pair of fp16 values (exponent all ones)
__device__ __forceinline__ bool half2_nonfinite(uint32_t u) {
    return ((u & 0x7C00u) == 0x7C00u) || ((u & 0x7C000000u) == 0x7C000000u);
}

// chunk bookkeeping shared by the backward kernels
struct ChunkSched {
    int n_units, ks, c0, n_c, n_mt, n_nt, n_g, C;
    float winv;
};

__device__ __forceinline__ bool chunk_setup(const ChunkParams& p, ChunkSched& sc, int C) {
    if (p.chunk >= p.counts[C_NCHUNKS]) return false;
    sc.C = C;
    if (p.cb) {
        sc.c0 = p.cb[p.chunk];
        sc.n_c = p.cb[p.chunk + 1] - sc.c0;
        sc.winv = p.oscale[p.chunk];
    } else {
        const int rc = p.counts[C_CHUNK_ROWS];
        sc.c0 = p.chunk * rc;
        sc.n_c = min(rc, p.counts[C_NVALID] - sc.c0);
        sc.winv = __int_as_float(p.counts[C_WINV]);
    }
    sc.n_mt = (sc.n_c + kBM - 1) / kBM;
    return sc.n_c > 0;
}

// ====================================================================== CTA-pair kernels
// The same stages on pairs of SMs with M=256 tcgen05 MMAs (cta_group::2): each
// CTA of a pair holds its own 128-row A tile and half of the 256-column B
// tile, so per SM a K-stage is 32 KB of shared memory instead of 48-64 KB, and
// its tensor memory holds a double-buffered 128x256 accumulator.

// Work-unit orders.  A unit is a pair (a, b); the a-indices are visited in
// groups of G: all b of a group run before the next group starts, and within a
// group the a-indices are fastest.  With G = 1 the b-index is fastest.  The
// group sizes were chosen by timing on GB300 (19 row tiles per group for the
// chunk forward: each W tile is then shared in L2 by 19 tiles).
constexpr int kFwdGroup = 19;   // chunk forward: a = 128-row tile, b = vocabulary split (19 divides 38 and 76)
constexpr int kDhGroup = 1;     // dH: a = pair of 128-row tiles, b = 256-wide d tile
constexpr int kDwGroup = 1;     // dW: a = pair of 128-row vocabulary tiles, b = 256-wide d tile

__device__ __forceinline__ void decode_grouped(int unit, int n_a, int n_b, int G, int* a, int* b) {
    const int full = (n_a / G) * G;
    if (unit < full * n_b) {
        const int gi = unit / (G * n_b);
        const int r = unit - gi * G * n_b;
        *b = r / G;
        *a = gi * G + (r - *b * G);
    } else {
        const int u2 = unit - full * n_b;
        const int g_last = n_a - full;
        *b = u2 / g_last;
        *a = full + (u2 - *b * g_last);
    }
}

struct DhPairT {
    static constexpr int kStages = 7;
    static constexpr int kStageBytes = 16384 + 16384;   // A (128 slots x 64 vocab), B half (64 vocab x 128 d)
    using Params = ChunkParams;
    using Sched = ChunkSched;
    struct Coord {
        int m0, n0;
    };
    struct Epi {
        int unused;
    };
    // unit -> (pair of 128-row tiles, d tile); the CTA of rank r takes m-tile 2*pair + r
    __device__ static bool setup(const Params& p, Sched& sc) {
        if (!chunk_setup(p, sc, 2)) return false;
        sc.n_nt = (p.d + kBN - 1) / kBN;
        sc.n_g = (sc.n_mt + 1) / 2;
        sc.ks = (p.V + kBK - 1) / kBK;
        sc.n_units = sc.n_g * sc.n_nt;
        return true;
    }
    __device__ static void decode(const Sched& sc, int unit, int* pair, int* dt) {
        decode_grouped(unit, sc.n_g, sc.n_nt, kDhGroup, pair, dt);
    }
    __device__ static int mtile(const Sched& sc, int unit, int rank) {
        int pair, dt;
        decode(sc, unit, &pair, &dt);
        return pair * 2 + rank;
    }
    __device__ static int dtile(const Sched& sc, int unit) {
        int pair, dt;
        decode(sc, unit, &pair, &dt);
        return dt;
    }
    __device__ static int items(const Params&, const Sched&, int) { return 1; }
    __device__ static int ksteps(const Params&, const Sched& sc, int) { return sc.ks; }
    __device__ static Coord coord(const Params&, const Sched& sc, int unit, int, int rank) {
        return Coord{mtile(sc, unit, rank) * kBM, dtile(sc, unit) * kBN};
    }
    __device__ static uint32_t tx_bytes(const Params& p, const Sched&, const Coord& c) {
        return 2 * 16384 + 8192 * min(4, (p.d - c.n0) / 64);
    }
    __device__ static void load(const Params& p, const Sched&, const Coord& c, int k, uint8_t* st, uint32_t bar,
                                const CUtensorMap* mA, const CUtensorMap*, const CUtensorMap* mB, int rank) {
        tma_load_2d_pair(mA, bar, st, k * kBK, c.m0);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = c.n0 + rank * 128 + 64 * j;
            if (col < p.d) tma_load_2d_pair(mB, bar, st + 16384 + 8192 * j, col, k * kBK);
        }
    }
    template <bool kBf16>
    __device__ static void mma(uint32_t st, uint32_t acc, bool first) {
        constexpr uint32_t idesc = make_idesc_f16(256, 256, kBf16, false, true);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            umma_pair_f16(acc, desc_kmajor(st + kk * 32), desc_mnmajor(st + 16384 + kk * 2048), idesc,
                          (first && kk == 0) ? 0u : 1u);
    }
    __device__ static void epi_begin(const Params&, const Sched&, int, int, int, Epi&) {}
    template <bool kBf16>
    __device__ static void epi_item(const Params& p, const Sched& sc, int unit, int, int rank, uint32_t tacc, Epi&) {
        const int row = (threadIdx.x & 31) + 32 * ((threadIdx.x >> 5) & 3);
        const int slot = mtile(sc, unit, rank) * kBM + row;
        const int n0 = dtile(sc, unit) * kBN;
        bool valid = slot < sc.n_c;
        if (!__any_sync(0xffffffffu, valid)) return;
        const int t = valid ? p.rows[sc.c0 + slot] : 0;
        if (valid && !GRPO_DCHECK(t >= 0 && t < p.N, p.status)) valid = false;
        uint16_t* out = p.dH + static_cast<int64_t>(t) * p.d;
        bool bad = false;
#pragma unroll 1
        for (int c = 0; c < kBN / 32; ++c) {
            const int col0 = n0 + c * 32;
            if (col0 >= p.d) break;
            float v[32];
            tmem_ld32(tacc + c * 32, v);
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) pk[j / 2] = pack2(v[j] * sc.winv, v[j + 1] * sc.winv, kBf16);
            if (!kBf16) {
#pragma unroll
                for (int j = 0; j < 16; ++j) bad |= half2_nonfinite(pk[j]);
            }
            if (valid) {
                // 64 bytes of one dH row as two whole sectors (dH is 32-byte aligned, d a multiple of 64)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    st_global_v8(out + col0 + 16 * h, pk[8 * h], pk[8 * h + 1], pk[8 * h + 2], pk[8 * h + 3],
                                 pk[8 * h + 4], pk[8 * h + 5], pk[8 * h + 6], pk[8 * h + 7]);
            }
        }
        if (bad && valid) atomicOr(p.found_inf, 1);
    }
    __device__ static void epi_end(const Params&, const Sched&, int, Epi&) {}
};

// dH with 512-column units: one staged 128-row dlogits tile feeds two 256-wide
// d tiles (two M=256 MMAs per K sub-step into the two halves of tensor
// memory), so the dlogits are read half as often and W in half as many waves.
// Used where its units still divide evenly over the SM pairs.
struct DhPairWideT {
    static constexpr int kStages = 4;
    static constexpr int kStageBytes = 16384 + 2 * 16384;   // A (128 slots x 64 vocab), 2 x B half (64 vocab x 128 d)
    static constexpr bool kWideAcc = true;
    using Params = ChunkParams;
    using Sched = ChunkSched;
    struct Coord {
        int m0, n0;
    };
    struct Epi {
        int unused;
    };
    // unit -> (pair of 128-row tiles, 512-wide d tile); the CTA of rank r takes m-tile 2*pair + r
    __device__ static bool setup(const Params& p, Sched& sc) {
        if (!chunk_setup(p, sc, 2)) return false;
        sc.n_nt = (p.d + 2 * kBN - 1) / (2 * kBN);
        sc.n_g = (sc.n_mt + 1) / 2;
        sc.ks = (p.V + kBK - 1) / kBK;
        sc.n_units = sc.n_g * sc.n_nt;
        return true;
    }
    __device__ static int mtile(const Sched& sc, int unit, int rank) { return (unit / sc.n_nt) * 2 + rank; }
    __device__ static int dtile(const Sched& sc, int unit) { return unit % sc.n_nt; }
    __device__ static int items(const Params&, const Sched&, int) { return 1; }
    __device__ static int ksteps(const Params&, const Sched& sc, int) { return sc.ks; }
    __device__ static Coord coord(const Params&, const Sched& sc, int unit, int, int rank) {
        return Coord{mtile(sc, unit, rank) * kBM, dtile(sc, unit) * 2 * kBN};
    }
    __device__ static uint32_t tx_bytes(const Params& p, const Sched&, const Coord& c) {
        uint32_t b = 2 * 16384;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (c.n0 + h * kBN + r * 128 + 64 * j < p.d) b += 8192;
        return b;
    }
    __device__ static void load(const Params& p, const Sched&, const Coord& c, int k, uint8_t* st, uint32_t bar,
                                const CUtensorMap* mA, const CUtensorMap*, const CUtensorMap* mB, int rank) {
        tma_load_2d_pair(mA, bar, st, k * kBK, c.m0);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = c.n0 + h * kBN + rank * 128 + 64 * j;
                if (col < p.d) tma_load_2d_pair(mB, bar, st + 16384 + 16384 * h + 8192 * j, col, k * kBK);
            }
    }
    template <bool kBf16>
    __device__ static void mma(uint32_t st, uint32_t acc, bool first) {
        constexpr uint32_t idesc = make_idesc_f16(256, 256, kBf16, false, true);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const uint64_t a = desc_kmajor(st + kk * 32);
            const uint32_t accum = (first && kk == 0) ? 0u : 1u;
            umma_pair_f16(acc, a, desc_mnmajor(st + 16384 + kk * 2048), idesc, accum);
            umma_pair_f16(acc + 256, a, desc_mnmajor(st + 32768 + kk * 2048), idesc, accum);
        }
    }
    __device__ static void epi_begin(const Params&, const Sched&, int, int, int, Epi&) {}
    template <bool kBf16>
    __device__ static void epi_item(const Params& p, const Sched& sc, int unit, int, int rank, uint32_t tacc, Epi&) {
        const int row = (threadIdx.x & 31) + 32 * ((threadIdx.x >> 5) & 3);
        const int slot = mtile(sc, unit, rank) * kBM + row;
        const int n0 = dtile(sc, unit) * 2 * kBN;
        bool valid = slot < sc.n_c;
        if (!__any_sync(0xffffffffu, valid)) return;
        const int t = valid ? p.rows[sc.c0 + slot] : 0;
        if (valid && !GRPO_DCHECK(t >= 0 && t < p.N, p.status)) valid = false;
        uint16_t* out = p.dH + static_cast<int64_t>(t) * p.d;
        bool bad = false;
#pragma unroll 1
        for (int c = 0; c < 2 * kBN / 32; ++c) {
            const int col0 = n0 + c * 32;
            if (col0 >= p.d) break;
            float v[32];
            tmem_ld32(tacc + c * 32, v);
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) pk[j / 2] = pack2(v[j] * sc.winv, v[j + 1] * sc.winv, kBf16);
            if (!kBf16) {
#pragma unroll
                for (int j = 0; j < 16; ++j) bad |= half2_nonfinite(pk[j]);
            }
            if (valid) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    st_global_v8(out + col0 + 16 * h, pk[8 * h], pk[8 * h + 1], pk[8 * h + 2], pk[8 * h + 3],
                                 pk[8 * h + 4], pk[8 * h + 5], pk[8 * h + 6], pk[8 * h + 7]);
            }
        }
        if (bad && valid) atomicOr(p.found_inf, 1);
    }
    __device__ static void epi_end(const Params&, const Sched&, int, Epi&) {}
};

struct DwPairT {
    static constexpr int kStages = 7;
    static constexpr int kStageBytes = 16384 + 16384;   // A (64 slots x 128 vocab), B half (128 d x 64 slots)
    using Params = ChunkParams;
    using Sched = ChunkSched;
    struct Coord {
        int v0, n0;
    };
    struct Epi {
        int unused;
    };
    // unit -> (pair of vocabulary tiles, d tile); the CTA of rank r takes vocabulary tile 2*pair + r
    __device__ static bool setup(const Params& p, Sched& sc) {
        if (!chunk_setup(p, sc, 2)) return false;
        sc.n_nt = (p.d + kBN - 1) / kBN;
        sc.n_g = ((p.V + kBM - 1) / kBM + 1) / 2;
        sc.ks = (sc.n_c + kBK - 1) / kBK;
        sc.n_units = sc.n_g * sc.n_nt;
        return true;
    }
    __device__ static void decode(const Sched& sc, int unit, int* pair, int* dt) {
        decode_grouped(unit, sc.n_g, sc.n_nt, kDwGroup, pair, dt);
    }
    __device__ static int vtile(const Sched& sc, int unit, int rank) {
        int pair, dt;
        decode(sc, unit, &pair, &dt);
        return pair * 2 + rank;
    }
    __device__ static int dtile(const Sched& sc, int unit) {
        int pair, dt;
        decode(sc, unit, &pair, &dt);
        return dt;
    }
    __device__ static int items(const Params&, const Sched&, int) { return 1; }
    __device__ static int ksteps(const Params&, const Sched& sc, int) { return sc.ks; }
    __device__ static Coord coord(const Params&, const Sched& sc, int unit, int, int rank) {
        return Coord{vtile(sc, unit, rank) * kBM, dtile(sc, unit) * kBN};
    }
    __device__ static uint32_t tx_bytes(const Params& p, const Sched&, const Coord& c) {
        return 2 * 16384 + 16384 * min(2, (p.d - c.n0 + 127) / 128);
    }
    __device__ static void load(const Params& p, const Sched&, const Coord& c, int k, uint8_t* st, uint32_t bar,
                                const CUtensorMap* mA, const CUtensorMap*, const CUtensorMap* mB, int rank) {
        tma_load_2d_pair(mA, bar, st, c.v0, k * kBK);
        tma_load_2d_pair(mA, bar, st + 8192, c.v0 + 64, k * kBK);
        // B: 128 rows of the transposed compact h_pol (d) x 64 chunk slots (K), K-major
        const int col = c.n0 + rank * 128;
        if (col < p.d) tma_load_2d_pair(mB, bar, st + 16384, k * kBK, col);
    }
    template <bool kBf16>
    __device__ static void mma(uint32_t st, uint32_t acc, bool first) {
        constexpr uint32_t idesc = make_idesc_f16(256, 256, kBf16, true, false);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            umma_pair_f16(acc, desc_mnmajor(st + kk * 2048), desc_kmajor(st + 16384 + kk * 32), idesc,
                          (first && kk == 0) ? 0u : 1u);
    }
    __device__ static void epi_begin(const Params&, const Sched&, int, int, int, Epi&) {}
    template <bool kBf16>
    __device__ static void epi_item(const Params& p, const Sched& sc, int unit, int, int rank, uint32_t tacc, Epi&) {
        const int row = (threadIdx.x & 31) + 32 * ((threadIdx.x >> 5) & 3);
        const int v = vtile(sc, unit, rank) * kBM + row;
        const int n0 = dtile(sc, unit) * kBN;
        const bool valid = v < p.V;
        if (!__any_sync(0xffffffffu, valid)) return;
        const bool first_chunk = p.chunk == 0;
        float* out = p.dW + static_cast<int64_t>(valid ? v : 0) * p.d;
        bool bad = false;
#pragma unroll 1
        for (int c = 0; c < kBN / 32; ++c) {
            const int col0 = n0 + c * 32;
            if (col0 >= p.d) break;
            float x[32];
            tmem_ld32(tacc + c * 32, x);
            if (valid) {
                // 128 bytes of one dW row as four whole sectors (dW is 32-byte aligned)
                float* o = out + col0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float r[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) r[i] = x[8 * j + i] * sc.winv;
                    if (!first_chunk) {
                        float prev[8];
                        ld_global_v8(o + 8 * j, prev);
#pragma unroll
                        for (int i = 0; i < 8; ++i) r[i] += prev[i];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) bad |= !isfinite(r[i]);
                    st_global_v8(o + 8 * j, __float_as_uint(r[0]), __float_as_uint(r[1]), __float_as_uint(r[2]),
                                 __float_as_uint(r[3]), __float_as_uint(r[4]), __float_as_uint(r[5]),
                                 __float_as_uint(r[6]), __float_as_uint(r[7]));
                }
            }
        }
        if (bad) atomicOr(p.found_inf, 1);
    }
    __device__ static void epi_end(const Params&, const Sched&, int, Epi&) {}
};

// Accumulators of the pair engine: by default two 256-column buffers in tensor
// memory, used alternately so an epilogue overlaps the next item's MMAs; a
// traits class with kWideAcc uses all 512 columns as one buffer (its items are
// long enough that the epilogue's share is small).
template <class T>
struct WideAcc {
    template <class U>
    static constexpr bool get(decltype(U::kWideAcc)*) { return U::kWideAcc; }
    template <class U>
    static constexpr bool get(...) { return false; }
    static constexpr bool value = get<T>(nullptr);
};

// Epilogue warps of the pair engine: four (one accumulator row per thread), or
// eight for a traits class with kEpiWarps = 8, whose second four take the upper
// half of the columns.
template <class T>
struct EpiWarps {
    template <class U>
    static constexpr int get(decltype(U::kEpiWarps)*) { return U::kEpiWarps; }
    template <class U>
    static constexpr int get(...) { return 4; }
    static constexpr int value = get<T>(nullptr);
};

// A traits class whose units are of several kinds has kMixed = true, kind(sc, unit)
// and, in place of mma(), mma_kind(kind, ...).
template <class T>
struct Mixed {
    template <class U>
    static constexpr bool get(decltype(U::kMixed)*) { return U::kMixed; }
    template <class U>
    static constexpr bool get(...) { return false; }
    static constexpr bool value = get<T>(nullptr);
};

// A traits class with kIdle = true has idle(), which runs in the peer CTA's MMA
// warp: that one has nothing to issue.
template <class T>
struct Idle {
    template <class U>
    static constexpr bool get(decltype(U::kIdle)*) { return U::kIdle; }
    template <class U>
    static constexpr bool get(...) { return false; }
    static constexpr bool value = get<T>(nullptr);
};

template <class T>
__device__ __forceinline__ int acc_buf(int it) {
    return WideAcc<T>::value ? 0 : (it & 1);
}

template <class T>
__device__ __forceinline__ uint32_t acc_phase(int it) {
    return WideAcc<T>::value ? (static_cast<uint32_t>(it) & 1u) : (static_cast<uint32_t>(it >> 1) & 1u);
}

template <class T, bool kBf16>
__device__ __forceinline__ void tc_pair_body(const typename T::Params& p, const CUtensorMap& mA, const CUtensorMap& mA2,
                                             const CUtensorMap& mB) {
    extern __shared__ uint8_t smem_raw[];
    typename T::Sched sc;
    // uniform across the pair: both CTAs read the same counters
    if (!T::setup(p, sc)) return;
    const int cid = static_cast<int>(blockIdx.x) >> 1;
    const int n_pairs = static_cast<int>(gridDim.x) >> 1;
    if (cid >= sc.n_units) return;   // no work for this pair: leave before touching TMEM
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;

    Smem sm = carve_smem<T::kStages, T::kStageBytes>(smem_raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    int* status = p.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < T::kStages; ++s) {
            mbar_init(&sm.full[s], 1);    // leader: its producer's expect_tx + both CTAs' bytes
            mbar_init(&sm.empty[s], 1);   // the leader's MMA commit, multicast to both CTAs
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.acc_full[b], 1);    // the leader's commit, multicast
            mbar_init(&sm.acc_empty[b], 2 * EpiWarps<T>::value);   // leader: the epilogue warps of both CTAs
        }
        mbar_init(sm.drain, 1);
        *sm.abort_flag = 0;
        sm.ld_count[0] = sm.ld_count[1] = sm.ld_count[2] = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&mA);
        tma_prefetch_desc(&mA2);
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

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        if (lane == 0) {
            int s = 0, n_issued = 0;
            uint32_t ph = 0;
            for (int unit = cid; unit < sc.n_units; unit += n_pairs) {
                const int n_items = T::items(p, sc, unit);
                const int ks = T::ksteps(p, sc, unit);
                for (int item = 0; item < n_items; ++item) {
                    const typename T::Coord c = T::coord(p, sc, unit, item, rank);
                    const uint32_t bytes = T::tx_bytes(p, sc, c);
                    for (int k = 0; k < ks; ++k) {
                        if (!mbar_wait(&sm.empty[s], ph ^ 1u, sm.abort_flag, status)) goto producer_done;
                        if (leader) mbar_arrive_expect_tx(&sm.full[s], bytes);
                        T::load(p, sc, c, k, sm.stages + s * T::kStageBytes, full0 + 8u * s, &mA, &mA2, &mB, rank);
                        ++n_issued;
                        if (++s == T::kStages) {
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
            int s = 0, n_used = 0;
            uint32_t ph = 0;
            int it = 0;
            for (int unit = cid; unit < sc.n_units; unit += n_pairs) {
                const int n_items = T::items(p, sc, unit);
                const int ks = T::ksteps(p, sc, unit);
                [[maybe_unused]] int kind = 0;
                if constexpr (Mixed<T>::value) kind = T::kind(sc, unit);
                for (int item = 0; item < n_items; ++item, ++it) {
                    const int b = acc_buf<T>(it);
                    const uint32_t aph = acc_phase<T>(it);
                    if (!mbar_wait(&sm.acc_empty[b], aph ^ 1u, sm.abort_flag, status)) goto mma_done;
                    tc_fence_after();
                    const uint32_t acc = tmem + b * 256;
                    for (int k = 0; k < ks; ++k) {
                        if (!mbar_wait(&sm.full[s], ph, sm.abort_flag, status)) goto mma_done;
                        ++n_used;
                        tc_fence_after();
                        const uint32_t stage = smem_u32(sm.stages + s * T::kStageBytes);
                        if constexpr (Mixed<T>::value)
                            T::template mma_kind<kBf16>(kind, stage, acc, k == 0);
                        else
                            T::template mma<kBf16>(stage, acc, k == 0);
                        umma_pair_commit_both(&sm.empty[s]);
                        if (++s == T::kStages) {
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
        if constexpr (Idle<T>::value)
            if (!leader) T::idle(p, lane);
    } else {
        // ------------------------------------------------ epilogue (both CTAs, own rows)
        const int row = lane + 32 * (warp & 3);
        const uint32_t tq = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        int it = 0;
        for (int unit = cid; unit < sc.n_units; unit += n_pairs) {
            const int n_items = T::items(p, sc, unit);
            typename T::Epi e;
            T::epi_begin(p, sc, unit, rank, row, e);
            for (int item = 0; item < n_items; ++item, ++it) {
                const int b = acc_buf<T>(it);
                const uint32_t aph = acc_phase<T>(it);
                if (!mbar_wait(&sm.acc_full[b], aph, sm.abort_flag, status)) goto epi_done;
                tc_fence_after();
                T::template epi_item<kBf16>(p, sc, unit, item, rank, tq + b * 256, e);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader)
                        mbar_arrive(&sm.acc_empty[b]);
                    else
                        mbar_arrive_cluster(acc_empty0 + 8u * b);
                }
            }
            T::epi_end(p, sc, rank, e);
        }
    epi_done:;
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // After an abort in either CTA, the loads still in flight (both CTAs' loads
    // complete on the leader's full barriers) must land before either CTA leaves.
    // The leader reads both CTAs' counts, waits for the K-stages both issued and
    // its MMA did not consume, and tells both CTAs whether that covered every
    // issued load; only when it did not do they fall back to the fixed wait.
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
            settled = wait_inflight<T::kStages>(sm.full, used, both) && issued == peer_issued ? 1 : 0;
        }
        sm.ld_count[2] = settled;
        st_shared_cluster_u32(peer_cnt + 8u, static_cast<uint32_t>(settled));
    }
    // the leader's MMAs write the peer's tensor memory, and the peer's loads
    // complete on the leader's barriers: nobody leaves before both are done
    cluster_sync();
    if (!sm.ld_count[2]) abort_grace(sm.abort_flag, true);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// Persistent launch: one CTA per SM, in clusters of kC; the grid is capped by
// how many clusters fit on the device at once, so every CTA runs concurrently.
template <class T, int kC, class K>
static cudaError_t launch_tc(K kern, const typename T::Params& p, const CUtensorMap& a, const CUtensorMap& a2,
                             const CUtensorMap& b, int n_sm, cudaStream_t st) {
    constexpr int smem = smem_bytes<T>();
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kC;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = n_sm / kC;
    if (kC > 1) {
        cfg.gridDim = dim3(clusters * kC);
        int active = 0;
        if (cudaOccupancyMaxActiveClusters(&active, kern, &cfg) == cudaSuccess && active > 0 && active < clusters)
            clusters = active;
    }
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3(clusters * kC);
    return cudaLaunchKernelEx(&cfg, kern, p, a, a2, b);
}

}  // namespace grpo
