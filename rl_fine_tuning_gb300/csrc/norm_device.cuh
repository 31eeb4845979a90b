// Device helpers of the norm and the checkpoints: 16-bit pairs, pairs of fp32
// numbers in one instruction, a row's loads, and the checkpoint's codes.
#pragma once
#include <atomic>
#include <cfloat>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "norm.h"
#include "ptx.cuh"

namespace grpo {

// ---------------------------------------------------------------- launches

// A kernel whose blocks may be brought onto the SMs while the kernel before it in the stream ends.  It touches no
// memory before chain_wait, so that for its results it is a launch like any other.
template <class P>
cudaError_t launch_chained(void (*f)(P), int64_t grid, int threads, size_t smem, const P& p, cudaStream_t st, int cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, f, p);
}

// Lets a kernel have the most shared memory that any call of it takes, once a device: the permission is the kernel's, not
// a launch's, so that with each call's own size calls from two threads would take it from one another.
struct MostSmem {
    std::atomic<unsigned long long> given{0};          // a bit a device

    template <class P>
    cudaError_t allow(void (*f)(P), int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
        if (given.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) given.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// ---------------------------------------------------------------- pairs of fp32 numbers
// sm_103 adds and multiplies two fp32 numbers in one instruction, each rounded as by
// itself.  Next to bandwidth these kernels are short of instructions: with one number an
// instruction, 8 elements a thread and the weight unpacked at each use, a gradient from a
// checkpoint took 929 us where HBM needs 351.  (The assembler may join a product with the sum
// after it into one rounding: where that matters the product is a single one, see encode.)

using F2 = unsigned long long;

__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 f2_values(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// ---------------------------------------------------------------- 16-bit pairs

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

template <bool kBf16>
__device__ __forceinline__ float2 pair_values(uint32_t p) {
    if (kBf16) return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&p));
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pair_bits(float lo, float hi) {
    if (kBf16) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}

// a b + c of pairs, rounded once.  For a sum (b = 1) that is the sum in fp32 rounded to
// 16 bits: 24 bits are at least twice 11 and two more, so rounding twice changes nothing.
template <bool kBf16>
__device__ __forceinline__ uint32_t pair_fma(uint32_t a, uint32_t b, uint32_t c) {
    if (kBf16) {
        const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                         *reinterpret_cast<const __nv_bfloat162*>(&b),
                                         *reinterpret_cast<const __nv_bfloat162*>(&c));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                              *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&r);
}

template <bool kBf16>
constexpr uint32_t kPairOne = kBf16 ? 0x3f803f80u : 0x3c003c00u;

// ---------------------------------------------------------------- a thread's 16 elements

// in 16 bits, and in fp32
struct Unit {
    uint32_t w[8];
};
struct Unit32 {
    F2 p[8];
};

// Later uses unpack x anew.  Without this the compiler keeps the 16 fp32 values of a unit from their first use to
// their second, beside the 8 registers that hold it, and spills for them (gradient from a checkpoint: 512 against 408 us).
__device__ __forceinline__ void forget_values(Unit* x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" : "+r"(x->w[i]));
}

template <bool kBf16>
__device__ __forceinline__ Unit32 values(const Unit& x) {
    Unit32 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = pair_values<kBf16>(x.w[i]);
        v.p[i] = f2(f.x, f.y);
    }
    return v;
}

template <bool kBf16>
__device__ __forceinline__ Unit rounded(const Unit32& v) {
    Unit x;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = f2_values(v.p[i]);
        x.w[i] = pair_bits<kBf16>(f.x, f.y);
    }
    return x;
}

// Loads of what is read once, past L1; zeros where `on` is false, without a branch.  (Not the read-only path: outputs may
// be in the place of inputs.)
__device__ __forceinline__ Unit load_unit(const uint16_t* a, bool on) {
    Unit x;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %9, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "mov.b32 %4, 0;\n\tmov.b32 %5, 0;\n\tmov.b32 %6, 0;\n\tmov.b32 %7, 0;\n\t"
        "@p ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t}"
        : "=&r"(x.w[0]), "=&r"(x.w[1]), "=&r"(x.w[2]), "=&r"(x.w[3]), "=&r"(x.w[4]), "=&r"(x.w[5]), "=&r"(x.w[6]),
          "=&r"(x.w[7])
        : "l"(a), "r"(static_cast<uint32_t>(on)));
    return x;
}

__device__ __forceinline__ uint4 load_codes(const int8_t* a, bool on) {
    uint4 x;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(x.x), "=&r"(x.y), "=&r"(x.z), "=&r"(x.w)
        : "l"(a), "r"(static_cast<uint32_t>(on)));
    return x;
}

__device__ __forceinline__ uint32_t load_scale(const uint16_t* a, bool on) {
    uint16_t x;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t@p ld.global.b16 %0, [%1];\n\t}"
        : "=&h"(x)
        : "l"(a), "r"(static_cast<uint32_t>(on)));
    return x;
}

// the same, leaving what was there where `on` is false
__device__ __forceinline__ void load_unit_if(const uint16_t* a, bool on, Unit* x) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %9, 0;\n\t"
        "@p ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t}"
        : "+r"(x->w[0]), "+r"(x->w[1]), "+r"(x->w[2]), "+r"(x->w[3]), "+r"(x->w[4]), "+r"(x->w[5]), "+r"(x->w[6]),
          "+r"(x->w[7])
        : "l"(a), "r"(static_cast<uint32_t>(on)));
}

__device__ __forceinline__ void load_codes_if(const int8_t* a, bool on, uint4* x) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "@p ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(x->x), "+r"(x->y), "+r"(x->z), "+r"(x->w)
        : "l"(a), "r"(static_cast<uint32_t>(on)));
}

__device__ __forceinline__ uint4 read16(uint32_t a) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a) : "memory");
    return x;
}

__device__ __forceinline__ Unit read_unit(uint32_t a) {
    const uint4 lo = read16(a), hi = read16(a + 16);
    return Unit{{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
}

__device__ __forceinline__ void store_unit(uint16_t* a, const Unit& x) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a), "r"(x.w[0]), "r"(x.w[1]),
                 "r"(x.w[2]), "r"(x.w[3]), "r"(x.w[4]), "r"(x.w[5]), "r"(x.w[6]), "r"(x.w[7])
                 : "memory");
}

// ---------------------------------------------------------------- 8 bits

// the largest scale of a checkpoint, 2^121 (bf16) or 2^9 (fp16), and its bits; the smallest bit pattern that is not finite
template <bool kBf16>
constexpr float kMostScale = kBf16 ? 2.658455992e36f : 512.f;
template <bool kBf16>
constexpr uint16_t kMostScaleBits = kBf16 ? 0x7c00 : 0x4400;
template <bool kBf16>
constexpr uint32_t kNotFinite = kBf16 ? 0x7f80u : 0x7c00u;

constexpr float kToInt = 12582912.f;   // 1.5 * 2^23: adding it leaves the nearest integer in the low bits

// 1 / s by one step of Newton's method from the approximate reciprocal: for every
// bf16 number from 2^-126 to 2^121 the correctly rounded one (a test runs it for all).
// __frcp_rn's handling of other numbers costs branches.
__device__ __forceinline__ float scale_reciprocal(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return fmaf(fmaf(-s, r, 1.f), r, r);
}

// The codes of a unit and the bits of its block's scale; 4 neighbouring lanes hold a block of kCkptBlock columns, and all
// lanes of the warp are here.  scale = max |x| / 127 in bf16, at least 2^-126.  Values are compared as bit
// patterns, so that a NaN is the largest; a block that is not finite gets the scale NaN.
// A scale rounded down puts the largest value at up to 127.5 steps: it still is
// within half a step of code 127.  Scales end where 127 of them still are finite in the
// 16-bit type; a block beyond that is divided by its own max |x| / 127 all the same.
template <bool kBf16>
__device__ __forceinline__ uint4 encode(const Unit& x, uint16_t* scale_bits) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, x.w[i] & 0x7fff7fffu);
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top & 0xffffu, top >> 16);
    const float s = fmaxf(__fmul_rn(pair_values<kBf16>(top).x, 1.f / 127), kLeastScale);
    const bool over = s > kMostScale<kBf16>;
    uint16_t bits = bf16_bits(s);
    const float inv = scale_reciprocal(over ? s : bf16_value(bits));
    bits = over ? kMostScaleBits<kBf16> : bits;
    *scale_bits = top >= kNotFinite<kBf16> ? 0x7fff : bits;
    const F2 to_int = f2(kToInt, kToInt);
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // single products: the assembler joins a product of a pair with a following sum into one rounding, and halves
        // would go to the wrong side
        const float2 v = pair_values<kBf16>(x.w[i]);
        const float2 f = f2_values(f2_add(f2(__fmul_rn(v.x, inv), __fmul_rn(v.y, inv)), to_int));
        q[i] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x0040);
    }
    return make_uint4(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410), __byte_perm(q[4], q[5], 0x5410),
                      __byte_perm(q[6], q[7], 0x5410));
}

// code * scale in fp32 (exact), rounded to 16 bits
template <bool kBf16>
__device__ __forceinline__ Unit decode(uint4 c, float scale) {
    const F2 s = f2(scale, scale), off = f2(-8388736.f, -8388736.f);
    const uint32_t u[4] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u, c.z ^ 0x80808080u, c.w ^ 0x80808080u};   // code + 128
    Unit32 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {                                     // 2^23 + code + 128 as a float's bits
        const float a = __uint_as_float(__byte_perm(u[i / 2], 0x4b000000u, 0x7540 + 2 * (i & 1)));
        const float b = __uint_as_float(__byte_perm(u[i / 2], 0x4b000000u, 0x7541 + 2 * (i & 1)));
        v.p[i] = f2_mul(f2_add(f2(a, b), off), s);
    }
    return rounded<kBf16>(v);
}

template <bool kE5m2>
__device__ __forceinline__ uint4 codes8(const Unit32& v) {
    constexpr __nv_fp8_interpretation_t t = kE5m2 ? __NV_E5M2 : __NV_E4M3;
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = __nv_cvt_float2_to_fp8x2(f2_values(v.p[i]), __NV_SATFINITE, t);
    return make_uint4(c[0] | c[1] << 16, c[2] | c[3] << 16, c[4] | c[5] << 16, c[6] | c[7] << 16);
}

// ---------------------------------------------------------------- a row's threads

enum Source { kX, kXResidual, kCkpt };

// What a thread holds of a row as it lies in memory.
template <int kSrc, int kUpt>
struct Raw {
    Unit x[kSrc == kCkpt ? 1 : kUpt];
    Unit r[kSrc == kXResidual ? kUpt : 1];
    uint4 c[kSrc == kCkpt ? kUpt : 1];
    uint32_t scale[kSrc == kCkpt ? kUpt : 1];
};

template <bool kWide>
__device__ __forceinline__ void load_matrix(const uint16_t* a, bool on, Unit* x) {
    if (kWide)
        load_unit_if(a, on, x);
    else
        *x = load_unit(a, on);
}

// A row's threads: `lane` of `width` (4, 8, 16 or 32 lanes of a warp, or whole warps), with units lane, lane + width.
// at: the thread's first element.  The rows of a warp get zeros where they do not count, and behind their end.  A wide
// row's threads keep there what they had: such a row is left out as a whole, and what lies behind a
// row's end is left out of the sums and of the outputs, so that it needs no zeros.
template <int kSrc, int kUpt, bool kWide>
__device__ __forceinline__ void load_row(const NormParams& p, int64_t at, bool on, int lane, int width, int n_unit,
                                         Raw<kSrc, kUpt>* raw) {
#pragma unroll
    for (int k = 0; k < kUpt; ++k) {
        const bool in = on && lane + k * width < n_unit;
        const int64_t e = at + k * width * kUnit;
        if (kSrc == kCkpt) {
            if (kWide)
                load_codes_if(p.codes + e, in, &raw->c[k]);
            else
                raw->c[k] = load_codes(p.codes + e, in);
            raw->scale[k] = load_scale(p.scales + (e >> 6), in);
        } else {
            load_matrix<kWide>(p.x + e, in, &raw->x[k]);
            if (kSrc == kXResidual) load_matrix<kWide>(p.residual + e, in, &raw->r[k]);
        }
    }
}

template <bool kBf16, int kSrc, int kUpt>
__device__ __forceinline__ Unit stream_of(const Raw<kSrc, kUpt>& raw, int k) {
    if (kSrc == kCkpt) return decode<kBf16>(raw.c[k], bf16_value(raw.scale[k]));
    Unit s = raw.x[k];
    if (kSrc == kXResidual) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s.w[i] = pair_fma<kBf16>(s.w[i], kPairOne<kBf16>, raw.r[k].w[i]);
    }
    return s;
}

// Which of the rows to come count, for rows t, t + step, ...  The lanes of a row look
// ahead together, each at one row, a window of 32 rows (of 4, 8 or 16 where fewer lanes have a row) and the one
// after it: a mask byte's way from memory takes longer than a row that does not count.
struct Ahead {
    uint32_t now, then;          // bit i: row i of this window, and of the next
    bool last;                   // this lane's row of the one after that
    int i;

    __device__ __forceinline__ bool look(const NormParams& p, uint32_t t, uint32_t step, int lane, int rows) const {
        const uint32_t r = t + lane * step;
        return lane < rows && r < static_cast<uint32_t>(p.N) && (!p.mask || p.mask[r]);
    }
    // the window of this lane's row
    __device__ __forceinline__ static uint32_t join(bool v, int width) {
        const uint32_t all = __ballot_sync(0xffffffffu, v);
        return width >= 32 ? all : all >> (threadIdx.x & 31 & ~(width - 1)) & ((1u << width) - 1);
    }
    __device__ __forceinline__ void begin(const NormParams& p, uint32_t t, uint32_t step, int width) {
        const int rows = width < 32 ? width : 32, lane = threadIdx.x & (rows - 1);
        const bool a = look(p, t, step, lane, rows), b = look(p, t + rows * step, step, lane, rows);
        last = look(p, t + 2 * rows * step, step, lane, rows);
        now = join(a, width);
        then = join(b, width);
        i = 0;
    }
    // bit q: row t + q step counts, q < the window's rows
    __device__ __forceinline__ uint32_t bits(int width) const {
        const int rows = width < 32 ? width : 32;
        return i == 0 ? now : now >> i | then << (rows - i);
    }
    // t: the row before, which is done
    __device__ __forceinline__ void advance(const NormParams& p, uint32_t t, uint32_t step, int width) {
        const int rows = width < 32 ? width : 32;
        if (++i < rows) return;
        i = 0;
        now = then;
        then = join(last, width);
        last = look(p, t + (2 * rows + 1) * step, step, threadIdx.x & (rows - 1), rows);
    }
};

// The weight (plus 0 or 1) in fp32 in shared memory, in four planes of 4 columns of every unit, so that neighbouring
// lanes read neighbouring 16 bytes; `pad` units a plane, zeros behind the row's end.  The caller's next barrier makes it
// visible.
template <bool kBf16>
__device__ __forceinline__ void stage_weight(const NormParams& p, float4* planes, int pad) {
    for (int i = threadIdx.x; i < 4 * pad; i += blockDim.x) {         // 4 columns each
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (4 * i < p.d) {
            if (p.weight_f32) {
                a = reinterpret_cast<const float4*>(p.weight)[i];
            } else {
                const uint2 w = reinterpret_cast<const uint2*>(p.weight)[i];
                const float2 lo = pair_values<kBf16>(w.x), hi = pair_values<kBf16>(w.y);
                a = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
            a = make_float4(a.x + p.plus, a.y + p.plus, a.z + p.plus, a.w + p.plus);
        }
        planes[(i & 3) * pad + (i >> 2)] = a;
    }
}

__device__ __forceinline__ Unit32 staged_weight(const float4* planes, int pad, int i) {
    Unit32 w;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 a = planes[q * pad + i];
        w.p[2 * q] = f2(a.x, a.y);
        w.p[2 * q + 1] = f2(a.z, a.w);
    }
    return w;
}

__device__ __forceinline__ float sum_of(F2 v) {
    const float2 f = f2_values(v);
    return f.x + f.y;
}

}  // namespace grpo
