// C ABI of the norm before the head, its gradient and the 8-bit checkpoints:
// argument checks, workspace layout and launches.
#include <cmath>
#include <cstring>

#include "abi_common.h"
#include "norm.h"

namespace grpo {

namespace {

constexpr int64_t kMostElements = 1LL << 43;   // 2^30 blocks of a checkpoint's kernels
constexpr size_t kMatrixAlign = 32;            // of a 16-bit matrix: its 32-byte sectors are loaded and stored whole

// What the gradient's workspace holds: sums of the weight's gradient, and flags.
struct NormWs {
    size_t part, bad, total;
};

NormWs norm_ws(int64_t N, int d) {
    const int parts = norm_parts(N, d);
    NormWs w;
    w.part = 0;
    w.bad = align_up(static_cast<size_t>(parts) * d * 4, 256);
    w.total = w.bad + align_up(static_cast<size_t>(parts) * 4, 256);
    return w;
}

// The current device's SMs; a device is asked once (its attributes take a microsecond a call).
int sm_count(int* out) {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GRPO_ERR_LAUNCH;
    if (dev < 64 && (*out = known[dev].load(std::memory_order_relaxed)) > 0) return GRPO_OK;
    DeviceInfo info;
    const int rc = device_info(&info);
    if (rc != GRPO_OK) return rc;
    *out = info.sm_count;
    if (dev < 64) known[dev].store(info.sm_count, std::memory_order_relaxed);
    return GRPO_OK;
}

int64_t rows_of(const grpo_shape& s) { return static_cast<int64_t>(s.n_groups) * s.G * s.L; }

int norm_shape(const grpo_shape* s, int most_d) {
    if (!s) return GRPO_ERR_SHAPE;
    if (!dtype_ok(*s)) return GRPO_ERR_DTYPE;
    if (!shape_ok(*s) || s->d > most_d || rows_of(*s) * s->d > kMostElements) return GRPO_ERR_SHAPE;
    return GRPO_OK;
}

int norm_opts_check(const grpo_shape& s, const grpo_norm_opts* o, bool forward) {
    if (!o) return GRPO_ERR_SHAPE;
    if (!(o->eps >= kLeastScale) || !std::isfinite(o->eps)) return GRPO_ERR_SHAPE;
    if ((o->weight_f32 | 1) != 1 || (o->plus_one | 1) != 1) return GRPO_ERR_SHAPE;
    if (!forward) return GRPO_OK;
    if (o->y_type != s.dtype && o->y_type != GRPO_E4M3 && o->y_type != GRPO_E5M2) return GRPO_ERR_DTYPE;
    if (o->y_scale != 0.f && (o->y_type == s.dtype || !(o->y_scale >= kLeastScale) || !(o->y_scale <= 1.f / kLeastScale)))
        return GRPO_ERR_SHAPE;
    return GRPO_OK;
}

template <class P>
bool given(const P* p, size_t a) { return p && aligned(p, a); }

// a matrix that may be left out
template <class P>
bool left_or(const P* p, size_t a) { return !p || aligned(p, a); }

bool ckpt_ok(const grpo_ckpt* c) { return given(c->codes, 16) && given(c->scales, 2); }

// s comes from exactly one of x and a checkpoint
bool source_ok(const void* x, const grpo_ckpt* c) {
    if (x) return !c && aligned(x, kMatrixAlign);
    return c && ckpt_ok(c);
}

void set_source(NormParams* p, const void* x, const grpo_ckpt* c) {
    p->x = static_cast<const uint16_t*>(x);
    if (c) {
        p->codes = c->codes;
        p->scales = c->scales;
    }
}

NormParams norm_params(const grpo_shape& s, const grpo_norm_opts& o, const void* weight, const uint8_t* mask) {
    NormParams p = {};
    p.weight = weight;
    p.mask = mask;
    p.N = rows_of(s);
    p.d = s.d;
    p.eps = o.eps;
    p.weight_f32 = o.weight_f32;
    p.plus = static_cast<float>(o.plus_one);
    p.y_type = o.y_type;
    p.y_inv = o.y_scale != 0.f ? 1.f / o.y_scale : 0.f;
    return p;
}

int launch_ckpt(cudaError_t (*f)(const CkptParams&, bool, cudaStream_t), const CkptParams& p, bool bf16, cudaStream_t st) {
    int sms = 0;
    const int rc = sm_count(&sms);
    if (rc != GRPO_OK) return rc;
    return launch(GRPO_PROF_CKPT, st, [&] { return f(p, bf16, st); }) == cudaSuccess ? GRPO_OK : GRPO_ERR_LAUNCH;
}

CkptParams ckpt_params(const grpo_shape& s, const uint8_t* mask) {
    CkptParams p = {};
    p.mask = mask;
    p.N = rows_of(s);
    p.d = s.d;
    p.per_row = ~0ull / static_cast<uint64_t>(s.d / 16) + 1;
    return p;
}

}  // namespace

}  // namespace grpo

using namespace grpo;

extern "C" {

void grpo_norm_opts_init(grpo_norm_opts* o, grpo_dtype dtype) {
    if (!o) return;
    std::memset(o, 0, sizeof(*o));
    o->eps = 1e-6f;
    o->y_type = dtype;
}

size_t grpo_norm_workspace_bytes(const grpo_shape* shape) {
    if (norm_shape(shape, kNormMaxD) != GRPO_OK) return 0;
    return norm_ws(rows_of(*shape), shape->d).total;
}

int grpo_norm_fwd(const void* x, const grpo_ckpt* x_ckpt, const void* residual, const void* weight, const uint8_t* mask,
                  const grpo_shape* shape, const grpo_norm_opts* opts, void* y, float* row_scale, void* sum_out,
                  const grpo_ckpt* sum_ckpt, grpo_stream_t stream) {
    int rc = norm_shape(shape, kNormMaxD);
    if (rc == GRPO_OK) rc = norm_opts_check(*shape, opts, true);
    if (rc != GRPO_OK) return rc;
    const bool y16 = opts->y_type == shape->dtype;
    if (!source_ok(x, x_ckpt) || !left_or(residual, kMatrixAlign) || !given(weight, 16) ||
        !given(y, y16 ? kMatrixAlign : 16) || !left_or(row_scale, 4) || !left_or(sum_out, kMatrixAlign) ||
        (sum_ckpt && !ckpt_ok(sum_ckpt)))
        return GRPO_ERR_POINTER;
    if (x_ckpt && (residual || sum_ckpt)) return GRPO_ERR_POINTER;
    if (y16 ? row_scale != nullptr : !row_scale && opts->y_scale == 0.f) return GRPO_ERR_POINTER;
    int sms = 0;
    rc = sm_count(&sms);
    if (rc != GRPO_OK) return rc;
    NormParams p = norm_params(*shape, *opts, weight, mask);
    set_source(&p, x, x_ckpt);
    p.residual = static_cast<const uint16_t*>(residual);
    p.y = y;
    p.row_scale = row_scale;
    p.sum = static_cast<uint16_t*>(sum_out);
    if (sum_ckpt) {
        p.codes_out = sum_ckpt->codes;
        p.scales_out = sum_ckpt->scales;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const NormPlan plan = norm_fwd_plan(p.N, p.d, sms);
    p.width = plan.width;
    return launch(GRPO_PROF_NORM, st, [&] { return launch_norm_fwd(p, plan, shape->dtype == GRPO_BF16, st); }) ==
                   cudaSuccess
               ? GRPO_OK
               : GRPO_ERR_LAUNCH;
}

int grpo_norm_bwd(const void* dy, const void* x, const grpo_ckpt* x_ckpt, const void* weight, const void* dsum,
                  const uint8_t* mask, const grpo_shape* shape, const grpo_norm_opts* opts, void* workspace, size_t ws_bytes,
                  void* dx, void* dweight, int32_t* found_inf, grpo_stream_t stream) {
    int rc = norm_shape(shape, kNormMaxD);
    if (rc == GRPO_OK) rc = norm_opts_check(*shape, opts, false);
    if (rc != GRPO_OK) return rc;
    if (!given(dy, kMatrixAlign) || !source_ok(x, x_ckpt) || !given(weight, 16) || !left_or(dsum, kMatrixAlign) ||
        !given(workspace, 256) || !given(dx, kMatrixAlign) || !left_or(dweight, 16) || !given(found_inf, 4))
        return GRPO_ERR_POINTER;
    NormParams p = norm_params(*shape, *opts, weight, mask);
    const NormWs w = norm_ws(p.N, p.d);
    if (ws_bytes < w.total) return GRPO_ERR_WORKSPACE;
    int sms = 0;
    rc = sm_count(&sms);
    if (rc != GRPO_OK) return rc;
    set_source(&p, x, x_ckpt);
    p.dy = static_cast<const uint16_t*>(dy);
    p.dsum = static_cast<const uint16_t*>(dsum);
    p.dx = static_cast<uint16_t*>(dx);
    p.dweight = dweight;
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.part);
    p.bad = reinterpret_cast<int*>(static_cast<char*>(workspace) + w.bad);
    NormPlan plan = norm_bwd_plan(p.N, p.d, sms, x_ckpt != nullptr, dsum != nullptr);
    const int parts = norm_parts(p.N, p.d);          // fewer only on more SMs than kSmCount
    if (plan.grid > parts) plan.grid = parts;
    p.width = plan.width;
    p.parts = plan.grid;
    p.joined = plan.joined;
    p.found_inf = found_inf;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = shape->dtype == GRPO_BF16;
    if (launch(GRPO_PROF_NORM_BWD, st, [&] { return launch_norm_bwd(p, plan, bf16, st); }) != cudaSuccess) return GRPO_ERR_LAUNCH;
    if (!plan.joined &&
        launch(GRPO_PROF_NORM_BWD, st, [&] { return launch_norm_join(p, bf16, st); }) != cudaSuccess)
        return GRPO_ERR_LAUNCH;
    return GRPO_OK;
}

int grpo_ckpt_pack(const void* x, const uint8_t* mask, const grpo_shape* shape, const grpo_ckpt* out, grpo_stream_t stream) {
    const int rc = norm_shape(shape, 65536);
    if (rc != GRPO_OK) return rc;
    if (!given(x, kMatrixAlign) || !out || !ckpt_ok(out)) return GRPO_ERR_POINTER;
    CkptParams p = ckpt_params(*shape, mask);
    p.x = static_cast<const uint16_t*>(x);
    p.codes_out = out->codes;
    p.scales_out = out->scales;
    return launch_ckpt(launch_ckpt_pack, p, shape->dtype == GRPO_BF16, reinterpret_cast<cudaStream_t>(stream));
}

int grpo_ckpt_unpack(const grpo_ckpt* ckpt, const uint8_t* mask, const grpo_shape* shape, void* x_out, grpo_stream_t stream) {
    const int rc = norm_shape(shape, 65536);
    if (rc != GRPO_OK) return rc;
    if (!ckpt || !ckpt_ok(ckpt) || !given(x_out, kMatrixAlign)) return GRPO_ERR_POINTER;
    CkptParams p = ckpt_params(*shape, mask);
    p.codes = ckpt->codes;
    p.scales = ckpt->scales;
    p.x_out = static_cast<uint16_t*>(x_out);
    return launch_ckpt(launch_ckpt_unpack, p, shape->dtype == GRPO_BF16, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
