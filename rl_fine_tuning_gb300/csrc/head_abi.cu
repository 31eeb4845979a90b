// C ABI of the head operators: argument checks, workspace layout and launch
// sequences of the log-probs, the clipped policy loss and the preference loss.
#include <cmath>
#include <cstring>

#include "abi_common.h"
#include "head.h"

namespace grpo {

namespace {

constexpr int64_t kPairChunkRowsMax = 19456;   // default chunks grow to hold one whole pair up to this (152 tiles of 128)

// bf16 chunks of at least this many logits use relative dlogits (k_head_scale)
// instead of a pass over the dlogits.  The pass against the relative way, for a
// whole backward call at d = 1024: 60 against 62 us for 1M logits, 78 against 79 for
// 4M, 165 against 152 for 8M (128 rows), 326 against 286 for 64M.
constexpr int64_t kRelativeMin = 1 << 22;

// Chunks of at most this much work per gradient (rows x V x d) compute dH and dW
// in one launch; above, each has a kernel of its own, whose inner loops know
// their operands.  One launch against two, for a whole backward call: 39 against
// 44 us at 3e7, 112 against 118 at 1.6e10, 188 against 188 at 2e10, 435 against 420 at 5e10.
constexpr double kOneLaunchMax = 2e10;

// Temperatures between which the logits kernels' numbers hold.  Above, kNoLogit /
// temperature, the stand-in for a column that does not count, would come near the
// logits (at 1e30 it is -1.3).  Below, logits of 100 would pass 1e8, where a step of
// fp32 is 8: an exponential relative to a rounded maximum can then leave fp16's range.
constexpr float kLeastTemperature = 1e-6f, kMostTemperature = 1e20f;

struct HeadLayout {
    size_t counts, off, cb, pb, dh_plan, lg_plan, gmax, far, oscale, rowf, rows, zt, lse2, gco, ell, q, pair_ell, hc, part, mx, ds, hct, dh_part,
        dw_acc, total;
    int64_t N;
    int n_seq, R, max_chunks, S, n_ntiles, n_vt, V_pad, nc32, slots, by_pair, relative, one_launch, dh_cols;
};

bool head_shape_ok(const grpo_shape& s, int op) {
    if (!shape_ok(s)) return false;
    if (op == GRPO_OP_PAIR && s.G != 2) return false;
    return op >= GRPO_OP_LOGPROBS && op <= GRPO_OP_PAIR;
}

bool has_backward(int op) { return op != GRPO_OP_LOGPROBS; }

// Rows per chunk.  Default: 76 tiles of 128 (9728).  A chunk's dlogits take
// V 2 bytes a row; fewer, larger chunks add fewer times to dW's fp32 sum (8 V d
// bytes each time).  The preference loss grows a default chunk to one whole
// pair (2 L rows): with whole pairs in a chunk the logits are computed once
// instead of twice, 6 N V d operations instead of 8 N V d.  Above
// kPairChunkRowsMax a chunk's buffers would outgrow that.
int head_chunk_rows(const grpo_shape& s, int op) {
    const int64_t N = static_cast<int64_t>(s.n_groups) * s.G * s.L;
    const int64_t nmax = (N + kBM - 1) / kBM * kBM;
    int64_t r = s.chunk_rows > 0 ? (s.chunk_rows + static_cast<int64_t>(kBM) - 1) / kBM * kBM
                                 : static_cast<int64_t>(kHeadChunkTiles) * kBM;
    if (op == GRPO_OP_PAIR && s.chunk_rows == 0) {
        const int64_t pair = (2LL * s.L + kBM - 1) / kBM * kBM;
        if (pair > r && pair <= kPairChunkRowsMax) r = pair;
    }
    return static_cast<int>(r < nmax ? r : nmax);
}

bool head_layout(const grpo_shape& s, int op, int dw_f32, HeadLayout* o) {
    if (!head_shape_ok(s, op)) return false;
    const int64_t N = static_cast<int64_t>(s.n_groups) * s.G * s.L;
    o->N = N;
    o->n_seq = s.n_groups * s.G;
    o->R = head_chunk_rows(s, op);
    o->by_pair = op == GRPO_OP_PAIR && 2LL * s.L <= o->R;
    o->max_chunks = static_cast<int>((N + o->R - 1) / o->R);
    if (o->by_pair) {
        const int ppc = static_cast<int>(o->R / (2LL * s.L));
        o->max_chunks = (s.n_groups + ppc - 1) / ppc;
    }
    o->relative = has_backward(op) && s.dtype == GRPO_BF16 && static_cast<int64_t>(o->R) * s.V >= kRelativeMin;
    o->n_ntiles = (s.V + kBN - 1) / kBN;
    o->n_vt = (s.V + kBM - 1) / kBM;
    o->one_launch = has_backward(op) && static_cast<double>(o->R) * s.V * s.d <= kOneLaunchMax;
    // splits: at most kHeadSplitsMax (half of that with many row tiles, whose units are many anyway), and at
    // least what 64 tiles a split give
    const int least = (o->n_ntiles + 63) / 64;
    const int splits = o->R > 16 * kBM ? kHeadSplitsMax / 2 : kHeadSplitsMax;
    o->S = o->n_ntiles < splits ? o->n_ntiles : least > splits ? least : splits;
    o->V_pad = (s.V + 63) / 64 * 64;
    o->nc32 = ((s.V + 31) / 32 + 7) / 8 * 8;
    // dH in units of 512 columns where d is whole units and a full chunk has two for every SM pair: 4.50
    // against 4.74 ms for dH of 7.5K rows of the 8B head; with fewer units their raggedness costs more
    // (d = 1536, 4.9K rows: 1.45 against 1.37 ms)
    const int row_pairs = (o->R + 2 * kBM - 1) / (2 * kBM);
    o->dh_cols = !o->one_launch && s.d % (2 * kBN) == 0 && row_pairs * (s.d / (2 * kBN)) >= 2 * kSmPairs ? 2 * kBN : kBN;
    const int64_t units = static_cast<int64_t>(row_pairs) * ((s.d + o->dh_cols - 1) / o->dh_cols);
    // up to 32 K-stages (V = 2048) a unit is not worth splitting: no partial tiles, and no launch to join them
    const int ks = (s.V + kBK - 1) / kBK;
    const int64_t pieces = ks > 32 ? units * ks : 0;
    const int most = o->dh_cols == kBN ? kDhSlotsMax : kDhWideSlotsMax;
    o->slots = static_cast<int>(pieces < most ? pieces : most);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    const size_t n = static_cast<size_t>(N), R = static_cast<size_t>(o->R), mc = static_cast<size_t>(o->max_chunks);
    o->counts = take(C_COUNT_WORDS * 4);
    o->off = take((static_cast<size_t>(o->n_seq) + 1) * 4);
    o->cb = take((mc + 1) * 4);
    o->pb = take((mc + 1) * 4);
    o->dh_plan = take(mc * 8);
    o->lg_plan = take(mc * 8);
    o->gmax = take(mc * 4);
    o->far = take(mc * 4);
    o->oscale = take(mc * 4);
    o->rows = take(n * 4);
    o->zt = take(n * 8);
    o->lse2 = take(n * 8);
    o->gco = take(n * 4);
    o->ell = take(n * 4);
    o->q = take(n * 4);
    o->pair_ell = take(op == GRPO_OP_PAIR ? static_cast<size_t>(s.n_groups) * 8 : 0);
    o->hc = take(R * s.d * 2);
    size_t part = R * 2 * o->S * 16;
    const size_t few = static_cast<size_t>(kFewRows) * kFewCtas * 16;   // the few-row kernel: one partial per row and CTA
    if (op == GRPO_OP_LOGPROBS && part < few) part = few;
    o->part = take(part);
    o->rowf = o->mx = o->ds = o->hct = o->dh_part = o->dw_acc = off;
    if (has_backward(op)) {
        o->rowf = take(R * 4);
        o->mx = take(R * o->nc32 * 4);
        o->ds = take(R * o->V_pad * 2);
        o->hct = take(R * s.d * 2);
        o->dh_part = take(static_cast<size_t>(o->slots) * 2 * kBM * o->dh_cols * 4);
        if (!dw_f32 && o->max_chunks > 1) o->dw_acc = take(static_cast<size_t>(s.V) * s.d * 4);
    }
    o->total = off;
    return true;
}

// What every operator takes; an operator leaves what it does not use at null.
struct HeadCall {
    const void *h, *W;
    const int32_t* tokens;
    const uint8_t* mask;
    const grpo_shape* shape;
    void* ws;
    size_t ws_bytes;
    int32_t* status;
    int op = GRPO_OP_LOGPROBS;
    int mode = HEAD_LOGP;
    bool backward = false;
    float temperature = 1.f;
    // outputs and per-row inputs
    float* loss = nullptr;
    float* logp = nullptr;
    float* entropy = nullptr;
    float* stats = nullptr;
    const float* dlogp = nullptr;
    const float* adv = nullptr;
    const float* logp_old = nullptr;
    const float* logp_ref = nullptr;
    grpo_clip_opts clip = {};
    grpo_pair_opts pair = {};
    float* pair_stats = nullptr;
    // gradients
    float loss_scale = 1.f;
    void* dH = nullptr;
    void* dW = nullptr;
    int dw_f32 = 0;
    int32_t* found_inf = nullptr;
};

bool f32_ok(const void* p) { return aligned(p, 4); }   // null counts as aligned

int head_validate(const HeadCall& c, HeadLayout* L) {
    if (!c.shape) return GRPO_ERR_SHAPE;
    const grpo_shape& s = *c.shape;
    if (!dtype_ok(s)) return GRPO_ERR_DTYPE;
    if (!head_layout(s, c.op, c.dw_f32, L)) return GRPO_ERR_SHAPE;
    if (!(c.temperature >= kLeastTemperature) || !(c.temperature <= kMostTemperature)) return GRPO_ERR_SHAPE;
    if (!c.h || !c.W || !c.tokens || !c.ws || !c.status) return GRPO_ERR_POINTER;
    if (!c.mask && c.mode != HEAD_LOGP) return GRPO_ERR_POINTER;
    if (!aligned(c.h, 16) || !aligned(c.W, 16) || !f32_ok(c.tokens) || !aligned(c.ws, 256) || !f32_ok(c.status))
        return GRPO_ERR_POINTER;
    if (!f32_ok(c.loss) || !f32_ok(c.logp) || !f32_ok(c.entropy) || !f32_ok(c.stats) || !f32_ok(c.dlogp) || !f32_ok(c.adv) ||
        !f32_ok(c.logp_old) || !f32_ok(c.logp_ref) || !f32_ok(c.pair_stats))
        return GRPO_ERR_POINTER;
    if (c.backward) {
        if (!c.dH || !c.dW || !c.found_inf || !aligned(c.dH, 32) || !aligned(c.dW, 32) || !f32_ok(c.found_inf))
            return GRPO_ERR_POINTER;
        if (!(c.loss_scale > 0.f) || !std::isfinite(c.loss_scale)) return GRPO_ERR_SHAPE;
        if (c.dw_f32 != 0 && c.dw_f32 != 1) return GRPO_ERR_SHAPE;
    }
    if (c.ws_bytes < L->total) return GRPO_ERR_WORKSPACE;
    return GRPO_OK;
}

// One kernel through launch(); false on error
#define HEAD_LAUNCH(kind, call)                                                     \
    do {                                                                            \
        if (launch(kind, st, [&] { return call; }) != cudaSuccess) return GRPO_ERR_LAUNCH; \
    } while (0)

// logit = zscale * accumulator, with the correction of the tensor cores' rounding
// (see head_tc.cu) for pieces of d / 16 / (pieces) additions
void logit_scale(const HeadCall& c, float* zscale, float* zscale2) {
    const int d = c.shape->d, pieces = (d + kPieceK - 1) / kPieceK;
    const double n_eff = d / 16.0 / pieces;
    const double z = (1.0 + kAddLoss * n_eff) / static_cast<double>(c.temperature);
    *zscale = static_cast<float>(z);
    *zscale2 = static_cast<float>(z * 1.4426950408889634074);
}

// Log-probs of at most kFewRows rows: no plan, no copies, one pass over W.
int run_few(const HeadCall& c, const HeadLayout& L, const DeviceInfo& dev, cudaStream_t st) {
    const grpo_shape& s = *c.shape;
    const bool bf16 = s.dtype == GRPO_BF16;
    char* w = static_cast<char*>(c.ws);
    const int N = static_cast<int>(L.N), nc = N <= 16 ? 16 : 32;
    CUtensorMap mH, mW;
    if (!make_map(&mH, c.h, bf16, s.d, N, s.d, kBK, nc) || !make_map(&mW, c.W, bf16, s.d, s.V, s.d, kBK, kFewVocab))
        return GRPO_ERR_LAUNCH;
    FewParams p = {};
    p.tokens = c.tokens;
    p.mask = c.mask;
    p.zt = reinterpret_cast<double*>(w + L.zt);
    p.part = reinterpret_cast<float4*>(w + L.part);
    p.counter = reinterpret_cast<int*>(w + L.counts);
    p.logp = c.logp;
    p.entropy = c.entropy;
    p.inv_t = 1.f / c.temperature;
    logit_scale(c, &p.zscale, &p.zscale2);
    p.N = N;
    p.V = s.V;
    p.d = s.d;
    p.n_tiles = (s.V + kFewVocab - 1) / kFewVocab;
    p.status = c.status;
    int grid = p.n_tiles < dev.sm_count ? p.n_tiles : dev.sm_count;
    if (grid > kFewCtas) grid = kFewCtas;
    HEAD_LAUNCH(GRPO_PROF_GATHER,
                launch_few_prep(p, static_cast<const uint16_t*>(c.h), static_cast<const uint16_t*>(c.W), bf16,
                                reinterpret_cast<double*>(w + L.zt), st));
    HEAD_LAUNCH(GRPO_PROF_FWD, launch_few(p, mH, mW, grid, bf16, nc, st));
    return GRPO_OK;
}

struct HeadRun {
    const HeadCall& c;
    const HeadLayout& L;
    const DeviceInfo& dev;
    cudaStream_t st;
    char* w;
    bool bf16;
    CUtensorMap mW_k, mH_k, mW_mn, mHct, mDS_k, mDS_mn;

    template <class T>
    T* at(size_t off) const { return reinterpret_cast<T*>(w + off); }

    int maps() {
        const grpo_shape& s = *c.shape;
        if (!make_map(&mW_k, c.W, bf16, s.d, s.V, s.d, kBK, kBN / 2) ||
            !make_map(&mH_k, at<void>(L.hc), bf16, s.d, L.R, s.d, kBK, kBM))
            return GRPO_ERR_LAUNCH;
        if (c.backward && (!make_map(&mW_mn, c.W, bf16, s.d, s.V, s.d, 64, kBK) ||
                           !make_map(&mHct, at<void>(L.hct), bf16, L.R, s.d, L.R, kBK, 128) ||
                           !make_map(&mDS_k, at<void>(L.ds), bf16, s.V, L.R, L.V_pad, kBK, kBM) ||
                           !make_map(&mDS_mn, at<void>(L.ds), bf16, s.V, L.R, L.V_pad, 64, kBK)))
            return GRPO_ERR_LAUNCH;
        return GRPO_OK;
    }

    int plan() {
        const grpo_shape& s = *c.shape;
        PlanParams p = {};
        p.mask = c.mask;
        p.N = L.N;
        p.L = s.L;
        p.n_seq = L.n_seq;
        p.R = L.R;
        p.by_pair = L.by_pair;
        p.max_chunks = L.max_chunks;
        p.n_nt = (s.d + L.dh_cols - 1) / L.dh_cols;
        p.ks = (s.V + kBK - 1) / kBK;
        p.n_pairs = dev.sm_count / 2;
        p.slots_max = L.slots;
        p.backward = c.backward;
        p.n_w = L.one_launch ? (L.n_vt + 1) / 2 * p.n_nt : 0;
        p.loss = c.loss;
        p.counts = at<int>(L.counts);
        p.off = at<int>(L.off);
        p.cb = at<int>(L.cb);
        p.pb = at<int>(L.pb);
        p.dh_plan = at<int2>(L.dh_plan);
        p.lg_plan = at<int2>(L.lg_plan);
        p.n_ntiles = L.n_ntiles;
        p.s_max = L.S;
        p.gmax = at<unsigned>(L.gmax);
        p.far = at<int>(L.far);
        p.rows = at<int>(L.rows);
        p.found_inf = c.found_inf;
        p.status = c.status;
        p.pairs_of_g2 = c.mode == HEAD_PAIR;
        HEAD_LAUNCH(GRPO_PROF_INDEX, launch_plan(p, st));
        return GRPO_OK;
    }

    // compact rows of a chunk, and with them (first: once per call) the zeros of masked rows
    int gather(int chunk, bool with_t, bool first) {
        const grpo_shape& s = *c.shape;
        GatherParams p = {};
        p.counts = at<int>(L.counts);
        p.cb = at<int>(L.cb);
        p.rows = at<int>(L.rows);
        p.tokens = c.tokens;
        p.mask = first ? c.mask : nullptr;
        p.h = static_cast<const uint16_t*>(c.h);
        p.W = static_cast<const uint16_t*>(c.W);
        p.hc = at<uint16_t>(L.hc);
        p.hct = with_t ? at<uint16_t>(L.hct) : nullptr;
        p.zt = at<double>(L.zt);
        if (first) {
            p.dH = static_cast<uint16_t*>(c.dH);
            p.dW = c.dW;
            p.dw_bytes = static_cast<int64_t>(s.V) * s.d * (c.dw_f32 ? 4 : 2);
            p.out0 = c.logp;
            p.out1 = c.entropy;
            p.stats = c.stats;
        }
        p.zscale = 1.f / c.temperature;
        p.N = L.N;
        p.d = s.d;
        p.V = s.V;
        p.R = L.R;
        p.chunk = chunk;
        p.status = c.status;
        HEAD_LAUNCH(GRPO_PROF_GATHER, launch_head_gather(p, bf16, dev.sm_count, st));
        return GRPO_OK;
    }

    int logits(int chunk, int mode, bool store, const int* only_if = nullptr) {
        const grpo_shape& s = *c.shape;
        LogitsParams p = {};
        p.counts = at<int>(L.counts);
        p.cb = at<int>(L.cb);
        p.rows = at<int>(L.rows);
        p.tokens = c.tokens;
        p.part = at<float4>(L.part);
        p.E = store ? at<uint16_t>(L.ds) : nullptr;
        p.mx = store ? at<float>(L.mx) : nullptr;
        logit_scale(c, &p.zscale, &p.zscale2);
        p.zt = at<double>(L.zt);
        p.only_if = only_if;
        p.N = L.N;
        p.chunk = chunk;
        p.V = s.V;
        p.d = s.d;
        p.plan = at<int2>(L.lg_plan);
        p.n_ntiles = L.n_ntiles;
        p.V_pad = L.V_pad;
        p.nc32 = L.nc32;
        p.R = L.R;
        p.status = c.status;
        HEAD_LAUNCH(GRPO_PROF_FWD, launch_head_logits(p, mH_k, mW_k, dev.sm_count, bf16, mode, st));
        return GRPO_OK;
    }

    HeadMergeParams merge_params(int chunk) const {
        const grpo_shape& s = *c.shape;
        HeadMergeParams p = {};
        p.part = at<float4>(L.part);
        p.plan = at<int2>(L.lg_plan);
        p.counts = at<int>(L.counts);
        p.cb = at<int>(L.cb);
        p.off = at<int>(L.off);
        p.rows = at<int>(L.rows);
        p.tokens = c.tokens;
        p.zt = at<double>(L.zt);
        p.lse2 = at<float2>(L.lse2);
        p.gco = at<float>(L.gco);
        p.ell = c.mode == HEAD_CLIP ? at<float>(L.ell) : nullptr;
        p.gmax = c.backward && !bf16 ? at<unsigned>(L.gmax) : nullptr;
        p.logp = c.logp ? c.logp : at<float>(L.q);
        p.entropy = c.entropy;
        p.dlogp = c.dlogp;
        p.adv = c.adv;
        p.logp_old = c.logp_old;
        p.logp_ref = c.mode == HEAD_CLIP && s.beta != 0.f ? c.logp_ref : nullptr;
        p.stats = c.stats;
        p.beta = s.beta;
        p.clip_lo = 1.f - c.clip.clip_low;
        p.clip_hi = 1.f + c.clip.clip_high;
        p.inv_t = 1.f / c.temperature;
        p.mode = c.mode;
        p.loss_mode = s.loss_mode;
        p.chunk = chunk;
        p.L = s.L;
        p.V = s.V;
        p.R = L.R;
        p.N = L.N;
        p.status = c.status;
        return p;
    }

    // set_far: note the chunk when a row's q is below kLeastQ
    int merge(int chunk, bool relative, const int* only_if, bool set_far) {
        HeadMergeParams p = merge_params(chunk);
        p.relative = relative;
        p.only_if = only_if;
        p.far = set_far ? at<int>(L.far) : nullptr;
        HEAD_LAUNCH(GRPO_PROF_MERGE, launch_head_merge(p, st));
        return GRPO_OK;
    }

    // the pairs of a chunk, or (chunk < 0) all of them
    int pair_coef(int chunk) {
        const grpo_shape& s = *c.shape;
        PairParams p = {};
        p.counts = at<int>(L.counts);
        p.off = at<int>(L.off);
        p.pb = chunk < 0 ? nullptr : at<int>(L.pb);
        p.rows = at<int>(L.rows);
        p.tokens = c.tokens;
        p.logp = c.logp ? c.logp : at<float>(L.q);
        p.logp_ref = c.logp_ref;
        p.gco = c.backward ? at<float>(L.gco) : nullptr;
        p.gmax = c.backward && !bf16 ? at<unsigned>(L.gmax) + (chunk < 0 ? 0 : chunk) : nullptr;
        p.pair_ell = at<double>(L.pair_ell);
        p.pair_stats = c.pair_stats;
        p.beta = s.beta;
        p.smoothing = c.pair.label_smoothing;
        p.kind = c.pair.kind;
        p.length_mean = c.pair.length_mean;
        p.n_pairs = s.n_groups;
        p.chunk = chunk < 0 ? 0 : chunk;
        p.V = s.V;
        p.N = L.N;
        p.status = c.status;
        HEAD_LAUNCH(GRPO_PROF_MERGE, launch_pair_coef(p, st));
        return GRPO_OK;
    }

    LossParams loss() const {
        LossParams l = {};
        l.loss = c.loss;
        if (c.mode == HEAD_PAIR) {
            l.pair_ell = at<double>(L.pair_ell);
            l.n_pairs = c.shape->n_groups;
        } else {
            l.ell = at<float>(L.ell);
        }
        return l;
    }

    // fused: the merge is part of it
    int gradients(int chunk, int gmax_chunk, bool fused = false) {
        const grpo_shape& s = *c.shape;
        HeadChunkParams p = {};
        p.counts = at<int>(L.counts);
        p.cb = at<int>(L.cb);
        p.oscale = at<float>(L.oscale);
        p.rows = at<int>(L.rows);
        p.tokens = c.tokens;
        p.lse2 = at<float2>(L.lse2);
        p.zt = at<double>(L.zt);
        p.gco = at<float>(L.gco);
        p.mx = at<float>(L.mx);
        p.scale = 1.f;
        p.chunk = chunk;
        p.V = s.V;
        p.d = s.d;
        p.V_pad = L.V_pad;
        p.nc32 = L.nc32;
        p.R = L.R;
        p.N = L.N;
        p.dS = at<uint16_t>(L.ds);
        p.dH = static_cast<uint16_t*>(c.dH);
        p.found_inf = c.found_inf;
        p.status = c.status;
        p.mHct = mHct;
        p.loss = loss();
        p.dw_acc = c.dw_f32 ? static_cast<float*>(c.dW) : at<float>(L.dw_acc);
        p.dw16 = c.dw_f32 ? nullptr : static_cast<uint16_t*>(c.dW);
        p.dh_part = at<float>(L.dh_part);
        p.dh_cols = L.dh_cols;
        p.dh_plan = at<int2>(L.dh_plan);
        p.logp = c.logp ? c.logp : at<float>(L.q);
        p.gmax = at<unsigned>(L.gmax);
        p.gmax_chunk = gmax_chunk;
        p.loss_scale = c.loss_scale;
        p.hct = at<uint16_t>(L.hct);
        p.hc = at<uint16_t>(L.hc);
        p.rowf = L.relative ? at<float>(L.rowf) : nullptr;
        p.far = L.relative ? at<int>(L.far) : nullptr;
        if (fused) HEAD_LAUNCH(GRPO_PROF_DLOGITS, launch_merge_dlogits(merge_params(chunk), p, at<float>(L.oscale), dev.sm_count, st));
        else HEAD_LAUNCH(GRPO_PROF_DLOGITS, launch_head_dlogits(p, at<float>(L.oscale), bf16, dev.sm_count, st));
        if (L.relative) HEAD_LAUNCH(GRPO_PROF_DLOGITS, launch_head_scale(p, at<float>(L.oscale), dev.sm_count, st));
        if (L.one_launch) HEAD_LAUNCH(GRPO_PROF_DH, launch_head_grads(p, mDS_k, mDS_mn, mW_mn, dev.sm_count, bf16, st));
        else HEAD_LAUNCH(GRPO_PROF_DH, launch_head_dh(p, mDS_k, mW_mn, dev.sm_count, bf16, st));
        if (L.slots > 0) HEAD_LAUNCH(GRPO_PROF_DH, launch_head_dh_join(p, bf16, dev.sm_count, st));
        if (!L.one_launch) HEAD_LAUNCH(GRPO_PROF_DW, launch_head_dw(p, mDS_mn, dev.sm_count, bf16, st));
        return GRPO_OK;
    }

#define HEAD_STEP(call)                       \
    do {                                      \
        const int rc_ = (call);               \
        if (rc_ != GRPO_OK) return rc_;       \
    } while (0)

    int run() {
        HEAD_STEP(maps());
        HEAD_STEP(plan());
        // a preference loss whose chunks do not hold whole pairs: all log-probs first, then the logits again
        const bool twice = c.mode == HEAD_PAIR && c.backward && !L.by_pair;
        const bool rel = L.relative;
        const int keep = rel ? LG_KEEP_TOKEN : LG_KEEP_MAX;
        // without gradients the same arithmetic, nothing kept: the same bits
        const int stats = rel ? LG_KEEP_TOKEN : c.entropy ? LG_ENTROPY : LG_STATS;
        for (int i = 0; i < L.max_chunks; ++i) {
            const bool grad = c.backward && !twice;
            const int* far = at<int>(L.far) + i;
            HEAD_STEP(gather(i, grad && !rel, i == 0));
            HEAD_STEP(logits(i, grad ? keep : stats, grad));
            if (grad && bf16 && !rel && c.mode != HEAD_PAIR) {
                HEAD_STEP(gradients(i, i, true));
                continue;
            }
            HEAD_STEP(merge(i, rel, nullptr, rel));
            if (rel) {   // only for a chunk with a far row
                HEAD_STEP(logits(i, grad ? LG_KEEP_MAX : LG_STATS, grad, far));
                HEAD_STEP(merge(i, false, far, false));
            }
            if (!grad) continue;
            if (c.mode == HEAD_PAIR) HEAD_STEP(pair_coef(i));
            HEAD_STEP(gradients(i, i));
        }
        if (c.mode == HEAD_PAIR && (twice || !c.backward)) HEAD_STEP(pair_coef(-1));
        for (int i = 0; twice && i < L.max_chunks; ++i) {
            HEAD_STEP(gather(i, !rel, false));
            HEAD_STEP(logits(i, keep, true));
            if (rel) HEAD_STEP(logits(i, LG_KEEP_MAX, true, at<int>(L.far) + i));
            HEAD_STEP(gradients(i, 0));
        }
        if (c.loss && !c.backward) HEAD_LAUNCH(GRPO_PROF_MERGE, launch_loss(loss(), at<int>(L.counts), st));
        return GRPO_OK;
    }
};

int head_call(const HeadCall& c, grpo_stream_t stream) {
    HeadLayout L;
    int rc = head_validate(c, &L);
    if (rc != GRPO_OK) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != GRPO_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (c.mode == HEAD_LOGP && L.N <= kFewRows) return run_few(c, L, dev, st);
    HeadRun run{c, L, dev, st, static_cast<char*>(c.ws), c.shape->dtype == GRPO_BF16, {}, {}, {}, {}, {}, {}};
    return run.run();
}

int clip_check(const HeadCall& c, const grpo_clip_opts* o) {
    if (!c.shape || !o) return GRPO_ERR_SHAPE;
    if (!std::isfinite(c.shape->beta) || c.shape->objective != GRPO_OBJ_GRPO) return GRPO_ERR_SHAPE;
    if (!(o->clip_low >= 0.f) || !(o->clip_low <= 1.f) || !(o->clip_high >= 0.f)) return GRPO_ERR_SHAPE;
    if (!c.adv || !c.logp_old || !c.loss || (c.shape->beta != 0.f && !c.logp_ref)) return GRPO_ERR_POINTER;
    return GRPO_OK;
}

int pair_check(const HeadCall& c, const grpo_pair_opts* o) {
    if (!c.shape || !o) return GRPO_ERR_SHAPE;
    if (!(c.shape->beta > 0.f) || !std::isfinite(c.shape->beta)) return GRPO_ERR_SHAPE;
    if (o->kind < GRPO_PAIR_SIGMOID || o->kind > GRPO_PAIR_SQUARE) return GRPO_ERR_SHAPE;
    if (!(o->label_smoothing >= 0.f) || !(o->label_smoothing < 0.5f)) return GRPO_ERR_SHAPE;
    if (o->kind != GRPO_PAIR_SIGMOID && o->label_smoothing != 0.f) return GRPO_ERR_SHAPE;
    if (!c.logp_ref || !c.loss) return GRPO_ERR_POINTER;
    return GRPO_OK;
}

}  // namespace

}  // namespace grpo

using namespace grpo;

extern "C" {

void grpo_clip_opts_init(grpo_clip_opts* o) {
    if (!o) return;
    std::memset(o, 0, sizeof(*o));
    o->temperature = 1.f;
    o->clip_low = o->clip_high = 0.2f;
}

void grpo_pair_opts_init(grpo_pair_opts* o) {
    if (!o) return;
    std::memset(o, 0, sizeof(*o));
    o->kind = GRPO_PAIR_SIGMOID;
}

size_t grpo_policy_workspace_bytes(const grpo_shape* shape, int op, int dw_f32) {
    if (!shape || !dtype_ok(*shape)) return 0;
    HeadLayout L;
    if (!head_layout(*shape, op, dw_f32, &L)) return 0;
    return L.total;
}

int grpo_logprobs(const void* h, const void* W, const int32_t* tokens, const uint8_t* mask, const grpo_shape* shape,
                  float temperature, void* workspace, size_t ws_bytes, float* logp_out, float* entropy_out,
                  int32_t* status, grpo_stream_t stream) {
    HeadCall c{h, W, tokens, mask, shape, workspace, ws_bytes, status};
    c.temperature = temperature;
    c.logp = logp_out;
    c.entropy = entropy_out;
    if (!logp_out) return shape ? GRPO_ERR_POINTER : GRPO_ERR_SHAPE;
    return head_call(c, stream);
}

int grpo_logprobs_bwd(const void* h, const void* W, const int32_t* tokens, const uint8_t* mask, const float* dlogp,
                      const grpo_shape* shape, float temperature, float loss_scale, int dw_f32, void* workspace,
                      size_t ws_bytes, void* dH, void* dW, int32_t* found_inf, int32_t* status, grpo_stream_t stream) {
    HeadCall c{h, W, tokens, mask, shape, workspace, ws_bytes, status};
    c.op = GRPO_OP_LOGPROBS_BWD;
    c.mode = HEAD_GRAD;
    c.backward = true;
    c.temperature = temperature;
    c.dlogp = dlogp;
    c.loss_scale = loss_scale;
    c.dw_f32 = dw_f32;
    c.dH = dH;
    c.dW = dW;
    c.found_inf = found_inf;
    if (!dlogp) return shape ? GRPO_ERR_POINTER : GRPO_ERR_SHAPE;
    return head_call(c, stream);
}

int grpo_clip_loss_fwd(const void* h, const void* W, const int32_t* tokens, const uint8_t* mask, const float* adv,
                       const float* logp_old, const float* logp_ref, const grpo_shape* shape, const grpo_clip_opts* opts,
                       void* workspace, size_t ws_bytes, float* loss_out, float* row_stats, int32_t* status,
                       grpo_stream_t stream) {
    HeadCall c{h, W, tokens, mask, shape, workspace, ws_bytes, status};
    c.op = GRPO_OP_CLIP;
    c.mode = HEAD_CLIP;
    c.adv = adv;
    c.logp_old = logp_old;
    c.logp_ref = logp_ref;
    c.loss = loss_out;
    c.stats = row_stats;
    const int rc = clip_check(c, opts);
    if (rc != GRPO_OK) return rc;
    c.clip = *opts;
    c.temperature = opts->temperature;
    c.dw_f32 = opts->dw_f32;
    return head_call(c, stream);
}

int grpo_clip_loss_fwd_bwd(const void* h, const void* W, const int32_t* tokens, const uint8_t* mask, const float* adv,
                           const float* logp_old, const float* logp_ref, const grpo_shape* shape,
                           const grpo_clip_opts* opts, float loss_scale, void* workspace, size_t ws_bytes, float* loss_out,
                           void* dH, void* dW, int32_t* found_inf, float* row_stats, int32_t* status,
                           grpo_stream_t stream) {
    HeadCall c{h, W, tokens, mask, shape, workspace, ws_bytes, status};
    c.op = GRPO_OP_CLIP;
    c.mode = HEAD_CLIP;
    c.backward = true;
    c.adv = adv;
    c.logp_old = logp_old;
    c.logp_ref = logp_ref;
    c.loss = loss_out;
    c.stats = row_stats;
    c.loss_scale = loss_scale;
    c.dH = dH;
    c.dW = dW;
    c.found_inf = found_inf;
    const int rc = clip_check(c, opts);
    if (rc != GRPO_OK) return rc;
    c.clip = *opts;
    c.temperature = opts->temperature;
    c.dw_f32 = opts->dw_f32;
    return head_call(c, stream);
}

int grpo_pair_loss_fwd(const void* h, const void* W, const int32_t* tokens, const uint8_t* mask, const float* logp_ref,
                       const grpo_shape* shape, const grpo_pair_opts* opts, void* workspace, size_t ws_bytes,
                       float* loss_out, float* logp_out, float* pair_stats, int32_t* status, grpo_stream_t stream) {
    HeadCall c{h, W, tokens, mask, shape, workspace, ws_bytes, status};
    c.op = GRPO_OP_PAIR;
    c.mode = HEAD_PAIR;
    c.logp_ref = logp_ref;
    c.loss = loss_out;
    c.logp = logp_out;
    c.pair_stats = pair_stats;
    const int rc = pair_check(c, opts);
    if (rc != GRPO_OK) return rc;
    c.pair = *opts;
    c.dw_f32 = opts->dw_f32;
    return head_call(c, stream);
}

int grpo_pair_loss_fwd_bwd(const void* h, const void* W, const int32_t* tokens, const uint8_t* mask, const float* logp_ref,
                           const grpo_shape* shape, const grpo_pair_opts* opts, float loss_scale, void* workspace,
                           size_t ws_bytes, float* loss_out, void* dH, void* dW, int32_t* found_inf, float* logp_out,
                           float* pair_stats, int32_t* status, grpo_stream_t stream) {
    HeadCall c{h, W, tokens, mask, shape, workspace, ws_bytes, status};
    c.op = GRPO_OP_PAIR;
    c.mode = HEAD_PAIR;
    c.backward = true;
    c.logp_ref = logp_ref;
    c.loss = loss_out;
    c.logp = logp_out;
    c.pair_stats = pair_stats;
    c.loss_scale = loss_scale;
    c.dH = dH;
    c.dW = dW;
    c.found_inf = found_inf;
    const int rc = pair_check(c, opts);
    if (rc != GRPO_OK) return rc;
    c.pair = *opts;
    c.dw_f32 = opts->dw_f32;
    return head_call(c, stream);
}

}  // extern "C"
