// How the norm's rows are dealt to threads and blocks.
#include "norm.h"

namespace grpo {

namespace {

// the row's threads, and their units; rows of up to `most` units take some lanes of a warp
NormPlan row_plan(int d, int most, bool two) {
    NormPlan o;
    const int n_unit = d / kUnit;
    o.wide = n_unit > most;
    if (!o.wide) {
        o.width = n_unit <= 4 ? 4 : n_unit <= 8 ? 8 : n_unit <= 16 ? 16 : 32;
        o.upt = (n_unit + o.width - 1) / o.width;
        o.threads = kWarpThreads;
    } else {
        o.upt = n_unit > kBlockMax || two ? 2 : 1;
        o.threads = o.width = (n_unit + 32 * o.upt - 1) / (32 * o.upt) * 32;
    }
    return o;
}

}  // namespace

// A block goes through at least 8 turns of rows, in whole waves of blocks: with many rows, blocks that
// come and go keep the rows that are worked on near one another in memory.  160,000 rows of 4096 with the
// residual: 661 us with one wave, 595 with 8, 589 with 16; 10,000 rows to 8 bits: 41 us with 8 turns a
// block or more, 42 with 4, 46 with 2, 57 with one.
NormPlan norm_fwd_plan(int64_t N, int d, int sm_count) {
    NormPlan o = row_plan(d, 64, false);
    const int64_t rows = o.threads / o.width, turns = (N + rows - 1) / rows;
    o.per_sm = (o.upt == 1 ? 1024 : 512) / o.threads;
    const int64_t once = static_cast<int64_t>(o.per_sm) * sm_count, waves = turns / 8 / once;
    o.grid = static_cast<int>(turns < once ? turns : waves > 1 ? waves * once : once);
    return o;
}

// Two units a thread where a block of one would fill an SM (d > 6144), and from a checkpoint, whose codes cost
// instructions, where that leaves no thread without one (160,000 x 4096, 54% of the rows: 373 against 388 us).
// Of wide rows an SM takes as many blocks as bring its copies under way, two rows a block, to 60 KB and 9/4 of a row (64
// with a checkpoint, 16 more with dsum); no block has less than one.  These numbers are fitted to the times that follow, and
// another machine or kernel would want others: 40,000 rows of 4096: 162 us with 64 KB, 149 with 96, 163 with 144; 80,000 of 2048:
// 170 with 48 KB, 153 with 64, 164 with 96; 160,000 of 1024: 149 with 64 KB, 162 with 80; 284,444 of 576: 255 with 36 KB,
// 226 with 54.  With dsum, or from a checkpoint, where instructions count too, more does less harm; and rows that leave
// threads without elements take longer and need more of them (131,072 of 1280: 171 us with 6 blocks, 159 with 8).
NormPlan norm_bwd_plan(int64_t N, int d, int sm_count, bool ckpt, bool dsum) {
    const bool two = d / kUnit > 384 || (ckpt && !dsum && d / kUnit % 64 == 0 && N >= 64LL * sm_count);
    NormPlan o = row_plan(d, 32, two);
    const int64_t rows = o.threads / o.width, turns = (N + rows - 1) / rows;
    if (o.wide) {
        const int row = d * (2 + (ckpt ? 1 : 2) + (dsum ? 2 : 0)), most = (o.upt == 1 ? 768 : 512) / o.threads;
        const int64_t room = (60 + 4 * ckpt + 16 * dsum) * 1024 + row * 9 / 4;
        o.per_sm = static_cast<int>(room * (o.width * o.upt * kUnit) / (2LL * row * d));
        if (o.per_sm > most) o.per_sm = most;
        if (o.per_sm < 1) o.per_sm = 1;
    } else {
        o.per_sm = 5;                          // what 96 registers a thread leave: 155 us; 4 take 167, 6 in two waves 200
    }
    const int64_t grid = static_cast<int64_t>(o.per_sm) * sm_count;
    o.grid = static_cast<int>(turns < grid ? turns : grid);
    // One cluster of blocks joins its sums itself, even if that takes a second turn of rows: 256 rows of 128 in one
    // launch of 3.8 us instead of two with 4.9 (7.2 against 8.9 with their host calls).
    o.joined = turns <= 2 * kClusterMax;
    if (o.joined) {
        const int want = turns < kClusterMax ? static_cast<int>(turns) : kClusterMax;
        for (o.grid = 1; o.grid < want;) o.grid *= 2;
    }
    return o;
}

int norm_parts(int64_t N, int d) {
    int most = 0;
    for (int i = 0; i < 4; ++i) {
        const NormPlan o = norm_bwd_plan(N, d, kSmCount, i & 1, i & 2);
        if (o.grid > most) most = o.grid;
    }
    return most;
}

}  // namespace grpo
