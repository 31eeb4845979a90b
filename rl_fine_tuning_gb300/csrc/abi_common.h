// Host-side helpers that the entry points of every translation unit share.
#pragma once
#include <atomic>
#include <mutex>
#include <vector>

#include "internal.h"

namespace grpo {

// ---- launch accounting and optional per-kernel event timing
extern std::atomic<unsigned long long> g_launches;

struct ProfRecord {
    int kind;
    cudaEvent_t a, b;
};

// `on` is read by every launch; the records and the event pool are touched
// only while profiling is on, under `mu`.
struct Profiler {
    std::atomic<bool> on{false};
    std::mutex mu;
    std::vector<ProfRecord> recs;
    std::vector<cudaEvent_t> pool;
    cudaEvent_t get() {
        if (!pool.empty()) {
            cudaEvent_t e = pool.back();
            pool.pop_back();
            return e;
        }
        cudaEvent_t e = nullptr;
        if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
        return e;
    }
};
extern Profiler g_prof;

// launch one kernel through `fn`, counting it and timing it when profiling is on
template <class F>
cudaError_t launch(int kind, cudaStream_t st, F&& fn) {
    if (!g_prof.on.load(std::memory_order_relaxed)) {
        const cudaError_t e = fn();
        if (e == cudaSuccess) g_launches.fetch_add(1, std::memory_order_relaxed);
        return e;
    }
    std::lock_guard<std::mutex> lock(g_prof.mu);
    cudaEvent_t a = g_prof.get(), b = g_prof.get();
    if (a) cudaEventRecord(a, st);
    const cudaError_t e = fn();
    if (e == cudaSuccess) g_launches.fetch_add(1, std::memory_order_relaxed);
    if (a && b) {
        cudaEventRecord(b, st);
        g_prof.recs.push_back(ProfRecord{kind, a, b});
    }
    return e;
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

template <class P>
bool aligned(const P* p, size_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

struct DeviceInfo {
    int sm_count = 0;
    bool ok = false;
};

int device_info(DeviceInfo* out);
bool shape_ok(const grpo_shape& s);
inline bool dtype_ok(const grpo_shape& s) { return s.dtype == GRPO_BF16 || s.dtype == GRPO_FP16; }


// 2-D row-major matrix [rows x cols] of 16-bit elements with row pitch `pitch`
// elements, 128-byte swizzled boxes of box_cols x box_rows.
bool make_map(CUtensorMap* m, const void* base, bool bf16, uint64_t cols, uint64_t rows, uint64_t pitch,
              uint32_t box_cols, uint32_t box_rows);

}  // namespace grpo
