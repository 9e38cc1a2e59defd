// Host helpers shared by the C ABI's translation units.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#define MOE_API extern "C" __attribute__((visibility("default")))

// NVTX range over one entry point (host side; shows each call in profiler
// timelines, does nothing when no profiling tool is attached).
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

// Device-side waits give up after this many SM clocks (about one second).
static const long long kTimeoutCycles = 2000000000LL;

static inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

static inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

static inline bool finite_f32(float v) { return v - v == 0.f; }
