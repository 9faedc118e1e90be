// api.cuh -- what the C entry points share: error reporting, argument checks, the device's SM count.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/prism.h"

namespace prism {

// PRISM_OK, or PRISM_ERR_CUDA with `err` kept for prism_last_cuda_error.
prism_status cuda_status(cudaError_t err);

// Records the launch probe's last event after a probed call's final launch and disarms the probe.
void probe_finish(cudaStream_t s);

// SMs of the current device (148 where there is none).
int sm_count();

// The process-wide flags of prism_debug_set_flags.
int debug_flags();

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool width_ok(int d) { return d == 32 || d == 64 || d == 128; }

// `n` bytes at `p` (nothing where p is null or n is 0).
struct ByteRange {
    const void *p;
    size_t n;
};

inline bool ranges_overlap(const ByteRange &a, const ByteRange &b) {
    return a.p && b.p && a.n && b.n && (const char *)a.p < (const char *)b.p + b.n &&
           (const char *)b.p < (const char *)a.p + a.n;
}

// Whether an output overlaps another output or an input.
inline bool outputs_alias(const ByteRange *outs, int n_outs, const ByteRange *ins, int n_ins) {
    for (int i = 0; i < n_outs; ++i) {
        for (int j = i + 1; j < n_outs; ++j)
            if (ranges_overlap(outs[i], outs[j])) return true;
        for (int j = 0; j < n_ins; ++j)
            if (ranges_overlap(outs[i], ins[j])) return true;
    }
    return false;
}

}  // namespace prism
