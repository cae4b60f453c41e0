// Host state and helpers shared by the files that implement the C ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "dense_gemm.h"

struct gemm_handle_s {
    int forced_variant;  // -1: automatic selection
    int last_variant;
    int stream_k_mode;   // -1: automatic, 0: never, 1: whenever the variant and workspace allow
    int last_stream_k;   // stream-K workgroups of the last call (0: data-parallel)
    void* ws;            // caller-owned device workspace for stream-K, or null
    size_t ws_bytes;
    int sk_spin;         // polls a stream-K finisher spends on each contributor
    int log;             // GEMM_LOG: one line per call on stderr
    int fail_launch;     // GEMM_DEBUG_FAIL_LAUNCH: report GEMM_ERR_HIP instead of launching
    int forced_rows;     // row-tile height the ragged calls take (0: automatic)
    int forced_nth;      // ... and which of the tiles of that height
    gemm_group_launch_t last_group;  // ... and the last one took (rows 0: none)
};

namespace dg {

// Compute units of the current device, or of the planning model.
int device_cus();

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned_to(const void* p, int64_t bytes)
{
    return (reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes) == 0;
}

inline bool ranges_overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

// Memory that a call reads or writes (p NULL or no bytes: none).
struct MemoryRange {
    const void* p;
    int64_t bytes;
};
// Whether one of the first `written` of n ranges overlaps another one.
template <int N>
bool written_overlap(const MemoryRange (&r)[N], int written)
{
    for (int i = 0; i < written; ++i)
        for (int j = i + 1; j < N; ++j)
            if (r[i].p && r[j].p && r[i].bytes > 0 && r[j].bytes > 0 &&
                ranges_overlap(r[i].p, r[i].bytes, r[j].p, r[j].bytes))
                return true;
    return false;
}

}  // namespace dg
