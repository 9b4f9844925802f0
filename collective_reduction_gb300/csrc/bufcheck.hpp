// Checks of the caller's rank buffers before any kernel may touch them, and
// the trace range every launching entry point opens.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include <cstdint>
#include <vector>

#include "ar.h"

namespace ar {

// An NVTX range over one C-ABI call, seen by profilers that attach an NVTX
// tool (a no-op function call otherwise).
struct TraceRange {
    explicit TraceRange(const char* name) { nvtxRangePushA(name); }
    ~TraceRange() { nvtxRangePop(); }
    TraceRange(const TraceRange&) = delete;
    TraceRange& operator=(const TraceRange&) = delete;
};

// P pointers to n elements of es bytes each.  Always checked: non-null,
// aligned to the element size, pairwise disjoint address ranges.  With
// `residency` also: each pointer is device memory of `device` (or managed
// memory) according to cudaPointerGetAttributes, and its n elements lie
// inside the allocation that holds it (cuMemGetAddressRange; skipped where the
// driver cannot report the range).  Launches nothing.  *aligned16 is set when
// every pointer is 16-byte aligned.  AR_ERR_INVALID_ARG on any failure.
ar_status check_rank_buffers(int P, uint64_t n, int es, int device, void* const* bufs, bool residency,
                             bool* aligned16);

// A buffer of `bytes` bytes of es-byte elements.
struct Span {
    const void* p;
    uint64_t bytes;
    int es;
};

// The same checks for buffers of unlike sizes: each non-null, aligned to its
// element size, resident on `device` with its bytes inside its allocation,
// and all pairwise disjoint.  A span of no bytes is not looked at.
ar_status check_spans(const std::vector<Span>& spans, int device);

// Bytes from a matrix's first element to behind its last: `rows` rows of `width`
// es-byte elements, `stride` >= width elements apart.  kTooManyBytes instead of
// 2^62 or more, so that nothing wraps.
constexpr uint64_t kTooManyBytes = ~0ull;
constexpr uint64_t matrix_bytes(uint64_t rows, uint64_t width, uint64_t stride, uint64_t es) {
    if (rows == 0 || width == 0) return 0;
    const uint64_t most = (1ull << 62) / es;  // elements
    if (width >= most || (rows > 1 && (rows - 1) > (most - 1 - width) / stride)) return kTooManyBytes;
    return ((rows - 1) * stride + width) * es;
}

// Device (or managed) memory of `device` that holds `bytes` bytes from p on.
bool device_resident(const void* p, uint64_t bytes, int device);

}  // namespace ar
