// Host-side pieces that every C-ABI entry point uses: the trace range, element
// sizes, footprints and overlaps, group checks, and the per-device queries.
#pragma once

#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "ptoc.h"
#include "ptoc_internal.h"

namespace ptoc {

// A named NVTX range around the host side of every entry point (checks and
// launches), so that timeline tools show the library's calls by name. With
// no tool attached a range costs a few nanoseconds.
struct TraceRange {
    explicit TraceRange(const char* name) { nvtxRangePushA(name); }
    ~TraceRange() { nvtxRangePop(); }
    TraceRange(const TraceRange&) = delete;
    TraceRange& operator=(const TraceRange&) = delete;
};

inline int elem_size(int dtype)
{
    switch (dtype) {
    case PTOC_F32: case PTOC_I32: return 4;
    case PTOC_F16: case PTOC_BF16: return 2;
    default: return 0;
    }
}

inline bool valid_dtype(int dtype) { return elem_size(dtype) != 0; }

// Byte range [lo, hi) a buffer occupies.
struct Range {
    uintptr_t lo, hi;
};

inline bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

// Footprint in bytes of a [rows, cols] box with pitch ld, or -1 on overflow.
inline int64_t footprint(int64_t rows, int64_t cols, int64_t ld, int eb)
{
    if (rows == 0 || cols == 0) return 0;
    const int64_t lim = INT64_MAX / 8;
    if (rows > lim / (ld > 0 ? ld : 1)) return -1;
    const int64_t elems = (rows - 1) * ld + cols;
    if (elems > lim / eb) return -1;
    return elems * eb;
}

inline ptoc_status check_group(const ptoc_group* g, bool need_root)
{
    if (!g || !g->tensors) return PTOC_ERR_INVALID_ARG;
    if (g->nranks < 1 || g->nranks > kMaxRanks) return PTOC_ERR_INVALID_ARG;
    if (need_root && (g->root < 0 || g->root >= g->nranks)) return PTOC_ERR_INVALID_ARG;
    for (int r = 0; r < g->nranks; ++r)
        if (!g->tensors[r]) return PTOC_ERR_INVALID_ARG;
    return PTOC_OK;
}

inline bool aligned(const void* p, int eb) { return ((uintptr_t)p % (uintptr_t)eb) == 0; }

// Shared checks of the calls with several outputs: `writes` are the spans the
// call writes, `reads` the ones it only reads; outputs must not overlap
// anything, inputs may overlap each other.
struct Span {
    const void* p;
    uintptr_t bytes;
};

inline ptoc_status check_disjoint_outputs(const Span* writes, int nw, const Span* reads, int nr)
{
    for (int a = 0; a < nw; ++a) {
        const Range ra{(uintptr_t)writes[a].p, (uintptr_t)writes[a].p + writes[a].bytes};
        for (int b = a + 1; b < nw; ++b) {
            const Range rb{(uintptr_t)writes[b].p, (uintptr_t)writes[b].p + writes[b].bytes};
            if (overlap(ra, rb)) return PTOC_ERR_ALIAS;
        }
        for (int b = 0; b < nr; ++b) {
            const Range rb{(uintptr_t)reads[b].p, (uintptr_t)reads[b].p + reads[b].bytes};
            if (overlap(ra, rb)) return PTOC_ERR_ALIAS;
        }
    }
    return PTOC_OK;
}

// The current device's ordinal (0 when it cannot be read) and its SM count
// (cached per device).
int current_device();
int sm_count();

// cuTensorMapEncodeTiled, reached through the runtime's driver entry point
// (the library links no driver library); null if the driver lacks it.
using TensorMapEncoder = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                      const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                      CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The encoder, looked up once; null if the driver lacks it.
TensorMapEncoder tensor_map_encoder();

}  // namespace ptoc
