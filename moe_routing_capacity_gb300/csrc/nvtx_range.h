// nvtx_range.h -- one NVTX range per C-ABI compute call (a no-op unless a
// profiler attaches), so that profiler timelines group each call's kernels
// under its name.
#pragma once

#include <nvtx3/nvToolsExt.h>

namespace {
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};
}  // namespace
#define MOE_NVTX_RANGE() NvtxRange moe_nvtx_range_(__func__)
