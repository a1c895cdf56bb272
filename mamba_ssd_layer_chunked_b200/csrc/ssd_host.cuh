// ssd_host.cuh -- host-side helpers shared by the translation units that
// implement C-ABI entry points. Not part of the C ABI.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include "ssd_common.cuh"

namespace ssd {

// An NVTX range around the host-side enqueue of one entry point or one kernel
// launch, named after it ("ssd_fwd", "fused_scan", ...): a profiler attaches
// the kernels launched inside a range to its name (Nsight Systems' timeline,
// `ncu --nvtx --nvtx-include`). With no tool attached a push or pop costs one
// check of a function pointer.
struct TraceRange {
    explicit TraceRange(const char* name) { nvtxRangePushA(name); }
    ~TraceRange() { nvtxRangePop(); }
    TraceRange(const TraceRange&) = delete;
    TraceRange& operator=(const TraceRange&) = delete;
};

// The status of a CUDA error; keeps its text for ssd_last_cuda_error_string.
ssd_status cuda_status(cudaError_t e);

// SSD_OK when the current device can run this build (see the definition).
ssd_status check_device();

}  // namespace ssd
