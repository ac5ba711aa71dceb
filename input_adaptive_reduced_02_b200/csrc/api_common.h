// What the files that define C ABI entry points share. Defined in api.cu.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include "../../include/rmm.h"
#include "rmm_internal.h"

namespace rmm {

// A named NVTX range around one stage of a call, so that a profiler's
// timeline (or an ncu --nvtx filter) shows score, select, pack and the product
// by name; header-only NVTX costs a branch when no tool is attached.
struct StageRange {
  explicit StageRange(const char* name) { nvtxRangePushA(name); }
  ~StageRange() { nvtxRangePop(); }
  StageRange(const StageRange&) = delete;
  StageRange& operator=(const StageRange&) = delete;
};

// Record the thread's error message and return s.
rmm_status fail(rmm_status s, const char* fmt, ...);
rmm_status cuda_fail(cudaError_t e, const char* what, const char* why = nullptr);

// Make the stream's device current for the rest of the call (the caller's
// framework may have made another device current); `g` puts the caller's
// device back when the entry point returns.
rmm_status bind_device(cudaStream_t st, DeviceGuard& g);

// Debug mode, after a fused call: wait for it and return its device status.
rmm_status debug_call_status(uint32_t* status, cudaStream_t st);

inline bool dtype_ok(rmm_dtype d) { return d == RMM_BF16 || d == RMM_F32; }
inline ElemKind kind(rmm_dtype d) { return d == RMM_BF16 ? kBF16 : kF32; }

// The error a device status word stands for (RMM_OK if no bit is set).
rmm_status status_error(uint32_t word);

// Slices per selection: the select kernel indexes keys with 32-bit integers
// and re-reads them from global memory beyond 32768; 2^21 bounds its work.
constexpr int64_t kMaxSelectK = int64_t(1) << 21;

}  // namespace rmm
