// Host helpers shared by the C-ABI sources: argument checks and NVTX ranges.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include <initializer_list>

#include "common.cuh"

namespace fdllm {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// An NVTX range around each entry point, so that a profiler's timeline shows
// which call launched which kernels (a no-op when no tool is attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

inline fdllm_status check_ws(void* ws, size_t bytes, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || bytes < need)
    return FDLLM_ERR_WORKSPACE;
  return FDLLM_OK;
}

inline fdllm_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FDLLM_OK : FDLLM_ERR_CUDA; }

inline char* ws_at(void* ws, size_t off) { return static_cast<char*>(ws) + off; }

inline bool all_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p || !aligned16(p)) return false;
  return true;
}

}  // namespace fdllm
