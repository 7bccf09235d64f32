// What the translation units of the C ABI share: the RoPE handle, alignment
// helpers and the per-call NVTX range.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include "../../include/medusa_tree.h"
#include "kernels.cuh"

// One NVTX range per library call, named after its C entry point, for a
// timeline tool (nothing is recorded unless such a tool is attached).
struct mt_call_range {
  explicit mt_call_range(const char* name) { nvtxRangePushA(name); }
  ~mt_call_range() { nvtxRangePop(); }
  mt_call_range(const mt_call_range&) = delete;
  mt_call_range& operator=(const mt_call_range&) = delete;
};

struct mt_rope {
  float2* table;  // [max_pos][D/2] (cos, sin)
  int head_dim;
  int max_pos;
  int device;
};

namespace mt {

constexpr size_t kAlign = 256;
constexpr int kMaxBatch = 8192;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Of 32-bit arrays; a null pointer is aligned.
template <typename... P>
inline bool aligned4(const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) % 4 == 0) && ...);
}

// The bound of the tensor-core kernels' waits and the timeout test hook, as
// mt_debug_set_wait left them.
void wait_bound(unsigned long long* limit_ns, int* stall);

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? MT_OK : MT_ERR_CUDA; }

}  // namespace mt
