// Host helpers of the entry points: status reporting, argument checks that
// several of them share, and the range a profiler sees around a call.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include "qsa_internal.cuh"

#define QSA_API extern "C" __attribute__((visibility("default")))

namespace qsa {

// An NVTX range around each call that enqueues work (named after the entry
// point): a profiler attributes the call's launches to the QSA step they
// serve.  Without a profiler attached the push and pop are no-ops.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// Set this thread's error text and return the status.
qsa_status fail(qsa_status s, const char* fmt, ...);
qsa_status ok();
qsa_status cuda_fail(cudaError_t e, const char* where);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool quantized(int d) { return d == QSA_FP8_E4M3 || d == QSA_Q8_0; }
inline size_t dtype_size(qsa_dtype d) { return d == QSA_F32 ? 4 : quantized(d) ? 1 : 2; }
inline bool valid_dtype(int d) { return d == QSA_F32 || d == QSA_BF16; }
// K/V state types: the value types plus the quantized states.
inline bool valid_kv_dtype(int d) { return valid_dtype(d) || quantized(d); }
inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

qsa_status check_attn_config(const qsa_attn_config* cfg, const char* fn);

}  // namespace qsa
