// host_common.h - host-side pieces shared by the library's translation units (caat_api.cu: the
// row-parallel layer; attn_api.cu: the attention block).  Internal; not part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <vector>

#include "caat.h"

// ---------------------------------------------------------------------------------------
// Timing recorder
// ---------------------------------------------------------------------------------------
struct caat_timing {
  int capacity = 0;
  int max_kernels = 8;
  int n = 0;
  std::vector<cudaEvent_t> ev;
  std::vector<int> nk;
};

namespace caat {
namespace host {

struct Recorder {
  caat_timing* t = nullptr;
  int rec = -1;
  int k = 0;
  void begin(caat_timing* tm, cudaStream_t s) {
    t = tm;
    if (!t || t->n >= t->capacity) {
      t = nullptr;
      return;
    }
    rec = t->n++;
    k = 0;
    cudaEventRecord(t->ev[rec * (t->max_kernels + 1)], s);
  }
  void after_kernel(cudaStream_t s) {
    if (!t || k >= t->max_kernels) return;
    ++k;
    cudaEventRecord(t->ev[rec * (t->max_kernels + 1) + k], s);
    t->nk[rec] = k;
  }
};

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Defined in caat_api.cu: the current device's SM count (CAAT_ERR_UNSUPPORTED unless sm_100), its
// context, the limit of device-side waits and the driver's tensor-map encoder (null if absent).
caat_status device_sms(int* sm_count);
CUcontext context();
uint64_t wait_limit_ns();
EncodeTiledFn tensor_map_encoder();

// Defined in attn_api.cu: reads and clears that translation unit's device status word (each unit
// of a library built without relocatable device code has its own); false on a CUDA error.
bool attn_take_status(int* v);

}  // namespace host
}  // namespace caat
