// Host-side helpers shared by the C ABI's translation units: the calling thread's error
// message, status macros, TMA descriptors and launches.
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <utility>

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "../../include/sla.h"

namespace sla_host {

// The calling thread's last failure (a fixed buffer: recording a message never throws).
inline char (&last_error())[512] {
  static thread_local char buf[512] = "";
  return buf;
}

inline sla_status fail(sla_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(last_error(), sizeof(last_error()), fmt, ap);
  va_end(ap);
  return st;
}

#define SLA_CUDA(call)                                                                     \
  do {                                                                                     \
    cudaError_t e_ = (call);                                                               \
    if (e_ != cudaSuccess) return fail(SLA_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_)); \
  } while (0)

#define SLA_TRY(x)                 \
  do {                             \
    sla_status st_ = (x);          \
    if (st_ != SLA_OK) return st_; \
  } while (0)

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

inline bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) % 16) == 0; }

// Whether the rows of D elements of an output [B, heads, N, D] lie apart: in ascending order, each stride over
// an extent above 1 passes what lies within it. (Rows that meet would be written by several blocks at once, and
// in place read by some after others have written them.)
inline bool rows_apart(const sla_tensor* t, int B, int heads, int N, int D) {
  const int64_t given[3] = {t->stride_b, t->stride_h, t->stride_n};
  const int extent[3] = {B, heads, N};
  unsigned __int128 span = D, last = 0;
  for (int done = 0; done < 3; ++done) {  // the smallest stride not yet taken
    int at = -1;
    unsigned __int128 stride = 0;
    for (int d = 0; d < 3; ++d) {
      const unsigned __int128 s = static_cast<unsigned __int128>(given[d] < 0 ? -static_cast<__int128>(given[d]) : given[d]) * 4 + d;
      if (extent[d] > 1 && (done == 0 || s > last) && (at < 0 || s < stride)) at = d, stride = s;
    }
    if (at < 0) return true;
    last = stride;
    if (stride / 4 < span) return false;
    span += stride / 4 * (extent[at] - 1);
  }
  return true;
}

// ------------------------------------------------------------------ TMA descriptors

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Tensor map with 128-byte swizzle (bf16, or uint8 for e4m3 codes). dims/strides in
// elements (innermost first).
inline sla_status make_map(CUtensorMap* m, const void* ptr, int rank, const uint64_t* dims, const uint64_t* strides_el,
                           const uint32_t* box, bool u8 = false) {
  auto fn = encode_fn();
  if (!fn) return fail(SLA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t d[5], st[4];
  cuuint32_t b[5], es[5];
  for (int r = 0; r < rank; ++r) {
    d[r] = dims[r];
    b[r] = box[r];
    es[r] = 1;
  }
  for (int r = 0; r + 1 < rank; ++r) st[r] = strides_el[r] * (u8 ? 1 : 2);
  CUresult res = fn(m, u8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), d, st, b, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (res != CUDA_SUCCESS) return fail(SLA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(res));
  return SLA_OK;
}

// ------------------------------------------------------------------ launches

inline int sm_count() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

template <typename K>
sla_status allow_smem(K kernel, int bytes) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return fail(SLA_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  return SLA_OK;
}

// Launch `kernel` as a programmatic dependent of the previous kernel in the stream: it may
// be scheduled while the predecessor drains and waits (griddepcontrol.wait) before
// reading the predecessor's results.
template <typename... KArgs, typename... Args>
sla_status launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                            const char* what, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  if (e != cudaSuccess) return fail(SLA_ERR_CUDA, "launch of %s failed: %s", what, cudaGetErrorString(e));
  return SLA_OK;
}

inline sla_status launched(const char* what) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SLA_ERR_CUDA, "launch of %s failed: %s", what, cudaGetErrorString(e));
  return SLA_OK;
}

}  // namespace sla_host
