// Shared pieces of the streaming-block operators (quant_linear.cu, short_conv.cu,
// selective_scan.cu, residual_norm.cu): element types, activations and the
// checks that every call makes before its launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <string>

#include "../../include/gam.h"
#include "common.cuh"

namespace gam {
namespace ops {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float v) { return __float2bfloat16_rn(v); }

// V consecutive elements, moved by accesses of 16 bytes (fewer if they are smaller).
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Vec {
  T v[V];
};

__device__ __forceinline__ float sigmoid_f(float v) { return 1.f / (1.f + __expf(-v)); }
__device__ __forceinline__ float swish_f(float v) { return v / (1.f + __expf(-v)); }

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case GAM_ACT_SWISH: return swish_f(v);
    case GAM_ACT_SIGMOID: return sigmoid_f(v);
    case GAM_ACT_TANH: return tanhf(v);
    default: return v;
  }
}

// --- host side -----------------------------------------------------------------

inline gam_status op_fail(gam_status s, const std::string& msg) {
  set_context_free_error(msg);
  return s;
}
inline bool is_float_dtype(int t) { return t == GAM_DTYPE_F32 || t == GAM_DTYPE_F16 || t == GAM_DTYPE_BF16; }
inline int dtype_size(int t) { return t == GAM_DTYPE_F32 ? 4 : 2; }
inline bool aligned(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Whether the rows of an output [batch, t, d] lie apart: sequence after sequence,
// or frame after frame.
inline bool rows_apart(int64_t batch, int64_t t, int64_t d, int64_t batch_stride, int64_t row_stride) {
  if (batch <= 1) return t <= 1 || row_stride >= d;
  if (t <= 1) return t == 0 || batch_stride >= d;
  if (batch_stride < d || row_stride < d) return false;
  return (batch_stride - d) / (t - 1) >= row_stride || (row_stride - d) / (batch - 1) >= batch_stride;
}

// Runs an entry point's body; an exception (out of host memory) becomes a status.
template <typename F>
gam_status guarded(F&& body) noexcept {
  try {
    set_context_free_error("");
    return body();
  } catch (...) {
    return GAM_ERR_INVALID_ARG;
  }
}

// The current device is a B200 (its number of SMs in *sms); cached per device.
gam_status check_device(int* sms);
// Status of the launches made since the call's checks.
gam_status launch_status(cudaError_t e);

}  // namespace ops
}  // namespace gam
