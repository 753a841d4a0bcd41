// Shared pieces of the streaming-block operators (quant_linear.cu, short_conv.cu,
// selective_scan.cuh, residual_norm.cu): element types, activations and the
// checks that every call makes before its launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <string>
#include <type_traits>
#include <utility>

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

// Packed fp32 (sm_100 f32x2): a 64-bit register holds two values, one instruction does both.
using u64 = unsigned long long;

__device__ __forceinline__ u64 pack2(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(u64 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 both(float v) { return pack2(v, v); }

// V values as they lie in memory.  A load waits for nothing and converts nothing, so
// that a thread can have many of them on their way; get(k) converts value k.
template <typename T, int V>
struct Raw {
  static constexpr int BYTES = V * sizeof(T), N = BYTES >= 4 ? BYTES / 4 : 1;
  static_assert(BYTES <= 8 || BYTES % 16 == 0, "one value, a pair, or whole 16-byte accesses");
  uint32_t w[N];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (BYTES < 4) {
      w[0] = *reinterpret_cast<const unsigned short*>(p);
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (BYTES == 8) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      w[0] = q.x, w[1] = q.y;
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (BYTES < 4) {
      *reinterpret_cast<unsigned short*>(p) = (unsigned short)w[0];
    } else if constexpr (BYTES == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
  __device__ __forceinline__ float get(int k) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[k]);
    } else {
      const uint32_t u = w[k / 2];
      if constexpr (std::is_same_v<T, bf16>) return __uint_as_float((k & 1) ? u & 0xffff0000u : u << 16);
      else return __half2float(__ushort_as_half((unsigned short)((k & 1) ? u >> 16 : u)));
    }
  }
  __device__ __forceinline__ void set(const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(v[i]);
    } else if constexpr (V == 1) {
      const T t = from_f<T>(v[0]);
      w[0] = *reinterpret_cast<const unsigned short*>(&t);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        if constexpr (std::is_same_v<T, bf16>) {
          const __nv_bfloat162 q = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&q);
        } else {
          const __half2 q = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&q);
        }
      }
    }
  }
};

__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ u64 exp2_approx2(u64 v) {
  const float2 e = unpack2(v);
  return pack2(exp2_approx(e.x), exp2_approx(e.y));
}
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// v between -bound and bound; NaN stays.  A negative bound gives the negated value.
__device__ __forceinline__ float bound_f(float v, float bound) {
  float r;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(bound));
  return r;
}

// e^v for two values in -200 .. 200, off by 6 u (u = 2^-24): 2^t by the hardware (4 u), t = v log2 e rounded, and
// what the rounding left of v, v - t ln 2 with ln 2 in two parts (Cody and Waite's reduction), as a factor 1 + d.
// The rounded t alone would be off by |v| u.
__device__ __forceinline__ u64 exp2v(u64 v) {
  const u64 t = mul2(v, both(1.4426950408889634f));
  const u64 d = fma2(t, both(1.9046543e-9f), fma2(t, both(-0.69314718246459961f), v));
  return mul2(exp2_approx2(t), fma2(d, both(1.f), both(1.f)));
}

// 1 / (1 + e^-v) for two values, off by 9 u at most: the exponential's 6, one for the sum, 2 for the hardware's
// reciprocal.  Below -87 the reciprocal is 0, at most 2e-38 off.
__device__ __forceinline__ u64 sigmoid2(u64 v) {
  const float2 w = unpack2(v);
  const u64 e = exp2v(pack2(bound_f(w.x, -200.f), bound_f(w.y, -200.f)));
  const float2 q = unpack2(fma2(e, both(1.f), both(1.f)));
  return pack2(rcp_approx(q.x), rcp_approx(q.y));
}
__device__ __forceinline__ u64 swish2(u64 v) { return mul2(v, sigmoid2(v)); }

// One value, for a result of type T.  For 16 bits the exponent is one rounded product, which takes half of the
// instructions: up to 1e-6 off for v in -20 .. 0 and 4e-6 in -87 .. -20, where half a step of the type is 5e-4 and
// more.
template <typename T>
__device__ __forceinline__ float sigmoid_f(float v) {
  if constexpr (std::is_same_v<T, float>) {  // as sigmoid2
    const float w = bound_f(v, -200.f), t = w * 1.4426950408889634f;
    const float d = fmaf(t, 1.9046543e-9f, fmaf(t, -0.69314718246459961f, w));
    return rcp_approx(1.f + exp2_approx(t) * (1.f + d));
  }
  return rcp_approx(1.f + exp2_approx(v * -1.4426950408889634f));
}
template <typename T>
__device__ __forceinline__ float swish_f(float v) { return v * sigmoid_f<T>(v); }

// --- host side -----------------------------------------------------------------

inline gam_status op_fail(gam_status s, const std::string& msg) {
  set_context_free_error(msg);
  return s;
}
constexpr int kMaxDim = 1 << 30;  // of one dimension: sums of two stay in 32 bits
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
// A launch's error as a status.
gam_status launch_status(cudaError_t e);

// A launch with the error of this launch alone: after <<<>>>, cudaGetLastError() also reports, and takes, what an
// earlier call of the caller's has left.
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace ops
}  // namespace gam
