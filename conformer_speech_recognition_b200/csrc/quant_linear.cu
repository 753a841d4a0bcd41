// Few-row linear layer on INT4-g64 weights: gam_quant_linear.
//
//   y[m, o] = act(bias[o] + sum_g scale[o, g] sum_{j in g} q[o, j] x[m, j])
//
// First form: one warp per output o.  A lane takes every 32nd word of 8 weights,
// so a group of 64 is 8 neighbouring lanes; scale times integer is exact in fp32,
// and the warp's partial sums are added by shuffles.  Rows go by eight, re-reading the weights from L1 / L2.
#include "stream_ops.cuh"

namespace gam {
namespace ops {
namespace {

constexpr int kRows = 8;

template <typename T>
__global__ void __launch_bounds__(256)
quant_linear_kernel(const T* __restrict__ x, int64_t ldx, const uint32_t* __restrict__ packed,
                    const __half* __restrict__ scale, const float* __restrict__ bias, int act, int rows, int n, int k,
                    T* __restrict__ y, int64_t ldy) {
  const int o = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (o >= n) return;
  const int words = k / 8;
  const uint32_t* w = packed + (size_t)o * words;
  const __half* sc = scale + (size_t)o * (k / 64);
  for (int m0 = 0; m0 < rows; m0 += kRows) {
    float acc[kRows] = {};
    for (int i = lane; i < words; i += 32) {
      const uint32_t u = __ldg(w + i);
      const float s = __half2float(sc[i >> 3]);
      float q[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q[2 * j] = s * (float)((int)((u >> (4 * j)) & 15u) - 8);  // 4 + 11 bits: exact
        q[2 * j + 1] = s * (float)((int)((u >> (16 + 4 * j)) & 15u) - 8);
      }
#pragma unroll
      for (int m = 0; m < kRows; ++m)
        if (m0 + m < rows) {
          const T* xr = x + (m0 + m) * ldx + (int64_t)i * 8;
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[m] = fmaf(q[j], to_f(xr[j]), acc[m]);
        }
    }
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
      for (int s = 16; s > 0; s >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], s);
      if (lane == 0 && m0 + m < rows) {
        const float v = acc[m] + (bias ? bias[o] : 0.f);
        y[(m0 + m) * ldy + o] = from_f<T>(act == GAM_ACT_SWISH ? swish_f(v) : v);
      }
    }
  }
}

template <typename T>
cudaError_t launch(const void* x, int64_t ldx, const uint8_t* packed, const void* scale, const float* bias, int act,
                   int rows, int n, int k, void* y, int64_t ldy, cudaStream_t s) {
  quant_linear_kernel<T><<<(n + 7) / 8, 256, 0, s>>>((const T*)x, ldx, (const uint32_t*)packed, (const __half*)scale,
                                                     bias, act, rows, n, k, (T*)y, ldy);
  return cudaGetLastError();
}

}  // namespace
}  // namespace ops
}  // namespace gam

using namespace gam::ops;

extern "C" gam_status gam_quant_linear_pack(const int8_t* q, int64_t n, int64_t k, uint8_t* packed) {
  return guarded([&] {
    if (!q || !packed) return op_fail(GAM_ERR_INVALID_ARG, "null pointer");
    if (n < 1 || k < 1) return op_fail(GAM_ERR_INVALID_ARG, "n and k must be >= 1");
    if (k % 64) return op_fail(GAM_ERR_SHAPE, "k must be a multiple of 64");
    for (int64_t i = 0; i < n * k; ++i)
      if (q[i] < -7 || q[i] > 7)
        return op_fail(GAM_ERR_WEIGHTS, "weight_q holds " + std::to_string((int)q[i]) + ", outside +-7");
    for (int64_t i = 0; i < n * k / 8; ++i) {
      uint32_t w = 0;
      for (int j = 0; j < 8; ++j) w |= (uint32_t)(q[8 * i + j] + 8) << ((j & 1) * 16 + (j >> 1) * 4);
      for (int j = 0; j < 4; ++j) packed[4 * i + j] = (uint8_t)(w >> (8 * j));
    }
    return GAM_OK;
  });
}

extern "C" gam_status gam_quant_linear(const void* x, int dtype, int64_t ldx, const uint8_t* packed, const void* scale,
                                       const float* bias, int act, int rows, int n, int k, void* y, int64_t ldy,
                                       void* stream) {
  return guarded([&] {
    if (!is_float_dtype(dtype)) return op_fail(GAM_ERR_INVALID_ARG, "dtype must be f32, f16 or bf16");
    if (act != GAM_ACT_NONE && act != GAM_ACT_SWISH) return op_fail(GAM_ERR_INVALID_ARG, "act must be none or swish");
    if (rows < 0 || n < 1 || k < 1) return op_fail(GAM_ERR_INVALID_ARG, "rows >= 0, n >= 1 and k >= 1");
    if (rows > GAM_QUANT_LINEAR_MAX_ROWS)
      return op_fail(GAM_ERR_CAPACITY, "rows above " + std::to_string(GAM_QUANT_LINEAR_MAX_ROWS));
    if (k % 64) return op_fail(GAM_ERR_SHAPE, "k must be a multiple of 64");
    if (rows == 0) return GAM_OK;
    if (!x || !packed || !scale || !y) return op_fail(GAM_ERR_INVALID_ARG, "null pointer");
    if (!aligned(packed, 16)) return op_fail(GAM_ERR_INVALID_ARG, "packed weights must be 16-byte aligned");
    const int es = dtype_size(dtype);
    if (!aligned(x, es) || !aligned(y, es) || !aligned(scale, 2) || !aligned(bias, 4))
      return op_fail(GAM_ERR_INVALID_ARG, "a buffer is not aligned to its element type");
    if (rows > 1 && (ldx < k || ldy < n)) return op_fail(GAM_ERR_SHAPE, "ldx >= k and ldy >= n");
    if (x == y) return op_fail(GAM_ERR_INVALID_ARG, "y must not be x");
    int sms = 0;
    if (gam_status st = check_device(&sms)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == GAM_DTYPE_F32   ? launch<float>(x, ldx, packed, scale, bias, act, rows, n, k, y, ldy, s)
                    : dtype == GAM_DTYPE_F16 ? launch<__half>(x, ldx, packed, scale, bias, act, rows, n, k, y, ldy, s)
                                             : launch<bf16>(x, ldx, packed, scale, bias, act, rows, n, k, y, ldy, s);
    return launch_status(e);
  });
}
