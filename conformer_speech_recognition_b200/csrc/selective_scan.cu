// Selective state-space scan: gam_selective_scan.
//
//   s = softplus(dt + dt_bias); h_i = exp(s a_i) h_i + s x b_i; y = (sum_i c_i h_i + skip x) z sigmoid(z)
//
// First form: L neighbouring lanes share a channel, each holding S of its n
// states (S L >= n; states past n have a = b = c = 0) in registers, and walk the
// time axis frame by frame; the lanes' partial outputs are added by shuffles.
#include "stream_ops.cuh"

namespace gam {
namespace ops {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// log(1 + e^v): v + log1p(e^-v) above 0, so neither form overflows or cancels
__device__ __forceinline__ float softplus_f(float v) {
  return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))) + (v != v ? v : 0.f);
}

template <typename T, int S, int L>
__global__ void __launch_bounds__(128) scan_kernel(const gam_scan_args p) {
  constexpr int kChannels = 128 / L;
  const int cblocks = (p.d + kChannels - 1) / kChannels;
  const int cb = blockIdx.x % cblocks, b = blockIdx.x / cblocks;
  const int part = threadIdx.x % L;
  const int c0 = cb * kChannels + threadIdx.x / L;
  const bool live = c0 < p.d;
  const int c = live ? c0 : p.d - 1;  // lanes past the last channel walk along, for the shuffles
  const int len = p.lengths ? min(max(p.lengths[b], 0), p.t_max) : p.t_max;
  float a[S], h[S];
  bool on[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int k = part * S + i;
    on[i] = k < p.n;
    a[i] = on[i] ? p.a[(int64_t)c * p.n + k] * kLog2e : 0.f;
    h[i] = on[i] && p.state_in ? p.state_in[((int64_t)b * p.d + c) * p.n + k] : 0.f;
  }
  const float skip = p.d_skip ? p.d_skip[c] : 0.f, bias = p.dt_bias ? p.dt_bias[c] : 0.f;
  const T* x = (const T*)p.x + b * p.x_batch_stride + c;
  const T* dt = (const T*)p.dt + b * p.dt_batch_stride + c;
  const T* z = p.z ? (const T*)p.z + b * p.z_batch_stride + c : nullptr;
  const T* bb = (const T*)p.b + b * p.b_batch_stride + part * S;
  const T* cc = (const T*)p.c + b * p.c_batch_stride + part * S;
  T* y = (T*)p.y + b * p.y_batch_stride + c;
  for (int t = 0; t < len; ++t) {
    float s = to_f(dt[t * p.dt_row_stride]) + bias;
    if (p.dt_softplus) s = softplus_f(s);
    const float xv = to_f(x[t * p.x_row_stride]);
    const float sx = s * xv;
    float out = 0.f;
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (on[i]) {
        h[i] = fmaf(exp2_approx(s * a[i]), h[i], sx * to_f(bb[t * p.b_row_stride + i]));
        out = fmaf(to_f(cc[t * p.c_row_stride + i]), h[i], out);
      }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) out += __shfl_xor_sync(0xffffffffu, out, o);
    out = fmaf(skip, xv, out);
    if (z) out *= swish_f(to_f(z[t * p.z_row_stride]));
    if (live && part == 0) y[t * p.y_row_stride] = from_f<T>(out);
  }
  if (live && part == 0)
    for (int t = len; t < p.t_max; ++t) y[t * p.y_row_stride] = from_f<T>(0.f);
  if (live && p.state_out)
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (on[i]) p.state_out[((int64_t)b * p.d + c) * p.n + part * S + i] = h[i];
}

template <typename T, int S, int L>
gam_status launch_sl(const gam_scan_args& p, cudaStream_t s) {
  const int64_t grid = (int64_t)((p.d + 128 / L - 1) / (128 / L)) * p.batch;
  if (grid > INT32_MAX) return op_fail(GAM_ERR_CAPACITY, "batch * d too large for one call");
  scan_kernel<T, S, L><<<(unsigned)grid, 128, 0, s>>>(p);
  return launch_status(cudaGetLastError());
}

template <typename T>
gam_status launch(const gam_scan_args& p, cudaStream_t s) {
  if (p.n <= 8) return launch_sl<T, 8, 1>(p, s);
  if (p.n <= 16) return launch_sl<T, 8, 2>(p, s);
  if (p.n <= 32) return launch_sl<T, 8, 4>(p, s);
  return launch_sl<T, 8, 8>(p, s);
}

}  // namespace
}  // namespace ops
}  // namespace gam

using namespace gam::ops;

extern "C" gam_status gam_selective_scan(const gam_scan_args* args, void* stream) {
  return guarded([&] {
    if (!args) return op_fail(GAM_ERR_INVALID_ARG, "null args");
    const gam_scan_args p = *args;
    if (!is_float_dtype(p.dtype)) return op_fail(GAM_ERR_INVALID_ARG, "dtype must be f32, f16 or bf16");
    if (p.batch < 0 || p.t_max < 0 || p.d < 1) return op_fail(GAM_ERR_INVALID_ARG, "batch >= 0, t_max >= 0 and d >= 1");
    if (p.n < 1 || p.n > 64) return op_fail(GAM_ERR_SHAPE, "n must be 1 .. 64");
    if (p.batch == 0) return GAM_OK;
    if (!p.a || (p.t_max > 0 && (!p.x || !p.dt || !p.b || !p.c || !p.y)))
      return op_fail(GAM_ERR_INVALID_ARG, "null pointer");
    const int es = dtype_size(p.dtype);
    if (!aligned(p.x, es) || !aligned(p.dt, es) || !aligned(p.b, es) || !aligned(p.c, es) || !aligned(p.z, es) ||
        !aligned(p.y, es) || !aligned(p.a, 4) || !aligned(p.d_skip, 4) || !aligned(p.dt_bias, 4) ||
        !aligned(p.lengths, 4) || !aligned(p.state_in, 4) || !aligned(p.state_out, 4))
      return op_fail(GAM_ERR_INVALID_ARG, "a buffer is not aligned to its element type");
    if (p.t_max > 0 && (p.y == p.x || p.y == p.dt || p.y == p.b || p.y == p.c || p.y == p.z))
      return op_fail(GAM_ERR_INVALID_ARG, "y must not be an input");
    if (!rows_apart(p.batch, p.t_max, p.d, p.y_batch_stride, p.y_row_stride))
      return op_fail(GAM_ERR_SHAPE, "rows of y overlap");
    int sms = 0;
    if (gam_status st = check_device(&sms)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.dtype == GAM_DTYPE_F32) return launch<float>(p, s);
    if (p.dtype == GAM_DTYPE_F16) return launch<__half>(p, s);
    return launch<bf16>(p, s);
  });
}
