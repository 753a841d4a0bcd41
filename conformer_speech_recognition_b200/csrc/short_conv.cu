// Short causal depthwise convolution with a state: gam_short_conv.
//
//   y[b, t, c] = act(bias[c] + sum_j w[c, j] v[b, t + j, c]),  v = [state ; x]
//
// A thread owns V channels (one 16-byte access; one channel when the rows are
// not 16-byte aligned) and a segment of the time axis.  It keeps the last
// taps - 1 rows in registers, so inside a segment every input is read once.
#include "stream_ops.cuh"

namespace gam {
namespace ops {
namespace {

struct ConvArgs {
  const void* x;
  const float* w;
  const float* bias;
  const int32_t* lengths;
  const void* state_in;
  void* state_out;
  void* y;
  int64_t xb, xr, yb, yr;
  int act, t_max, d, seg, segs, cblocks;
};

constexpr int kThreads = 128;

template <typename T, int V, int TAPS>
__global__ void __launch_bounds__(kThreads) short_conv_kernel(const ConvArgs p) {
  using Vt = Vec<T, V>;
  constexpr int H = TAPS - 1;                  // rows of history
  constexpr int R = TAPS <= 5 ? 8 : 4;         // rows loaded ahead of their use
  const int cb = blockIdx.x % p.cblocks;
  const int rest = blockIdx.x / p.cblocks;
  const int seg = rest % p.segs, b = rest / p.segs;
  const int c = (cb * kThreads + threadIdx.x) * V;
  if (c >= p.d) return;
  const int len = p.lengths ? min(max(p.lengths[b], 0), p.t_max) : p.t_max;
  const T* x = (const T*)p.x + b * p.xb + c;
  T* y = (T*)p.y + b * p.yb + c;
  const T* sin = p.state_in ? (const T*)p.state_in + (int64_t)b * H * p.d + c : nullptr;
  // row r of the input, r >= -H: the state's before 0
  auto row = [&](int r) -> Vt {
    if (r >= 0) return *reinterpret_cast<const Vt*>(x + r * p.xr);
    if (sin) return *reinterpret_cast<const Vt*>(sin + (int64_t)(r + H) * p.d);
    Vt z;
#pragma unroll
    for (int i = 0; i < V; ++i) z.v[i] = from_f<T>(0.f);
    return z;
  };
  const int t0 = seg * p.seg, t1 = min(t0 + p.seg, p.t_max);
  float h[H][V];
#pragma unroll
  for (int j = 0; j < H; ++j) {
    Vt r;
    if (t0 < len) r = row(t0 - H + j);  // a segment behind the length reads nothing
#pragma unroll
    for (int i = 0; i < V; ++i) h[j][i] = t0 < len ? to_f(r.v[i]) : 0.f;
  }
  if (seg == 0 && p.state_out) {
    // this thread alone touches its channels' state: all of it is read first, so
    // state_out may be state_in
    Vt keep[H];
#pragma unroll
    for (int j = 0; j < H; ++j) keep[j] = row(len - H + j);
    T* so = (T*)p.state_out + (int64_t)b * H * p.d + c;
#pragma unroll
    for (int j = 0; j < H; ++j) *reinterpret_cast<Vt*>(so + (int64_t)j * p.d) = keep[j];
  }
  float w[TAPS][V], bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bias[i] = p.bias ? __ldg(p.bias + c + i) : 0.f;
#pragma unroll
    for (int j = 0; j < TAPS; ++j) w[j][i] = __ldg(p.w + (int64_t)(c + i) * TAPS + j);
  }
  for (int t = t0; t < t1; t += R) {
    Vt in[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (t + r < min(t1, len)) in[r] = row(t + r);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (t + r >= t1) break;
      Vt out;
      if (t + r < len) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float cur = to_f(in[r].v[i]);
          float acc = bias[i];
#pragma unroll
          for (int j = 0; j < H; ++j) acc = fmaf(w[j][i], h[j][i], acc);
          acc = fmaf(w[H][i], cur, acc);
#pragma unroll
          for (int j = 0; j + 1 < H; ++j) h[j][i] = h[j + 1][i];
          h[H - 1][i] = cur;
          out.v[i] = from_f<T>(p.act == GAM_ACT_SWISH ? swish_f(acc) : acc);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out.v[i] = from_f<T>(0.f);
      }
      *reinterpret_cast<Vt*>(y + (t + r) * p.yr) = out;
    }
  }
}

template <typename T, int V>
cudaError_t launch_taps(int taps, dim3 grid, const ConvArgs& p, cudaStream_t s) {
  switch (taps) {
    case 2: short_conv_kernel<T, V, 2><<<grid, kThreads, 0, s>>>(p); break;
    case 3: short_conv_kernel<T, V, 3><<<grid, kThreads, 0, s>>>(p); break;
    case 4: short_conv_kernel<T, V, 4><<<grid, kThreads, 0, s>>>(p); break;
    case 5: short_conv_kernel<T, V, 5><<<grid, kThreads, 0, s>>>(p); break;
    case 6: short_conv_kernel<T, V, 6><<<grid, kThreads, 0, s>>>(p); break;
    case 7: short_conv_kernel<T, V, 7><<<grid, kThreads, 0, s>>>(p); break;
    default: short_conv_kernel<T, V, 8><<<grid, kThreads, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

template <typename T>
gam_status launch(int taps, int batch, ConvArgs p, int sms, cudaStream_t s) {
  constexpr int VW = 16 / sizeof(T);
  const bool wide = p.d % VW == 0 && aligned(p.x, 16) && aligned(p.y, 16) && aligned(p.state_in, 16) &&
                    aligned(p.state_out, 16) && p.xb % VW == 0 && p.xr % VW == 0 && p.yb % VW == 0 && p.yr % VW == 0;
  const int V = wide ? VW : 1;
  p.cblocks = (p.d / V + kThreads - 1) / kThreads;
  // segments: enough CTAs for 8 to an SM, none shorter than 16 rows
  const int64_t base = (int64_t)p.cblocks * batch, want = (int64_t)sms * 8;
  int64_t segs = (want + base - 1) / base;
  const int64_t most = p.t_max / 16 > 1 ? p.t_max / 16 : 1;
  if (segs > most) segs = most;
  p.seg = p.t_max ? (int)((p.t_max + segs - 1) / segs) : 1;
  p.seg = (p.seg + 7) / 8 * 8;
  p.segs = p.t_max ? (p.t_max + p.seg - 1) / p.seg : 1;
  const int64_t grid = base * p.segs;
  if (grid > INT32_MAX) return op_fail(GAM_ERR_CAPACITY, "batch * t_max * d too large for one call");
  return launch_status(wide ? launch_taps<T, VW>(taps, dim3((unsigned)grid), p, s)
                            : launch_taps<T, 1>(taps, dim3((unsigned)grid), p, s));
}

}  // namespace
}  // namespace ops
}  // namespace gam

using namespace gam::ops;

extern "C" gam_status gam_short_conv(const void* x, int dtype, int64_t x_batch_stride, int64_t x_row_stride,
                                     const float* w, const float* bias, int taps, int act, int batch, int t_max, int d,
                                     const int32_t* lengths, const void* state_in, void* state_out, void* y,
                                     int64_t y_batch_stride, int64_t y_row_stride, void* stream) {
  return guarded([&] {
    if (!is_float_dtype(dtype)) return op_fail(GAM_ERR_INVALID_ARG, "dtype must be f32, f16 or bf16");
    if (act != GAM_ACT_NONE && act != GAM_ACT_SWISH) return op_fail(GAM_ERR_INVALID_ARG, "act must be none or swish");
    if (batch < 0 || t_max < 0 || d < 1) return op_fail(GAM_ERR_INVALID_ARG, "batch >= 0, t_max >= 0 and d >= 1");
    if (taps < 2 || taps > 8) return op_fail(GAM_ERR_SHAPE, "taps must be 2 .. 8");
    if (batch == 0) return GAM_OK;
    if (!w || (t_max > 0 && (!x || !y))) return op_fail(GAM_ERR_INVALID_ARG, "null pointer");
    const int es = dtype_size(dtype);
    if (!aligned(x, es) || !aligned(y, es) || !aligned(state_in, es) || !aligned(state_out, es) || !aligned(w, 4) ||
        !aligned(bias, 4) || !aligned(lengths, 4))
      return op_fail(GAM_ERR_INVALID_ARG, "a buffer is not aligned to its element type");
    if (t_max > 0 && x == y) return op_fail(GAM_ERR_INVALID_ARG, "y must not be x");
    if (!rows_apart(batch, t_max, d, y_batch_stride, y_row_stride))
      return op_fail(GAM_ERR_SHAPE, "rows of y overlap");
    int sms = 0;
    if (gam_status st = check_device(&sms)) return st;
    ConvArgs p{x,  w, bias, lengths, state_in, state_out, y, x_batch_stride, x_row_stride, y_batch_stride, y_row_stride,
               act, t_max, d, 0, 0, 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == GAM_DTYPE_F32) return launch<float>(taps, batch, p, sms, s);
    if (dtype == GAM_DTYPE_F16) return launch<__half>(taps, batch, p, sms, s);
    return launch<bf16>(taps, batch, p, sms, s);
  });
}
