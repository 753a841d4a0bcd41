// Short causal depthwise convolution with a state: gam_short_conv.
//
//   y[b, t, c] = act(bias[c] + sum_j w[c, j] v[b, t + j, c]),  v = [state ; x]
//
// A thread owns V channels (one 16-byte access; one channel when the rows are
// not 16-byte aligned) and a segment of the time axis.  It keeps the last
// taps - 1 rows in registers, so inside a segment every input is read once, and
// has R rows on their way while it works on R others.  The multiply-adds go two
// channels at a time in packed fp32.  32 clips of up to 749 frames of 2048 channels:
// fp32 56 us (298 MB, 5.3 TB/s); fp16 34.5 us (150 MB, 4.3 TB/s), where the latency
// bounds it: the rows in flight take 168 registers, which leaves 10 warps to an SM.
// With 128 registers it spills (64 us).
#include <algorithm>

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
  int act, batch, t_max, d, seg, segs, vecs;
};

constexpr int kThreads = 128;

template <typename T, int V, int TAPS, int R>
__global__ void __launch_bounds__(kThreads) short_conv_kernel(const ConvArgs p) {
  using Row = Raw<T, V>;
  constexpr int H = TAPS - 1;                  // rows of history
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t item = id / p.vecs;
  if (item >= (int64_t)p.batch * p.segs) return;
  const int c = (int)(id - item * p.vecs) * V;
  const int seg = (int)(item % p.segs), b = (int)(item / p.segs);
  const int len = p.lengths ? min(max(p.lengths[b], 0), p.t_max) : p.t_max;
  const T* x = (const T*)p.x + b * p.xb + c;
  T* y = (T*)p.y + b * p.yb + c;
  const T* past = p.state_in ? (const T*)p.state_in + (int64_t)b * H * p.d + c : nullptr;
  // row r >= -H of the input: the state's before 0
  auto row = [&](int r) {
    Row v;
    v.zero();
    if (r >= 0) v.load(x + r * p.xr);
    else if (past) v.load(past + (int64_t)(r + H) * p.d);
    return v;
  };
  const int t0 = seg * p.seg, t1 = min(t0 + p.seg, p.t_max), tv = min(t1, len);
  Row in[R], h[H];
  const bool work = t0 < tv;
  if (work) {
#pragma unroll
    for (int r = 0; r < R; ++r) in[r].load(x + min(t0 + r, tv - 1) * p.xr);  // repeats beyond the end are not used
#pragma unroll
    for (int j = 0; j < H; ++j) h[j] = row(t0 - H + j);
  }
  if (seg == 0 && p.state_out) {
    // this thread alone touches its channels' state, and has read all of it: state_out may be state_in
    Row keep[H];
#pragma unroll
    for (int j = 0; j < H; ++j) keep[j] = row(len - H + j);
    T* so = (T*)p.state_out + (int64_t)b * H * p.d + c;
#pragma unroll
    for (int j = 0; j < H; ++j) keep[j].store(so + (int64_t)j * p.d);
  }
  if (work) {
    constexpr int P = V > 1 ? V / 2 : 1;       // pairs of channels (a single one in both halves)
    constexpr int B = V > 1 ? 1 : 0;
    float wf[V * TAPS];                        // channel i, tap j at i TAPS + j
    const float* pw = p.w + (int64_t)c * TAPS;
    if constexpr (V > 1) {                     // 16-byte aligned with the rows
#pragma unroll
      for (int i = 0; i < V * TAPS / 4; ++i) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(pw) + i);
        wf[4 * i] = q.x, wf[4 * i + 1] = q.y, wf[4 * i + 2] = q.z, wf[4 * i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < TAPS; ++j) wf[j] = __ldg(pw + j);
    }
    u64 w[TAPS][P], bias[P], v[H][P];          // v: the last H rows, oldest first
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
      for (int j = 0; j < TAPS; ++j) w[j][i] = pack2(wf[2 * i * TAPS + j], wf[(2 * i + B) * TAPS + j]);
      bias[i] = p.bias ? pack2(__ldg(p.bias + c + 2 * i), __ldg(p.bias + c + 2 * i + B)) : 0ull;
#pragma unroll
      for (int j = 0; j < H; ++j) v[j][i] = pack2(h[j].get(2 * i), h[j].get(2 * i + B));
    }
    for (int t = t0; t < tv; t += R) {
      Row next[R];
      if (t + R < tv) {
#pragma unroll
        for (int r = 0; r < R; ++r) next[r].load(x + min(t + R + r, tv - 1) * p.xr);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float out[V];
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const u64 cur = pack2(in[r].get(2 * i), in[r].get(2 * i + B));
          u64 acc = bias[i];
#pragma unroll
          for (int j = 0; j < H; ++j) acc = fma2(w[j][i], v[j][i], acc);
          acc = fma2(w[H][i], cur, acc);
#pragma unroll
          for (int j = 0; j + 1 < H; ++j) v[j][i] = v[j + 1][i];
          v[H - 1][i] = cur;
          const bool swish = p.act == GAM_ACT_SWISH;
          if constexpr (sizeof(T) == 4) {
            if (swish) acc = swish2(acc);
          }
          const float2 q = unpack2(acc);
          out[2 * i] = sizeof(T) == 2 && swish ? swish_f<T>(q.x) : q.x;
          if constexpr (V > 1) out[2 * i + 1] = sizeof(T) == 2 && swish ? swish_f<T>(q.y) : q.y;
        }
        if (t + r < tv) {
          Row o;
          o.set(out);
          o.store(y + (t + r) * p.yr);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) in[r] = next[r];
    }
  }
  Row zero;
  zero.zero();
  for (int t = max(t0, len); t < t1; ++t) zero.store(y + t * p.yr);
}

template <typename T, int V, int R>
cudaError_t launch_taps(int taps, unsigned grid, const ConvArgs& p, cudaStream_t s) {
  auto go = [&](auto kernel) { return launch_kernel(kernel, grid, kThreads, 0, s, p); };
  switch (taps) {
    case 2: return go(short_conv_kernel<T, V, 2, R>);
    case 3: return go(short_conv_kernel<T, V, 3, R>);
    case 4: return go(short_conv_kernel<T, V, 4, R>);
    case 5: return go(short_conv_kernel<T, V, 5, R>);
    case 6: return go(short_conv_kernel<T, V, 6, R>);
    case 7: return go(short_conv_kernel<T, V, 7, R>);
    default: return go(short_conv_kernel<T, V, 8, R>);
  }
}

template <typename T>
gam_status launch(int taps, ConvArgs p, int sms, cudaStream_t s) {
  constexpr int VW = 16 / sizeof(T);
  const bool wide = p.d % VW == 0 && aligned(p.x, 16) && aligned(p.y, 16) && aligned(p.state_in, 16) &&
                    aligned(p.state_out, 16) && aligned(p.w, 16) && p.xb % VW == 0 && p.xr % VW == 0 &&
                    p.yb % VW == 0 && p.yr % VW == 0;
  p.vecs = wide ? p.d / VW : p.d;
  // Segments short enough for 512 threads to an SM, of 8 rows on their way at a time; a call too small for
  // that takes 2 rows to a thread, since one warp's instructions then are its time.
  const int64_t columns = (int64_t)p.vecs * p.batch, want = (int64_t)sms * 512;
  const int64_t segs = std::max<int64_t>(1, (want + columns - 1) / columns);
  const int R = p.t_max == 1 ? 1 : p.t_max / segs >= 8 ? 8 : 2;
  // A segment is no shorter than the history, so that only segment 0 reads the state that it may replace.
  p.seg = (int)((std::max<int64_t>((p.t_max + segs - 1) / segs, taps - 1) + R - 1) / R * R);
  p.segs = p.t_max ? (p.t_max + p.seg - 1) / p.seg : 1;
  const int64_t grid = (columns * p.segs + kThreads - 1) / kThreads;
  if (grid > INT32_MAX) return op_fail(GAM_ERR_CAPACITY, "batch * t_max * d too large for one call");
  const unsigned g = (unsigned)grid;
  if (R == 1) return launch_status(wide ? launch_taps<T, VW, 1>(taps, g, p, s) : launch_taps<T, 1, 1>(taps, g, p, s));
  if (R == 2) return launch_status(wide ? launch_taps<T, VW, 2>(taps, g, p, s) : launch_taps<T, 1, 2>(taps, g, p, s));
  return launch_status(wide ? launch_taps<T, VW, 8>(taps, g, p, s) : launch_taps<T, 1, 8>(taps, g, p, s));
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
    if (t_max > kMaxDim || d > kMaxDim) return op_fail(GAM_ERR_CAPACITY, "t_max and d up to 2^30");
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
               act, batch, t_max, d, 0, 0, 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == GAM_DTYPE_F32) return launch<float>(taps, p, sms, s);
    if (dtype == GAM_DTYPE_F16) return launch<__half>(taps, p, sms, s);
    return launch<bf16>(taps, p, sms, s);
  });
}
