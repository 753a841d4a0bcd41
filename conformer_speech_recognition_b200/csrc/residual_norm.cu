// Residual update with the norms around it: gam_residual_norm.
//
//   x' = x + alpha * layer_scale * gate_act(gate) * post_norm(y),  u = pre_norm(x')
//
// One pass: a group of G threads (a warp, or a CTA for wide or few rows) holds a
// row of y and x in registers, so each is read once; all loads of a row are on
// their way before the first is used, and a warp's next row while it works on
// this one.  Statistics are two-pass in fp32 (mean, then the centred squares)
// over those registers.  The bound is memory.
//
// Accesses are 16 bytes where rows are 16-byte aligned.  Else they are pairs of
// values: a row of odd offset starts with the second half of a pair, so pair i
// holds columns 2 i - phase and the next, phase being the offset's last bit, and
// every whole pair is aligned whatever the row.  Without that (arrays whose rows
// differ in that bit) they are single values.
#include <algorithm>

#include "stream_ops.cuh"

namespace gam {
namespace ops {
namespace {

// Sum over the G threads of a row: a warp by shuffles, a CTA through shared
// memory (red holds two alternating sets of 32 partial sums, so one barrier per
// sum is enough).
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (WARP) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float* r = red[turn];
  turn ^= 1;
  if (lane == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? r[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Row position of a thread: it holds accesses j G + tid of V columns, j < NV, the first
// column of an access being `phase` (pairs only) before its multiple of V.
template <int V>
struct Place {
  int tid, G, d, phase;
  __device__ __forceinline__ int col(int j) const { return (j * G + tid) * V - (V == 2 ? phase : 0); }
  __device__ __forceinline__ bool on(int j, int i) const {  // value i of access j is a column of the row
    const int c = col(j) + i;
    return V == 2 ? (unsigned)c < (unsigned)d : c < d;
  }
  __device__ __forceinline__ bool whole(int j) const { return V == 2 ? on(j, 0) && on(j, 1) : on(j, 0); }
};

// Access j of a row; what lies beside the row is 0 and not read.
template <typename T, int V>
__device__ __forceinline__ void load_at(Raw<T, V>& r, const T* row, const Place<V>& at, int j) {
  r.zero();
  if (at.whole(j)) r.load(row + at.col(j));
}
// ... the halves of a pair at the row's ends (after all whole accesses are on their way)
template <typename T, int V>
__device__ __forceinline__ void load_ends(Raw<T, V>& r, const T* row, const Place<V>& at, int j) {
  if constexpr (V == 2) {
    if (!at.whole(j) && (at.on(j, 0) || at.on(j, 1))) {
      const int i = at.on(j, 1);
      Raw<T, 1> one;
      one.load(row + at.col(j) + i);
      if constexpr (sizeof(T) == 4) r.w[i] = one.w[0];
      else r.w[0] = one.w[0] << (16 * i);
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_at(T* row, const Place<V>& at, int j, const float (&v)[V]) {
  if (at.whole(j)) {
    Raw<T, V> o;
    o.set(v);
    o.store(row + at.col(j));
  } else if constexpr (V == 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (at.on(j, i)) row[at.col(j) + i] = from_f<T>(v[i]);
  }
}

template <int V>
__device__ __forceinline__ void load_param(const float* p, const Place<V>& at, int j, float fill, float (&out)[V]) {
  const int c = at.col(j);
  if constexpr (V <= 2) {
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = p ? __ldg(p + min(max(c + i, 0), at.d - 1)) : fill;
  } else {  // 16-byte aligned with the rows
    const float* q = p + min(c, at.d - V);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 f = p ? __ldg(reinterpret_cast<const float4*>(q) + i) : make_float4(fill, fill, fill, fill);
      out[4 * i] = f.x, out[4 * i + 1] = f.y, out[4 * i + 2] = f.z, out[4 * i + 3] = f.w;
    }
  }
}

// v <- norm(v) over the row
template <bool WARP, int V, int NV>
__device__ __forceinline__ void norm_row(float (&v)[NV][V], int kind, const float* w, const float* b, float eps,
                                         const Place<V>& at, float (*red)[32], int& turn) {
  // one access a thread: its weights come while the row is summed
  float w0[V], b0[V];
  if constexpr (NV == 1) {
    load_param<V>(w, at, 0, 1.f, w0);
    load_param<V>(kind == GAM_NORM_LAYER ? b : nullptr, at, 0, 0.f, b0);
  }
  const float inv = 1.f / at.d;
  if (kind == GAM_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) s += v[j][i];
    const float mean = row_sum<WARP>(s, red, turn) * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] = at.on(j, i) ? v[j][i] - mean : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) q = fmaf(v[j][i], v[j][i], q);
  const float r = rsqrtf(fmaf(row_sum<WARP>(q, red, turn), inv, eps));
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if constexpr (NV > 1) {
      load_param<V>(w, at, j, 1.f, w0);
      load_param<V>(kind == GAM_NORM_LAYER ? b : nullptr, at, j, 0.f, b0);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[j][i] = at.on(j, i) ? fmaf(v[j][i] * r, w0[i], b0[i]) : 0.f;
  }
}

constexpr int kWarps = 4;  // rows of a CTA at a time in the warp form

template <typename TX, typename TY, bool WARP, int V, int NV, bool GATE>
__global__ void __launch_bounds__(WARP ? 32 * kWarps : V == 8 ? 512 : 1024, WARP && NV == 4 ? 3 : 1)
residual_norm_kernel(const gam_residual_norm_args p, const int64_t per_gate) {
  __shared__ float red[2][32];
  const int64_t step = WARP ? (int64_t)gridDim.x * kWarps : (int64_t)gridDim.x;
  int64_t row = WARP ? (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  Place<V> at{(int)(WARP ? threadIdx.x & 31 : threadIdx.x), (int)(WARP ? 32 : blockDim.x), p.d, 0};
  Raw<TX, V> rx[NV];
  Raw<TY, V> ry[NV], rg[GATE ? NV : 1];
  auto fetch = [&](int64_t r) {
    const TX* xr = (const TX*)p.x + r * p.x_stride;
    const TY* yr = (const TY*)p.y + r * p.y_stride;
    const TY* gr = GATE ? (const TY*)p.gate + r / per_gate * p.gate_stride : nullptr;
    at.phase = (int)(r * p.y_stride) & 1;
#pragma unroll
    for (int j = 0; j < NV; ++j) load_at<TY, V>(ry[j], yr, at, j);
#pragma unroll
    for (int j = 0; j < NV; ++j) load_at<TX, V>(rx[j], xr, at, j);
    if constexpr (GATE)
#pragma unroll
      for (int j = 0; j < NV; ++j) load_at<TY, V>(rg[j], gr, at, j);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_ends<TY, V>(ry[j], yr, at, j);
      load_ends<TX, V>(rx[j], xr, at, j);
      if constexpr (GATE) load_ends<TY, V>(rg[j], gr, at, j);
    }
  };
  if (row >= p.rows) return;
  fetch(row);
  int turn = 0;
  while (true) {
    float y[NV][V], x[NV][V], g[GATE ? NV : 1][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        y[j][i] = ry[j].get(i);
        x[j][i] = rx[j].get(i);
        if constexpr (GATE) g[j][i] = rg[j].get(i);
      }
    const Place<V> here = at;
    if (WARP && row + step < p.rows) fetch(row + step);
    if (p.post_norm) norm_row<WARP, V, NV>(y, p.post_norm, p.post_weight, p.post_bias, p.eps, here, red, turn);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float ls[V];
      load_param<V>(p.layer_scale, here, j, 1.f, ls);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (GATE) y[j][i] *= activate(g[j][i], p.gate_act);
        x[j][i] = here.on(j, i) ? fmaf(p.alpha * ls[i], y[j][i], x[j][i]) : 0.f;
      }
      if (p.x_out) store_at<TX, V>((TX*)p.x_out + row * p.x_out_stride, here, j, x[j]);
    }
    if (p.u) {
      if (p.pre_norm) norm_row<WARP, V, NV>(x, p.pre_norm, p.pre_weight, p.pre_bias, p.eps, here, red, turn);
#pragma unroll
      for (int j = 0; j < NV; ++j) store_at<TY, V>((TY*)p.u + row * p.u_stride, here, j, x[j]);
    }
    row += step;
    if (!WARP || row >= p.rows) return;
  }
}

template <typename TX, typename TY, int V, bool GATE>
gam_status launch_v(const gam_residual_norm_args& p, int64_t per_gate, int sms, cudaStream_t s) {
  const int vecs = (p.d + V - 1) / V + (V == 2);  // a phase can cut one pair in two
  // rows enough for 8 warps to an SM: a warp holds a row, up to 4 accesses to a lane, and walks over the rows
  if (vecs <= 128 && (p.rows >= 8 * sms || vecs <= 32)) {
    auto grid = [&](int per_sm) { return (unsigned)std::min<int64_t>((p.rows + kWarps - 1) / kWarps, (int64_t)sms * per_sm); };
    if (vecs <= 32) residual_norm_kernel<TX, TY, true, V, 1, GATE><<<grid(8), 32 * kWarps, 0, s>>>(p, per_gate);
    else if (vecs <= 64) residual_norm_kernel<TX, TY, true, V, 2, GATE><<<grid(5), 32 * kWarps, 0, s>>>(p, per_gate);
    else residual_norm_kernel<TX, TY, true, V, 4, GATE><<<grid(3), 32 * kWarps, 0, s>>>(p, per_gate);
    return launch_status(cudaGetLastError());
  }
  if (p.rows > INT32_MAX) return op_fail(GAM_ERR_CAPACITY, "too many rows for one call");
  const unsigned grid = (unsigned)p.rows;
  auto threads = [&](int nv) { return ((vecs + nv - 1) / nv + 31) / 32 * 32; };
  // as few accesses to a thread as the CTA's size allows
  if (vecs <= 512) residual_norm_kernel<TX, TY, false, V, 1, GATE><<<grid, threads(1), 0, s>>>(p, per_gate);
  else if (vecs <= 1024) residual_norm_kernel<TX, TY, false, V, 2, GATE><<<grid, threads(2), 0, s>>>(p, per_gate);
  else if (vecs <= 2048) residual_norm_kernel<TX, TY, false, V, 4, GATE><<<grid, threads(4), 0, s>>>(p, per_gate);
  else if constexpr (V < 8) {
    if (vecs <= 4096) residual_norm_kernel<TX, TY, false, V, 4, GATE><<<grid, threads(4), 0, s>>>(p, per_gate);
    else if constexpr (V <= 2) {
      if (vecs <= 8192) residual_norm_kernel<TX, TY, false, V, 8, GATE><<<grid, threads(8), 0, s>>>(p, per_gate);
      else residual_norm_kernel<TX, TY, false, V, 16, GATE><<<grid, threads(16), 0, s>>>(p, per_gate);
    }
  }
  return launch_status(cudaGetLastError());
}

template <typename TX, typename TY, int V>
gam_status launch_g(const gam_residual_norm_args& p, int64_t per_gate, int sms, cudaStream_t s) {
  return p.gate ? launch_v<TX, TY, V, true>(p, per_gate, sms, s) : launch_v<TX, TY, V, false>(p, per_gate, sms, s);
}

template <typename TX, typename TY>
gam_status launch(const gam_residual_norm_args& p, int64_t per_gate, int sms, cudaStream_t s) {
  constexpr int V = 16 / sizeof(TY);
  auto rows_at = [&](size_t align_x, size_t align_y) {
    return aligned(p.x, align_x) && aligned(p.x_out, align_x) && aligned(p.y, align_y) && aligned(p.u, align_y) &&
           aligned(p.gate, align_y);
  };
  const int64_t strides[5] = {p.x_stride, p.y_stride, p.x_out_stride, p.u_stride, p.gate_stride};
  bool wide = p.d % V == 0 && rows_at(16, 16) && aligned(p.layer_scale, 16) && aligned(p.post_weight, 16) &&
              aligned(p.post_bias, 16) && aligned(p.pre_weight, 16) && aligned(p.pre_bias, 16);
  bool pairs = rows_at(2 * sizeof(TX), 2 * sizeof(TY));
  for (int i = 0; i < (p.gate ? 5 : 4); ++i) {
    wide = wide && strides[i] % V == 0;
    pairs = pairs && (strides[i] - p.y_stride) % 2 == 0;
  }
  // a gate row that serves several rows has the rows' phase only if that is always 0
  if (p.gate && per_gate > 1 && p.y_stride % 2) pairs = false;
  if (wide) return launch_g<TX, TY, V>(p, per_gate, sms, s);
  return pairs ? launch_g<TX, TY, 2>(p, per_gate, sms, s) : launch_g<TX, TY, 1>(p, per_gate, sms, s);
}

bool norm_kind(int k) { return k == GAM_NORM_NONE || k == GAM_NORM_LAYER || k == GAM_NORM_RMS; }

}  // namespace
}  // namespace ops
}  // namespace gam

using namespace gam::ops;

extern "C" gam_status gam_residual_norm(const gam_residual_norm_args* args, void* stream) {
  return guarded([&] {
    if (!args) return op_fail(GAM_ERR_INVALID_ARG, "null args");
    gam_residual_norm_args p = *args;
    if (!is_float_dtype(p.dtype)) return op_fail(GAM_ERR_INVALID_ARG, "dtype must be f32, f16 or bf16");
    if (p.x_dtype != p.dtype && p.x_dtype != GAM_DTYPE_F32)
      return op_fail(GAM_ERR_INVALID_ARG, "x_dtype must be dtype or f32");
    if (!norm_kind(p.post_norm) || !norm_kind(p.pre_norm)) return op_fail(GAM_ERR_INVALID_ARG, "unknown norm");
    if (p.gate_act < GAM_ACT_NONE || p.gate_act > GAM_ACT_TANH) return op_fail(GAM_ERR_INVALID_ARG, "unknown gate_act");
    if (p.rows < 0 || p.d < 1) return op_fail(GAM_ERR_INVALID_ARG, "rows >= 0 and d >= 1");
    if (p.d > 16384) return op_fail(GAM_ERR_CAPACITY, "d above 16384");
    if ((p.post_norm || p.pre_norm) && !(p.eps >= 0.f)) return op_fail(GAM_ERR_INVALID_ARG, "eps must be >= 0");
    if (p.rows == 0) return GAM_OK;
    if (!p.x || !p.y || (!p.x_out && !p.u)) return op_fail(GAM_ERR_INVALID_ARG, "null pointer");
    if (!p.gate) p.gate_rows = 1, p.gate_stride = 0;
    if (p.gate_rows < 1 || p.rows % p.gate_rows) return op_fail(GAM_ERR_SHAPE, "rows must be a multiple of gate_rows");
    if (!p.x_out) p.x_out_stride = p.x_stride;
    if (!p.u) p.u_stride = p.y_stride;
    if (p.rows == 1) p.x_stride = p.y_stride = p.x_out_stride = p.u_stride = p.gate_stride = p.d;
    if (p.rows > 1 && (p.x_stride < p.d || p.y_stride < p.d || p.x_out_stride < p.d || p.u_stride < p.d))
      return op_fail(GAM_ERR_SHAPE, "rows must be at least d apart");
    if (p.gate && p.gate_rows > 1 && p.gate_stride < p.d) return op_fail(GAM_ERR_SHAPE, "gate rows must be at least d apart");
    const int es = dtype_size(p.dtype), xs = dtype_size(p.x_dtype);
    if (!aligned(p.x, xs) || !aligned(p.x_out, xs) || !aligned(p.y, es) || !aligned(p.u, es) || !aligned(p.gate, es) ||
        !aligned(p.layer_scale, 4) || !aligned(p.post_weight, 4) || !aligned(p.post_bias, 4) ||
        !aligned(p.pre_weight, 4) || !aligned(p.pre_bias, 4))
      return op_fail(GAM_ERR_INVALID_ARG, "a buffer is not aligned to its element type");
    if ((p.x_out == p.x && p.x_out_stride != p.x_stride) || (p.u == p.y && p.u_stride != p.y_stride))
      return op_fail(GAM_ERR_INVALID_ARG, "a call in place keeps the row stride");
    if (p.u && (p.u == p.x || p.u == p.gate || p.u == p.x_out))
      return op_fail(GAM_ERR_INVALID_ARG, "u may share a buffer with y only");
    if (p.x_out && (p.x_out == p.y || p.x_out == p.gate))
      return op_fail(GAM_ERR_INVALID_ARG, "x_out may share a buffer with x only");
    int sms = 0;
    if (gam_status st = check_device(&sms)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t per_gate = p.rows / p.gate_rows;
    if (p.x_dtype == GAM_DTYPE_F32) {
      if (p.dtype == GAM_DTYPE_F32) return launch<float, float>(p, per_gate, sms, s);
      if (p.dtype == GAM_DTYPE_F16) return launch<float, __half>(p, per_gate, sms, s);
      return launch<float, bf16>(p, per_gate, sms, s);
    }
    if (p.dtype == GAM_DTYPE_F16) return launch<__half, __half>(p, per_gate, sms, s);
    return launch<bf16, bf16>(p, per_gate, sms, s);
  });
}
