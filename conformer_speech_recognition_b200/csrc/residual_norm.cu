// Residual update with the norms around it: gam_residual_norm.
//
//   x' = x + alpha * layer_scale * gate_act(gate) * post_norm(y),  u = pre_norm(x')
//
// One pass: a group of G threads (a warp, or a CTA for wide or few rows) holds a
// row of y and x in registers, so each is read once; all loads of a row are on
// their way before the first is used, and a warp's next row while it works on
// this one.  Statistics are two-pass in fp32 (mean, then the centred squares)
// over those registers.  The bound is memory: 23968 rows of 1024 (fp32 residual, fp16
// branch, 295 MB) in 59 us, 5.0 TB/s; a CTA to each of those rows 69 us.
//
// Accesses are 16 bytes where rows are 16-byte aligned.  Else they are pairs of
// values: a row of odd offset starts with the second half of a pair, so pair i
// holds columns 2 i - phase and the next, phase being the offset's last bit, and
// every whole pair is aligned whatever the row.  Without that (arrays whose rows
// differ in that bit) they are single values.  2047 rows of 4099 in bf16 with a gate: 37 us
// in pairs (2.3 TB/s; its 4-byte accesses and the parameters' single ones take 21.2 M
// instructions, at 2.2 a clock), 79 us in single values.
#include <algorithm>

#include "stream_ops.cuh"

namespace gam {
namespace ops {
namespace {

// Sum over the G threads of a row: a warp by shuffles, a CTA through shared
// memory (red holds two alternating sets of 32 partial sums, so one barrier per
// sum is enough).
template <int G>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (G == 32) return v;
  const int lane = threadIdx.x & 31;
  float* r = red[turn];
  turn ^= 1;
  if (lane == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < G / 32 ? r[lane] : 0.f;
#pragma unroll
  for (int o = G / 64; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return __shfl_sync(0xffffffffu, v, 0);
}

// A thread's part of a row: accesses j < NV of V columns from j G V + first on, first being
// its own multiple of V less the phase (pairs).  G is known at compile time, so that an
// access is one base register and a constant.  Only a pair can lie partly beside the row.
// The first FULL accesses lie in the row for every thread (the row is long enough), but for
// the column before the first.
template <int G, int V, int FULL>
struct Place {
  int first, d;
  __device__ __forceinline__ bool on(int j, int i) const {
    if (j < FULL) return V != 2 || j > 0 || i > 0 || first >= 0;
    return (unsigned)(first + j * G * V + i) < (unsigned)d;
  }
  __device__ __forceinline__ bool whole(int j) const { return on(j, 0) && (V != 2 || on(j, 1)); }
};

// The row's values; 0 for what lies beside it, which is not read.  Whole accesses first,
// then the halves of cut pairs, so that nothing waits on the way.
template <int G, int V, int NV, int FULL, typename T>
__device__ __forceinline__ void load_row(Raw<T, V> (&r)[NV], const T* row, const Place<G, V, FULL>& at) {
  const T* mine = row + at.first;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    r[j].zero();
    if (at.whole(j)) r[j].load(mine + j * G * V);
  }
  if constexpr (V == 2) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if ((j == 0 || j >= FULL) && at.on(j, 0) != at.on(j, 1)) {
        const int i = at.on(j, 1);
        Raw<T, 1> one;
        one.load(mine + j * G * V + i);
        if constexpr (sizeof(T) == 4) r[j].w[i] = one.w[0];
        else r[j].w[0] = one.w[0] << (16 * i);
      }
  }
}
template <int G, int V, int NV, int FULL, typename T>
__device__ __forceinline__ void store_row(T* row, const Place<G, V, FULL>& at, const float (&v)[NV][V]) {
  T* mine = row + at.first;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (at.whole(j)) {
      Raw<T, V> o;
      o.set(v[j]);
      o.store(mine + j * G * V);
    } else if constexpr (V == 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (at.on(j, i)) mine[j * G * V + i] = from_f<T>(v[j][i]);
    }
  }
}
// Access j of a parameter vector [d]; 0 beside the row.
template <int G, int V, int FULL>
__device__ __forceinline__ void load_param(float (&out)[V], const float* p, const Place<G, V, FULL>& at, int j) {
  const float* mine = p + at.first + j * G * V;
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = 0.f;
  if constexpr (V <= 2) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at.on(j, i)) out[i] = __ldg(mine + i);
  } else if (at.whole(j)) {  // 16-byte aligned with the rows
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(mine) + i);
      out[4 * i] = f.x, out[4 * i + 1] = f.y, out[4 * i + 2] = f.z, out[4 * i + 3] = f.w;
    }
  }
}

// v <- norm(v) over the row; v is 0 beside it, before and after.
template <int G, int V, int NV, int FULL>
__device__ __forceinline__ void norm_row(float (&v)[NV][V], bool layer, const float* w, const float* b, float eps,
                                         const Place<G, V, FULL>& at, float (*red)[32], int& turn) {
  // one access a thread: its weights come while the row is summed
  float w0[V], b0[V];
  if constexpr (NV == 1) {
    if (w) load_param<G, V, FULL>(w0, w, at, 0);
    if (b) load_param<G, V, FULL>(b0, b, at, 0);
  }
  const float inv = 1.f / at.d;
  if (layer) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) s += v[j][i];
    const float mean = row_sum<G>(s, red, turn) * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] = at.on(j, V == 2 ? i : 0) ? v[j][i] - mean : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) q = fmaf(v[j][i], v[j][i], q);
  const float r = rsqrtf(fmaf(row_sum<G>(q, red, turn), inv, eps));
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) v[j][i] *= r;
  if (w)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (NV > 1) load_param<G, V, FULL>(w0, w, at, j);
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] *= w0[i];
    }
  if (b)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (NV > 1) load_param<G, V, FULL>(b0, b, at, j);
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] += b0[i];
    }
}

constexpr int kWarps = 4;  // rows of a CTA at a time in the warp form

// GATE: 0 none, 1 as it is, 2 its sigmoid or swish, 3 its tanh.  In one kernel the largest of them took the registers
// of all: 4562 rows of 4520, fp32 + fp16, plain gate 94 us, 56 apart.
template <typename TX, typename TY, int G, int V, int NV, int FULL, int GATE>
__global__ void __launch_bounds__(G == 32 ? 32 * kWarps : G, G == 32 ? (NV == 4 ? 3 : 5) : NV * V <= 12 ? 1024 / G : 1)
residual_norm_kernel(const gam_residual_norm_args p, const int64_t per_gate) {
  constexpr bool WARP = G == 32;
  __shared__ float red[2][32];
  const int64_t step = WARP ? (int64_t)gridDim.x * kWarps : (int64_t)gridDim.x;
  int64_t row = WARP ? (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const int own = (int)(WARP ? threadIdx.x & 31 : threadIdx.x) * V;
  const float* post_b = p.post_norm == GAM_NORM_LAYER ? p.post_bias : nullptr;
  const float* pre_b = p.pre_norm == GAM_NORM_LAYER ? p.pre_bias : nullptr;
  Place<G, V, FULL> at{own, p.d};
  Raw<TX, V> rx[NV];
  Raw<TY, V> ry[NV], rg[GATE ? NV : 1];
  auto fetch = [&](int64_t r) {
    if constexpr (V == 2) at.first = own - ((int)(r * p.y_stride) & 1);
    load_row<G, V, NV, FULL>(ry, (const TY*)p.y + r * p.y_stride, at);
    load_row<G, V, NV, FULL>(rx, (const TX*)p.x + r * p.x_stride, at);
    if constexpr (GATE != 0) load_row<G, V, NV, FULL>(rg, (const TY*)p.gate + r / per_gate * p.gate_stride, at);
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
        if constexpr (GATE != 0) g[j][i] = rg[j].get(i);
      }
    const Place<G, V, FULL> here = at;
    if (WARP && row + step < p.rows) fetch(row + step);
    if (p.post_norm)
      norm_row<G, V, NV, FULL>(y, p.post_norm == GAM_NORM_LAYER, p.post_weight, post_b, p.eps, here, red, turn);
    if constexpr (GATE != 0) {
      auto gate = [&](auto act) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) y[j][i] *= act(g[j][i]);
      };
      auto gate2 = [&](auto act) {                     // of pairs
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const float2 f = unpack2(act(pack2(g[j][i], g[j][i + 1])));
            y[j][i] *= f.x;
            y[j][i + 1] *= f.y;
          }
      };
      constexpr bool PAIRS = sizeof(TX) == 4 && V > 1; // a factor of the residual: in its type's precision
      if constexpr (GATE == 1) {
        gate([](float v) { return v; });
      } else if constexpr (GATE == 3) {
        gate([](float v) { return tanhf(v); });
      } else if (p.gate_act == GAM_ACT_SWISH) {
        if constexpr (PAIRS) gate2([](u64 v) { return swish2(v); });
        else gate([](float v) { return swish_f<TX>(v); });
      } else {
        if constexpr (PAIRS) gate2([](u64 v) { return sigmoid2(v); });
        else gate([](float v) { return sigmoid_f<TX>(v); });
      }
    }
    if (p.layer_scale)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float ls[V];
        load_param<G, V, FULL>(ls, p.layer_scale, here, j);
#pragma unroll
        for (int i = 0; i < V; ++i) y[j][i] *= ls[i];
      }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) x[j][i] = fmaf(p.alpha, y[j][i], x[j][i]);
    if (p.x_out) store_row<G, V, NV, FULL>((TX*)p.x_out + row * p.x_out_stride, here, x);
    if (p.u) {
      if (p.pre_norm)
        norm_row<G, V, NV, FULL>(x, p.pre_norm == GAM_NORM_LAYER, p.pre_weight, pre_b, p.eps, here, red, turn);
      store_row<G, V, NV, FULL>((TY*)p.u + row * p.u_stride, here, x);
    }
    row += step;
    if (!WARP || row >= p.rows) return;
  }
}

template <typename TX, typename TY, int V, int GATE>
gam_status launch_v(const gam_residual_norm_args& p, int64_t per_gate, int sms, cudaStream_t s) {
  if (p.rows > INT32_MAX) return op_fail(GAM_ERR_CAPACITY, "too many rows for one call");
  const int vecs = (p.d + V - 1) / V + (V == 2);  // a phase can cut one pair in two
  auto warps = [&](auto kernel, int per_sm) {     // warps walk over the rows
    const int64_t groups = (p.rows + kWarps - 1) / kWarps;
    const unsigned grid = (unsigned)std::min<int64_t>(groups, (int64_t)sms * per_sm);
    return launch_status(launch_kernel(kernel, grid, 32 * kWarps, 0, s, p, per_gate));
  };
  auto cta = [&](auto kernel, int threads) {      // a CTA to a row; walking over them was slower
    return launch_status(launch_kernel(kernel, (unsigned)p.rows, threads, 0, s, p, per_gate));
  };
#define GAM_WARPS(NV, FULL, PER_SM) return warps(residual_norm_kernel<TX, TY, 32, V, NV, FULL, GATE>, PER_SM)
#define GAM_CTA(G, NV, FULL) return cta(residual_norm_kernel<TX, TY, G, V, NV, FULL, GATE>, G)
  // Rows enough for 8 warps to an SM: a warp holds a row, up to 4 accesses to a lane; else a CTA holds it.
  const bool many = p.rows >= 8 * sms;
  // (accesses, of which whole in every row of this branch's lengths; vecs counts one pair more than a row may have)
  if constexpr (V > 2) {
    if (vecs <= 32) GAM_WARPS(1, 0, 8);
    if (vecs <= 64 && many) GAM_WARPS(2, 1, 5);
    if (vecs <= 128 && many) GAM_WARPS(4, 2, 3);
    if (vecs <= 128) GAM_CTA(128, 1, 0);
    if (vecs <= 256) GAM_CTA(256, 1, 0);
    if (vecs <= 512) GAM_CTA(512, 1, 0);
    if (vecs <= 768) GAM_CTA(256, 3, 2);
    if (vecs <= 1024) GAM_CTA(512, 2, 1);
    if constexpr (V == 4) {
      if (vecs > 2048) GAM_CTA(512, 8, 4);
    }
    GAM_CTA(512, 4, 2);
  } else if constexpr (V == 2) {
    if (vecs <= 32) GAM_WARPS(1, 0, 8);
    if (vecs <= 128 && many) GAM_WARPS(4, 0, 3);
    if (vecs <= 384) GAM_CTA(128, 3, 0);
    if (vecs <= 768) GAM_CTA(256, 3, 1);
    if (vecs <= 1536) GAM_CTA(512, 3, 1);
    if (vecs <= 2560) GAM_CTA(512, 5, 2);
    if (vecs <= 4096) GAM_CTA(512, 8, 4);
    GAM_CTA(512, 16, 7);
  } else {
    if (vecs <= 2048) GAM_CTA(512, 4, 0);
    GAM_CTA(1024, 16, 2);
  }
#undef GAM_WARPS
#undef GAM_CTA
}

template <typename TX, typename TY, int V>
gam_status launch_g(const gam_residual_norm_args& p, int64_t per_gate, int sms, cudaStream_t s) {
  if (!p.gate) return launch_v<TX, TY, V, 0>(p, per_gate, sms, s);
  if (p.gate_act == GAM_ACT_SWISH || p.gate_act == GAM_ACT_SIGMOID) return launch_v<TX, TY, V, 2>(p, per_gate, sms, s);
  if (p.gate_act == GAM_ACT_TANH) return launch_v<TX, TY, V, 3>(p, per_gate, sms, s);
  return launch_v<TX, TY, V, 1>(p, per_gate, sms, s);
}

template <typename TX, typename TY>
gam_status launch(const gam_residual_norm_args& p, int64_t per_gate, int sms, cudaStream_t s) {
  constexpr int V = 16 / sizeof(TY);
  auto bases = [&](size_t align_x, size_t align_y) {
    return aligned(p.x, align_x) && aligned(p.x_out, align_x) && aligned(p.y, align_y) && aligned(p.u, align_y) &&
           aligned(p.gate, align_y);
  };
  const int64_t strides[5] = {p.x_stride, p.y_stride, p.x_out_stride, p.u_stride, p.gate_stride};
  bool wide = p.d % V == 0 && bases(16, 16) && aligned(p.layer_scale, 16) && aligned(p.post_weight, 16) &&
              aligned(p.post_bias, 16) && aligned(p.pre_weight, 16) && aligned(p.pre_bias, 16);
  bool pairs = p.d < 16382 && bases(2 * sizeof(TX), 2 * sizeof(TY));  // 16 pairs to each of 512 threads, and a cut one
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
