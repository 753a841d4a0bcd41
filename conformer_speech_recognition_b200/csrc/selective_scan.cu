// Selective state-space scan: gam_selective_scan.
//
//   s = softplus(dt + dt_bias); h_i = exp(s a_i) h_i + s x b_i; y = (sum_i c_i h_i + skip x) z sigmoid(z)
//
// Every frame, channel and state takes one exponential, and the recurrence is
// element by element, so the bound is the exponentials (16 per clock and SM), then
// the fp32 multiply-adds; the bytes come far behind for 16 states and more.
//
// Frames in numbers (scan_kernel): a CTA takes 128 / L channels of one sequence;
// L neighbouring lanes share a channel and hold S states each in registers (S L
// >= n; states past n have a = b = c = 0).  Time goes in tiles of 8 L frames, 1024
// (frame, channel) pairs, 8 neighbouring channels of a frame to a thread: it
// fetches them one tile ahead in 16-byte accesses, forms s and s x once for the L
// lanes, and later applies skip and gate to the y the lanes have left in shared
// memory.  Inside a tile the lanes only read shared memory and their registers;
// two states go through one packed fp32 instruction.
//
// A call with few channels would leave the GPU empty and walk a long chain, so
// the time axis is split over the R CTAs of a cluster: each CTA first runs its
// piece from a zero state for the piece's end state and its sum of s (the product
// of a channel's decays is exp(a sum s)), the pieces are joined in frame order
// over distributed shared memory, and each CTA runs its piece again from its true
// state.  Twice the exponentials, R times the SMs.
//
// Few frames (step_kernel, t_max <= 4): the states are the traffic; a thread holds
// 4 states (one 16-byte access) and keeps them in registers over the frames.
#include <cooperative_groups.h>

#include <algorithm>

#include "stream_ops.cuh"

namespace gam {
namespace ops {
namespace {

namespace cg = cooperative_groups;

constexpr float kLog2e = 1.4426950408889634f;
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
__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// log(1 + e^v) = max(v, 0) + log1p(e), e = e^-|v| in (0, 1].  log1p(e) = 2 atanh(w)
// with w = e / (2 + e) <= 1/3, by its series to w^13: the rest is below 2 w^15 / 15,
// 1.5e-8 of the sum, and nothing cancels, so small steps keep their digits.
__device__ __forceinline__ float softplus_f(float v) {
  const float e = exp2_approx(-fabsf(v) * kLog2e);
  const float w = e * rcp_approx(2.f + e), w2 = w * w;
  float q = fmaf(w2, 1.f / 13, 1.f / 11);
  q = fmaf(w2, q, 1.f / 9);
  q = fmaf(w2, q, 1.f / 7);
  q = fmaf(w2, q, 1.f / 5);
  q = fmaf(w2, q, 1.f / 3);
  q = fmaf(w2 * q, w, w);
  return v != v ? v : fmaf(2.f, q, fmaxf(v, 0.f));
}
__device__ __forceinline__ float gate_f(float z) { return z * rcp_approx(1.f + exp2_approx(-z * kLog2e)); }

__device__ __forceinline__ int length_of(const gam_scan_args& p, int b) {
  return p.lengths ? min(max(p.lengths[b], 0), p.t_max) : p.t_max;
}

constexpr int kThreads = 128;

// One value's bits, zero-extended: a load that nothing has to wait for before its use.
__device__ __forceinline__ uint32_t load_bits(const float* p) { return __float_as_uint(*p); }
__device__ __forceinline__ uint32_t load_bits(const __half* p) { return *reinterpret_cast<const unsigned short*>(p); }
__device__ __forceinline__ uint32_t load_bits(const bf16* p) { return *reinterpret_cast<const unsigned short*>(p); }
template <typename T>
__device__ __forceinline__ float from_bits(uint32_t u);
template <>
__device__ __forceinline__ float from_bits<float>(uint32_t u) { return __uint_as_float(u); }
template <>
__device__ __forceinline__ float from_bits<__half>(uint32_t u) {
  return __half2float(__ushort_as_half((unsigned short)u));
}
template <>
__device__ __forceinline__ float from_bits<bf16>(uint32_t u) { return __uint_as_float(u << 16); }

// 8 neighbouring channels of a frame as they lie in memory: 16-byte accesses where
// WIDE (rows 16-byte aligned, d a multiple of 8), else value by value.  Channels
// past d and frames past the end are 0.
template <typename T, bool WIDE>
struct Octet {
  static constexpr int N = WIDE ? 8 * sizeof(T) / 16 : 8;
  uint4 q[WIDE ? N : 1];
  uint32_t u[WIDE ? 1 : N];
  __device__ __forceinline__ void load(const T* p, bool on, int left) {
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        q[i] = make_uint4(0, 0, 0, 0);
        if (on) q[i] = *reinterpret_cast<const uint4*>(p + i * (16 / sizeof(T)));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] = 0;
        if (on && i < left) u[i] = load_bits(p + i);
      }
    }
  }
  __device__ __forceinline__ float get(int k) const {  // k known at compile time
    if constexpr (!WIDE) {
      return from_bits<T>(u[k]);
    } else {
      const uint4& v = q[k * sizeof(T) / 16];
      const int w = k * sizeof(T) / 4 % 4;
      const uint32_t word = w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
      if constexpr (sizeof(T) == 4) return from_bits<T>(word);
      else return from_bits<T>((k & 1) ? word >> 16 : word & 0xffffu);
    }
  }
};

template <typename T, int S, int L, bool WIDE>
__global__ void __launch_bounds__(kThreads) scan_kernel(const gam_scan_args p) {
  constexpr int CT = kThreads / L, TT = 1024 / CT, NP = S * L;
  constexpr int OCT = CT / 8;                        // groups of 8 channels in a row of the tile
  constexpr int BC = (TT * NP + kThreads - 1) / kThreads;  // values of b (and of c) a thread stages
  // (s, s x); the 16-byte chunk j of the 8 channels o lies at j ^ (o / 2) % 4, for the banks
  __shared__ __align__(16) float2 s_in[TT][CT];
  __shared__ __align__(16) float s_b[TT][NP], s_c[TT][NP];
  __shared__ __align__(16) float s_y[TT][CT];
  // per rank: the end states of its piece [CT][NP], then its sums of s [CT] (only in a cluster)
  extern __shared__ __align__(16) float s_join[];
  constexpr int JOIN = CT * (NP + 1);
  cg::cluster_group cluster = cg::this_cluster();
  const int R = cluster.num_blocks(), rank = cluster.block_rank();
  const int cblocks = (p.d + CT - 1) / CT;
  const int item = blockIdx.x / R;
  const int cb = item % cblocks, b = item / cblocks, c0 = cb * CT;
  const int tid = threadIdx.x, part = tid % L, ch = tid / L;
  const int len = length_of(p, b);
  // this CTA's piece of the valid frames, whole tiles
  const int piece = ((len + R - 1) / R + TT - 1) / TT * TT;
  const int lo = min(rank * piece, len), hi = min(lo + piece, len);

  const bool ch_on = c0 + ch < p.d;
  const int cc = ch_on ? c0 + ch : p.d - 1;          // lanes past the last channel walk along, for the shuffles
  u64 a[S / 2], h[S / 2];
#pragma unroll
  for (int i = 0; i < S / 2; ++i) {
    const int k = part * S + 2 * i;
    a[i] = pack2(k < p.n ? p.a[(int64_t)cc * p.n + k] * kLog2e : 0.f,
                 k + 1 < p.n ? p.a[(int64_t)cc * p.n + k + 1] * kLog2e : 0.f);
    h[i] = 0ull;
  }
  if (rank == 0 && p.state_in) {
    const float* st = p.state_in + ((int64_t)b * p.d + cc) * p.n;
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
      const int k = part * S + 2 * i;
      h[i] = pack2(k < p.n ? st[k] : 0.f, k + 1 < p.n ? st[k + 1] : 0.f);
    }
  }

  // staging: thread -> frame tt of the tile, channels c8 .. c8 + 7
  const int o8 = tid % OCT, tt = tid / OCT, c8 = c0 + o8 * 8, left = p.d - c8;
  const int mine = (ch / 8 * 4 + ((ch % 8 / 2) ^ (ch / 16 % 4))) * 2 + ch % 2;  // this lane's channel in s_in
  const T* px = (const T*)p.x + b * p.x_batch_stride + c8;
  const T* pdt = (const T*)p.dt + b * p.dt_batch_stride + c8;
  const T* pz = p.z ? (const T*)p.z + b * p.z_batch_stride + c8 : nullptr;
  const T* pb = (const T*)p.b + b * p.b_batch_stride;
  const T* pc = (const T*)p.c + b * p.c_batch_stride;
  T* py = (T*)p.y + b * p.y_batch_stride + c8;
  float bias[8], skip[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    bias[k] = p.dt_bias && k < left ? p.dt_bias[c8 + k] : 0.f;
    skip[k] = p.d_skip && k < left ? p.d_skip[c8 + k] : 0.f;
  }

  // One run over the piece; OUT: with outputs, else for the end state alone.
  auto pass = [&](auto out_tag, float& sum_s) {
    constexpr bool OUT = decltype(out_tag)::value;
    Octet<T, WIDE> x, dt, z, nx, ndt, nz;
    uint32_t nb[BC], nc[BC];
    auto fetch = [&](int t0) {
      const int t = t0 + tt;
      const bool on = t < hi && left > 0;
      nx.load(px + t * p.x_row_stride, on, left);
      ndt.load(pdt + t * p.dt_row_stride, on, left);
      if (OUT && pz) nz.load(pz + t * p.z_row_stride, on, left);
#pragma unroll
      for (int i = 0; i < BC; ++i) {
        const int e = tid + i * kThreads, r = t0 + e / NP, k = e % NP;
        const bool use = e < TT * NP && r < hi && k < p.n;
        nb[i] = nc[i] = 0;
        if (use) nb[i] = load_bits(pb + r * p.b_row_stride + k);
        if (OUT && use) nc[i] = load_bits(pc + r * p.c_row_stride + k);
      }
    };
    if (lo < hi) fetch(lo);
    for (int t0 = lo; t0 < hi; t0 += TT) {
      x = nx, dt = ndt;
      if (OUT && pz) z = nz;
      const bool on = t0 + tt < hi;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4 q;
        float s[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          s[k] = dt.get(2 * j + k) + bias[2 * j + k];
          if (p.dt_softplus) s[k] = softplus_f(s[k]);
          if (!on) s[k] = 0.f;                       // a frame past the end changes nothing: x is 0 there too
        }
        q = make_float4(s[0], s[0] * x.get(2 * j), s[1], s[1] * x.get(2 * j + 1));
        *reinterpret_cast<float4*>(&s_in[tt][o8 * 8 + (j ^ (o8 / 2 % 4)) * 2]) = q;
      }
#pragma unroll
      for (int i = 0; i < BC; ++i) {
        const int e = tid + i * kThreads;
        if (e < TT * NP) {
          s_b[e / NP][e % NP] = from_bits<T>(nb[i]);
          if (OUT) s_c[e / NP][e % NP] = from_bits<T>(nc[i]);
        }
      }
      __syncthreads();
      if (t0 + TT < hi) fetch(t0 + TT);
#pragma unroll 1
      for (int t4 = 0; t4 < TT; t4 += 4) {
        float v[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int t = t4 + f;
          const float2 in = s_in[t][mine];
          const u64 s2 = pack2(in.x, in.x), sx2 = pack2(in.y, in.y);
          if (!OUT) sum_s += in.x;
          u64 y2 = 0ull;
#pragma unroll
          for (int i = 0; i < S / 4; ++i) {
            const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(&s_b[t][part * S + 4 * i]);
            ulonglong2 cv;
            if (OUT) cv = *reinterpret_cast<const ulonglong2*>(&s_c[t][part * S + 4 * i]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float2 e = unpack2(mul2(s2, a[2 * i + k]));
              const u64 decay = pack2(exp2_approx(e.x), exp2_approx(e.y));
              h[2 * i + k] = fma2(decay, h[2 * i + k], mul2(sx2, k ? bv.y : bv.x));
              if (OUT) y2 = i + k ? fma2(k ? cv.y : cv.x, h[2 * i + k], y2) : mul2(cv.x, h[0]);
            }
          }
          const float2 yy = unpack2(y2);
          if (OUT) v[f] = yy.x + yy.y;
        }
        if constexpr (OUT) {
          // the lanes of a channel add their parts of 4 frames; with L >= 2 each ends with its own share of the frames
          if constexpr (L == 1) {
#pragma unroll
            for (int f = 0; f < 4; ++f) s_y[t4 + f][ch] = v[f];
          } else {
            const bool up = part & 1;
            float w[2];
#pragma unroll
            for (int f = 0; f < 2; ++f)
              w[f] = (up ? v[f + 2] : v[f]) + __shfl_xor_sync(0xffffffffu, up ? v[f] : v[f + 2], 1);
            if constexpr (L == 2) {
#pragma unroll
              for (int f = 0; f < 2; ++f) s_y[t4 + (up ? 2 : 0) + f][ch] = w[f];
            } else {
              const bool up2 = part & 2;
              float q = (up2 ? w[1] : w[0]) + __shfl_xor_sync(0xffffffffu, up2 ? w[0] : w[1], 2);
#pragma unroll
              for (int o = 4; o < L; o <<= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
              if (part < 4) s_y[t4 + (up ? 2 : 0) + (up2 ? 1 : 0)][ch] = q;
            }
          }
        }
      }
      __syncthreads();
      if (OUT && on && left > 0) {
        T o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float v = fmaf(skip[k], x.get(k), s_y[tt][o8 * 8 + k]);
          if (pz) v *= gate_f(z.get(k));
          o[k] = from_f<T>(v);
        }
        T* dst = py + (t0 + tt) * p.y_row_stride;
        if constexpr (WIDE) {
          constexpr int V = 16 / sizeof(T);
#pragma unroll
          for (int i = 0; i < 8 / V; ++i) {
            Vec<T, V> q;
#pragma unroll
            for (int k = 0; k < V; ++k) q.v[k] = o[i * V + k];
            *reinterpret_cast<Vec<T, V>*>(dst + i * V) = q;
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < left) dst[k] = o[k];
        }
      }
    }
  };

  float sum_s = 0.f;
  if (R > 1) {
    if (rank == 0) pass(std::true_type(), sum_s);    // the first piece knows its state
    else if (rank < R - 1) pass(std::false_type(), sum_s);
    cluster.sync();                                  // every CTA of the cluster has started: its shared memory is there
    // to every later piece (stores over the cluster need no answer; loads were ten times slower)
    for (int r = rank + 1; r < R; ++r) {
      float* to = cluster.map_shared_rank(s_join, r) + rank * JOIN;
#pragma unroll
      for (int i = 0; i < S / 4; ++i)
        *reinterpret_cast<ulonglong2*>(to + ch * NP + part * S + 4 * i) = make_ulonglong2(h[2 * i], h[2 * i + 1]);
      if (part == 0) to[CT * NP + ch] = sum_s;
    }
    cluster.sync();
    if (rank > 0) {
      for (int r = 0; r < rank; ++r) {
        const float* e = s_join + r * JOIN;
        const float q = e[CT * NP + ch];
#pragma unroll
        for (int i = 0; i < S / 4; ++i) {
          const ulonglong2 end = *reinterpret_cast<const ulonglong2*>(e + ch * NP + part * S + 4 * i);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 x2 = unpack2(mul2(pack2(q, q), a[2 * i + k]));
            const u64 decay = pack2(exp2_approx(x2.x), exp2_approx(x2.y));
            // the first piece's end state is whole already
            h[2 * i + k] = r ? fma2(decay, h[2 * i + k], k ? end.y : end.x) : (k ? end.y : end.x);
          }
        }
      }
      pass(std::true_type(), sum_s);
    }
  } else {
    pass(std::true_type(), sum_s);
  }

  if (rank == R - 1 && p.state_out && ch_on) {
    float* st = p.state_out + ((int64_t)b * p.d + cc) * p.n;
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
      const int k = part * S + 2 * i;
      const float2 v = unpack2(h[i]);
      if (k < p.n) st[k] = v.x;
      if (k + 1 < p.n) st[k + 1] = v.y;
    }
  }
  // frames behind the end are zero
  for (int t = len + rank * TT + tt; t < p.t_max; t += R * TT)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) py[t * p.y_row_stride + k] = from_f<T>(0.f);
}

// A few frames: L lanes of 4 states to a channel, neighbouring lanes on neighbouring memory.
template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(256) step_kernel(const gam_scan_args p) {
  constexpr int CT = 256 / L;
  const int cblocks = (p.d + CT - 1) / CT;
  const int cb = blockIdx.x % cblocks, b = blockIdx.x / cblocks;
  const int part = threadIdx.x % L, c0 = cb * CT + threadIdx.x / L;
  const bool on = c0 < p.d;
  const int c = on ? c0 : p.d - 1;                   // lanes past the last channel walk along, for the shuffles
  const int k0 = part * 4;
  const int len = length_of(p, b);
  const int64_t at = ((int64_t)b * p.d + c) * p.n + k0;
  float a[4] = {}, h[4] = {};
  if constexpr (VEC) {                               // n a multiple of 4, 16-byte aligned
    if (k0 < p.n) {
      const float4 q = *reinterpret_cast<const float4*>(p.a + (int64_t)c * p.n + k0);
      a[0] = q.x, a[1] = q.y, a[2] = q.z, a[3] = q.w;
      if (p.state_in) {
        const float4 w = *reinterpret_cast<const float4*>(p.state_in + at);
        h[0] = w.x, h[1] = w.y, h[2] = w.z, h[3] = w.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k0 + i < p.n) {
        a[i] = p.a[(int64_t)c * p.n + k0 + i];
        if (p.state_in) h[i] = p.state_in[at + i];
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] *= kLog2e;
  const float skip = p.d_skip ? p.d_skip[c] : 0.f, bias = p.dt_bias ? p.dt_bias[c] : 0.f;
  T* y = (T*)p.y + b * p.y_batch_stride + c;
  for (int t = 0; t < len; ++t) {
    const T* bb = (const T*)p.b + b * p.b_batch_stride + t * p.b_row_stride + k0;
    const T* cc = (const T*)p.c + b * p.c_batch_stride + t * p.c_row_stride + k0;
    const float xv = to_f(((const T*)p.x)[b * p.x_batch_stride + t * p.x_row_stride + c]);
    float s = to_f(((const T*)p.dt)[b * p.dt_batch_stride + t * p.dt_row_stride + c]) + bias;
    const float z = p.z ? to_f(((const T*)p.z)[b * p.z_batch_stride + t * p.z_row_stride + c]) : 0.f;
    float bv[4], cv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bv[i] = k0 + i < p.n ? to_f(bb[i]) : 0.f;
      cv[i] = k0 + i < p.n ? to_f(cc[i]) : 0.f;
    }
    if (p.dt_softplus) s = softplus_f(s);
    const float sx = s * xv;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fmaf(exp2_approx(s * a[i]), h[i], sx * bv[i]);
      v = fmaf(cv[i], h[i], v);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    v = fmaf(skip, xv, v);
    if (p.z) v *= gate_f(z);
    if (on && part == 0) y[t * p.y_row_stride] = from_f<T>(v);
  }
  if (on && part == 0)
    for (int t = len; t < p.t_max; ++t) y[t * p.y_row_stride] = from_f<T>(0.f);
  if (!on || !p.state_out) return;
  if constexpr (VEC) {
    if (k0 < p.n) *reinterpret_cast<float4*>(p.state_out + at) = make_float4(h[0], h[1], h[2], h[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k0 + i < p.n) p.state_out[at + i] = h[i];
  }
}

template <typename T, int L>
gam_status launch_step(const gam_scan_args& p, cudaStream_t s) {
  const int64_t grid = (int64_t)((p.d + 256 / L - 1) / (256 / L)) * p.batch;
  if (grid > INT32_MAX) return op_fail(GAM_ERR_CAPACITY, "batch * d too large for one call");
  const bool vec = p.n % 4 == 0 && aligned(p.a, 16) && aligned(p.state_in, 16) && aligned(p.state_out, 16);
  if (vec) step_kernel<T, L, true><<<(unsigned)grid, 256, 0, s>>>(p);
  else step_kernel<T, L, false><<<(unsigned)grid, 256, 0, s>>>(p);
  return launch_status(cudaGetLastError());
}

template <typename T, int S, int L>
gam_status launch_scan(const gam_scan_args& p, int sms, cudaStream_t s) {
  constexpr int CT = kThreads / L, TT = 1024 / CT;
  const int64_t ctas = (int64_t)((p.d + CT - 1) / CT) * p.batch;
  // split while the pieces keep two tiles and the CTAs do not fill the SMs four times
  int R = 1;
  while (R < 8 && ctas * R * 2 <= (int64_t)sms * 4 && p.t_max >= R * 2 * 2 * TT) R *= 2;
  if (R == 2) R = 1;                                 // twice the work for twice the SMs gains nothing
  if (ctas * R > INT32_MAX) return op_fail(GAM_ERR_CAPACITY, "batch * d too large for one call");
  constexpr int V = 16 / sizeof(T);
  const bool wide = p.d % 8 == 0 && aligned(p.x, 16) && aligned(p.dt, 16) && aligned(p.z, 16) && aligned(p.y, 16) &&
                    p.x_batch_stride % V == 0 && p.x_row_stride % V == 0 && p.dt_batch_stride % V == 0 &&
                    p.dt_row_stride % V == 0 && p.z_batch_stride % V == 0 && p.z_row_stride % V == 0 &&
                    p.y_batch_stride % V == 0 && p.y_row_stride % V == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas * R));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.dynamicSmemBytes = R > 1 ? (R - 1) * CT * (S * L + 1) * sizeof(float) : 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = R;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = wide ? scan_kernel<T, S, L, true> : scan_kernel<T, S, L, false>;
  if (R > 1) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return launch_status(e);
  }
  return launch_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

template <typename T>
gam_status launch(const gam_scan_args& p, int sms, cudaStream_t s) {
  if (p.t_max <= 4) {
    if (p.n <= 4) return launch_step<T, 1>(p, s);
    if (p.n <= 8) return launch_step<T, 2>(p, s);
    if (p.n <= 16) return launch_step<T, 4>(p, s);
    if (p.n <= 32) return launch_step<T, 8>(p, s);
    return launch_step<T, 16>(p, s);
  }
  if (p.n <= 4) return launch_scan<T, 4, 1>(p, sms, s);
  if (p.n <= 8) return launch_scan<T, 8, 1>(p, sms, s);
  if (p.n <= 16) return launch_scan<T, 8, 2>(p, sms, s);
  if (p.n <= 32) return launch_scan<T, 8, 4>(p, sms, s);
  return launch_scan<T, 16, 4>(p, sms, s);
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
    if (p.dtype == GAM_DTYPE_F32) return launch<float>(p, sms, s);
    if (p.dtype == GAM_DTYPE_F16) return launch<__half>(p, sms, s);
    return launch<bf16>(p, sms, s);
  });
}
