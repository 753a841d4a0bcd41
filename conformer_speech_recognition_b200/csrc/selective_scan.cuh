// Selective state-space scan: the kernels of gam_selective_scan and their launch for one
// type (each type is a translation unit of its own, so that they compile in parallel).
//
//   s = softplus(dt + dt_bias); h_i = exp(s a_i) h_i + s x b_i; y = (sum_i c_i h_i + skip x) z sigmoid(z)
//
// Every frame, channel and state takes one exponential, and the recurrence is
// element by element, so the bound is the exponentials (16 per clock and SM), then
// the fp32 multiply-adds; the bytes come far behind for 16 states and more.
//
// Frames in numbers (scan_kernel): a CTA takes 64 / L channels (or twice as many) of
// one sequence; L neighbouring lanes share a channel and hold S states each in
// registers (S L >= n; states past n have a = b = c = 0).  Time goes in tiles of 512
// (frame, channel) pairs.  A producer's share of a tile is 8 neighbouring channels of a
// frame: it copies them ahead, forms s and s x once for the L lanes, and later applies
// skip and gate to the y the lanes have left in shared memory.  Inside a tile the lanes
// only read shared memory and their registers; two states go through one packed fp32
// instruction.  Small calls, where a tile's latency counts, have producer warps beside the
// lanes (2 x 4011 frames of 192 channels: 96 us without them, 63 with); in large calls a
// thread does both, with two channels to a lane (32 x 390 frames of 2048 channels: 179 us,
// with producers 249), which halves the reads of b and c.
//
// What it measured (16 states): 12.5 k frames of 2048 channels in 210 us, the special-function
// pipe 56 % busy (exponentials and the gates' reciprocals) and 1.9 instructions a clock; the main loop alone, without
// the producers' work, runs at 91 % of that pipe's rate.  A share of the exponentials as polynomials on the
// fp32 pipe was slower (one pair in 4: +5 %): the instructions it adds cost more than the
// pipe it frees.
//
// A call with few channels would leave the GPU empty and walk a long chain, so
// the time axis is split over the R CTAs of a cluster: each CTA first runs its
// piece from a zero state for the piece's end state and its sum of s (the product
// of a channel's decays is exp(a sum s)), the pieces are joined in frame order
// over distributed shared memory, and each CTA runs its piece again from its true
// state.  Twice the exponentials, R times the SMs.
//
// A tile runs all its frames whatever is valid (32 with 16 states on small calls, 8 on large
// ones), so that 5 frames take the time of a tile: one stream of 2048 channels 3.6 us for 4
// frames, 4.6 for 5 to 32; 64 streams 10.5 for 4, 15.3 for 5 to 8, 34 for 32.
//
// Few frames (step_kernel, t_max <= 4): the states are the traffic; a thread holds
// 4 states of two channels (16-byte accesses) and keeps them in registers over the frames.
#pragma once

#include <cooperative_groups.h>

#include <algorithm>

#include "stream_ops.cuh"

namespace gam {
namespace ops {
namespace {

namespace cg = cooperative_groups;

// a lambda left as a call would keep the states it refers to in local memory (three times the time)
#define GAM_INLINE __attribute__((always_inline))

constexpr float kLog2e = 1.4426950408889634f;

// 2^x for two values on the fp32 and integer pipes: x = n + f, n whole and |f| <= 1/2 by
// the rounding of an addition, 2^(f+1) by the polynomial of degree 5 with 2^1 = 2 and the
// least largest relative error (8e-8; 1.6e-7 evaluated in fp32, 6e-8 for |f| < 0.001), and a
// product with 2^(n-1), whose exponent field is n + 126.  Below -125.5 the field is 0 and so
// is the result; 128 gives infinity; NaN comes through the product.
__device__ __forceinline__ float clamp_exponent(float v) {
  float r;
  asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, 0fC2FC0000;\n\tmin.NaN.f32 %0, t, 0f43000000;\n\t}" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ u64 exp2_poly2(u64 x) {
  const float2 c = unpack2(x);
  const u64 v = pack2(clamp_exponent(c.x), clamp_exponent(c.y));
  const u64 one = both(1.f);
  const u64 t = fma2(v, one, both(12583038.f));      // 1.5 * 2^23 + 126: its last bit counts ones
  const u64 f = fma2(fma2(t, one, both(-12583038.f)), both(-1.f), v);
  u64 q = both(0.0026549266185611486f);
  q = fma2(q, f, both(0.019343923777341843f));
  q = fma2(q, f, both(0.11101356893777847f));
  q = fma2(q, f, both(0.48044469952583313f));
  q = fma2(q, f, both(1.3862941265106201f));
  q = fma2(q, f, both(2.f));
  const float2 n = unpack2(t);
  return mul2(q, pack2(__int_as_float(__float_as_int(n.x) << 23), __int_as_float(__float_as_int(n.y) << 23)));
}
// A decay 2^(s a).  A state that decays slowly adds up the decays' errors over many frames: with the hardware's
// 2^x (2^-22) an fp32 call's outputs came out 1e-6 off, so fp32 calls take the polynomial.  16-bit calls keep the
// hardware's, but not its mean error: that is -6e-9 for x in -0.003 .. 0 and -2e-8 in -0.7 .. -0.003 (measured),
// so x is raised by kRaise, which the multiply-add gives for nothing and which leaves 7e-9 either way (49
// sequences of 88 frames, fp16: states 1.6e-6 off without it, 7.3e-7 with).  2^kRaise is 1 in 32 bits: a step of 0
// leaves the state as it was.
constexpr float kRaise = 1.9e-8f;
template <typename T>
__device__ __forceinline__ u64 decay2(u64 s, u64 a) {
  if constexpr (sizeof(T) == 4) return exp2_poly2(mul2(s, a));
  else return exp2_approx2(fma2(s, a, both(kRaise)));
}

// h 2^(q a) where the exponent sums up many frames and may leave fp32's range although h 2^(q a) does not: beyond
// 2^+-120 it goes in two halves.  A state of 0 or of infinity stays what it is, as it does frame by frame.
template <typename T>
__device__ __forceinline__ u64 carry2(u64 h, float q, u64 a) {
  const float2 r = unpack2(a), v = unpack2(h);
  const bool far = fmaxf(fabsf(q * r.x), fabsf(q * r.y)) > 120.f;
  const u64 decay = decay2<T>(both(far ? 0.5f * q : q), a);
  u64 w = mul2(h, decay);
  if (far) w = mul2(w, decay);
  const float2 u = unpack2(w);
  auto rigid = [](float x) { return x == 0.f || isinf(x); };
  return pack2(rigid(v.x) ? v.x : u.x, rigid(v.y) ? v.y : u.y);
}

// An infinite rate stands for the largest finite one: a step of 0, as behind a sequence's end, then keeps the
// state, where 0 times infinity would be NaN.
__device__ __forceinline__ float finite_rate(float v) { return bound_f(v, 3.4028235e38f); }

// log(1 + e^v) = max(v, 0) + log1p(e), e = e^-|v| in (0, 1], for two values; fp32 in every type, since the states
// are.  log1p(e) / e by the polynomial of degree 8 with the least largest relative error on [0, 1] (3e-8; 1.7e-7
// evaluated in fp32): nothing cancels, so small steps keep their digits.  With e within 6 u and the last product
// at most 9 u = 5.4e-7 off.  A NaN comes through e.
__device__ __forceinline__ float2 softplus2(float2 v) {
  const u64 e = exp2v(pack2(-fabsf(bound_f(v.x, 200.f)), -fabsf(bound_f(v.y, 200.f))));
  u64 q = both(0.0052326930941379795f);
  q = fma2(q, e, both(-0.02950523979961872f));
  q = fma2(q, e, both(0.07822595536708832f));
  q = fma2(q, e, both(-0.13663245737552643f));
  q = fma2(q, e, both(0.19106006622314453f));
  q = fma2(q, e, both(-0.2484298199415207f));
  q = fma2(q, e, both(0.3331909775733948f));
  q = fma2(q, e, both(-0.4999949336051941f));
  q = fma2(q, e, both(0.9999999403953552f));
  return unpack2(fma2(q, e, pack2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f))));
}

__device__ __forceinline__ int length_of(const gam_scan_args& p, int b) {
  return p.lengths ? min(max(p.lengths[b], 0), p.t_max) : p.t_max;
}

constexpr int kLanes = 64, kTile = kLanes * 8;  // lanes of a CTA, (frame, channel) pairs of a tile at most

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

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  Vec<__half2, 4> q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q.v[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<Vec<__half2, 4>*>(p) = q;
}
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) {
  Vec<__nv_bfloat162, 4> q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q.v[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<Vec<__nv_bfloat162, 4>*>(p) = q;
}

// 8 values from memory to shared memory, asynchronously; zeros where !on (nothing is read then).
template <typename T>
__device__ __forceinline__ void copy8(T* dst, const T* src, bool on) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  const int bytes = on ? 16 : 0;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + 16 * i),
                 "l"(reinterpret_cast<const char*>(src) + 16 * i), "r"(bytes)
                 : "memory");
}

// The first `bytes` (0 .. 4) of 4 bytes, zeros behind them.
template <typename T>
__device__ __forceinline__ void copy4(T* dst, const T* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}

// Frames of a tile: 8 channels of a frame to each producer, and at most 1024 values of b.
constexpr int tile_frames(int CT, int NP) { return kTile / CT < 1024 / NP ? kTile / CT : 1024 / NP; }

template <typename T, int S, int L, int CH>
struct ScanShape {
  static constexpr bool SPLIT = CH == 1;                 // producers beside the lanes
  static constexpr int THREADS = SPLIT ? 2 * kLanes : kLanes;
  static constexpr int CT1 = kLanes / L, CT = CT1 * CH;  // channels of a CTA: a lane's are ch + j CT1, j < CH
  static constexpr int NP = S * L, TT = tile_frames(CT, NP);
  static constexpr int JOIN = CT * (NP + 1);             // a piece's end states [CT][NP] and its sums of s [CT]
  // shared memory: copies as they lie in memory, then two tiles of (s, s x), b, c and y; the pieces' end
  // states take the tiles' place between two runs
  static constexpr int RAW = 9 * kTile * sizeof(T), RAW_BC = 4 * TT * NP * sizeof(T);
  static constexpr int TILES = 2 * TT * (CT * 3 + NP * 2) * sizeof(float);
  static size_t bytes(bool wide, bool pair, int R) {
    const int join = (R - 1) * JOIN * (int)sizeof(float);
    return (wide ? RAW : 0) + (pair ? RAW_BC : 0) + (join > TILES ? join : TILES);
  }
};

// States past n: with an infinite s x they would be infinity times b = 0, a NaN that reaches y through c = 0.  A lane
// that has no others adds 0 to y; where a lane has some of both kinds (PAD: n no multiple of S) they are put back to
// 0 after every frame.
template <typename T, int S, int L, int CH, bool WIDE, bool PAD>
__global__ void __launch_bounds__(ScanShape<T, S, L, CH>::THREADS, ScanShape<T, S, L, CH>::SPLIT ? 6 : 8)
scan_kernel(const gam_scan_args p, const int sms, const bool pair) {
  using Shape = ScanShape<T, S, L, CH>;
  constexpr int CT1 = Shape::CT1, CT = Shape::CT, TT = Shape::TT, NP = Shape::NP, JOIN = Shape::JOIN;
  constexpr int OCT = CT / 8;                        // groups of 8 channels in a row of the tile
  constexpr int PER = 4 / sizeof(T);                 // values of b in 4 bytes
  constexpr bool SPLIT = Shape::SPLIT;
  constexpr int kThreads = Shape::THREADS;
  __shared__ __align__(16) float s_bias[CT], s_skip[CT];
  __shared__ int s_seq;
  extern __shared__ __align__(16) uint8_t s_dyn[];
  // x, dt and z of three tiles as they lie in memory (WIDE), b and c of two (pair: their rows are 4-byte
  // aligned); a thread reads only what it copied itself
  T* const s_raw = reinterpret_cast<T*>(s_dyn);
  T* const s_raw_bc = reinterpret_cast<T*>(s_dyn + (WIDE ? Shape::RAW : 0));
  uint8_t* const s_tiles = s_dyn + (WIDE ? Shape::RAW : 0) + (pair ? Shape::RAW_BC : 0);
  // two tiles each: (s, s x), the 16-byte chunk j of the 8 channels o at j ^ (o / 2) % 4 for the banks; y; b; c
  float2(*const s_in)[TT][CT] = reinterpret_cast<float2(*)[TT][CT]>(s_tiles);
  float(*const s_y)[TT][CT] = reinterpret_cast<float(*)[TT][CT]>(s_tiles + 2 * TT * CT * 8);
  float(*const s_b)[TT][NP] = reinterpret_cast<float(*)[TT][NP]>(s_tiles + 2 * TT * CT * 12);
  float(*const s_c)[TT][NP] = s_b + 2;
  float* const s_join = reinterpret_cast<float*>(s_tiles);  // [rank][JOIN], in a cluster
  cg::cluster_group cluster = cg::this_cluster();
  const int R = cluster.num_blocks(), rank = cluster.block_rank();
  const int cblocks = (p.d + CT - 1) / CT;
  const int item = blockIdx.x / R;
  // Longest sequences first, in rounds of one CTA to an SM that run to and fro, so that an SM whose
  // first piece of work is long gets a short second one: sequence b has `before` longer ones.
  int place_of = item;
  if (p.lengths && p.batch > 1 && p.batch <= 256) {
    const int items = cblocks * p.batch, round = item / sms, left_over = items - round * sms;
    if (round & 1) place_of = round * sms + min(sms, left_over) - 1 - item % sms;
    for (int i = threadIdx.x; i < p.batch; i += kThreads) {
      const int own = p.lengths[i];
      int before = 0;
      for (int k = 0; k < p.batch; ++k) {
        const int other = p.lengths[k];
        before += other > own || (other == own && k < i);
      }
      if (before == place_of / cblocks) s_seq = i;
    }
  } else if (threadIdx.x == 0) {
    s_seq = item / cblocks;
  }
  const int cb = place_of % cblocks, c0 = cb * CT;
  for (int i = threadIdx.x; i < CT; i += kThreads) {
    s_bias[i] = p.dt_bias && c0 + i < p.d ? p.dt_bias[c0 + i] : 0.f;
    s_skip[i] = p.d_skip && c0 + i < p.d ? p.d_skip[c0 + i] : 0.f;
  }
  __syncthreads();
  const int b = s_seq, len = length_of(p, b);
  // this CTA's piece of the valid frames, whole tiles
  const int piece = ((len + R - 1) / R + TT - 1) / TT * TT;
  const int lo = min(rank * piece, len), hi = min(lo + piece, len);
  const int tiles = (hi - lo + TT - 1) / TT;

  // ---- producers: 8 neighbouring channels of one frame of each tile ----
    const int tid = threadIdx.x % kLanes, o8 = tid % OCT, tt = tid / OCT, left = p.d - c0 - o8 * 8;
    const bool mine = tt < TT && left > 0;
    const int64_t at = c0 + o8 * 8;
    const T* px = (const T*)p.x + b * p.x_batch_stride + at;
    const T* pdt = (const T*)p.dt + b * p.dt_batch_stride + at;
    const T* pz = p.z ? (const T*)p.z + b * p.z_batch_stride + at : nullptr;
    const T* pb = (const T*)p.b + b * p.b_batch_stride;
    const T* pc = (const T*)p.c + b * p.c_batch_stride;
    T* py = (T*)p.y + b * p.y_batch_stride + at;
    auto fetch = [&](auto out_tag, int k) GAM_INLINE {          // tile k on its way
        constexpr bool OUT = decltype(out_tag)::value;
        const int t0 = lo + k * TT, t = t0 + tt;
        if (k < tiles) {
          if constexpr (WIDE) {
            T* raw = s_raw + k % 3 * 3 * kTile + tid * 8;
            const bool on = mine && t < hi;
            copy8(raw, px + (on ? t * p.x_row_stride : 0), on);
            copy8(raw + kTile, pdt + (on ? t * p.dt_row_stride : 0), on);
            if (OUT && pz) copy8(raw + 2 * kTile, pz + (on ? t * p.z_row_stride : 0), on);
          }
          if (pair) {
            T* raw = s_raw_bc + (k & 1) * 2 * TT * NP;
#pragma unroll 4
            for (int e = tid * PER; e < TT * NP; e += kLanes * PER) {
              const int r = t0 + e / NP, i = e % NP;
              const int bytes = r < hi && i < p.n ? min(4, (p.n - i) * (int)sizeof(T)) : 0;  // the rest of the 4 is zero
              copy4(raw + e, bytes ? pb + r * p.b_row_stride + i : pb, bytes);
              if (OUT) copy4(raw + TT * NP + e, bytes ? pc + r * p.c_row_stride + i : pc, bytes);
            }
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      // 8 values of x (0), dt (1) or z (2) of this thread's frame of tile k
      auto octet = [&](int k, int which, const T* g) {
        Octet<T, WIDE> r;
        if constexpr (WIDE) r.load(s_raw + (k % 3 * 3 + which) * kTile + tid * 8, true, 8);
        else r.load(g, mine && lo + k * TT + tt < hi, left);
        return r;
      };
      auto prepare = [&](auto out_tag, int k) GAM_INLINE {      // s, s x, b and c of tile k
        constexpr bool OUT = decltype(out_tag)::value;
        const int t0 = lo + k * TT, t = t0 + tt;
        if (tt < TT) {
          const bool on = mine && t < hi;
          const Octet<T, WIDE> x = octet(k, 0, px + t * p.x_row_stride), dt = octet(k, 1, pdt + t * p.dt_row_stride);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 bias = *reinterpret_cast<const float2*>(&s_bias[o8 * 8 + 2 * j]);
            float2 st = make_float2(dt.get(2 * j) + bias.x, dt.get(2 * j + 1) + bias.y);
            if (p.dt_softplus) st = softplus2(st);
            if (!on) st = make_float2(0.f, 0.f);     // a frame past the end changes nothing: x is 0 there too
            *reinterpret_cast<float4*>(&s_in[k & 1][tt][o8 * 8 + (j ^ (o8 / 2 % 4)) * 2]) =
                make_float4(st.x, st.x * x.get(2 * j), st.y, st.y * x.get(2 * j + 1));
          }
        }
        float* const db = &s_b[k & 1][0][0];
        float* const dc = &s_c[k & 1][0][0];
        if (pair) {
          const T* raw = s_raw_bc + (k & 1) * 2 * TT * NP;
#pragma unroll 4
          for (int e = tid * PER; e < TT * NP; e += kLanes * PER)
#pragma unroll
            for (int i = 0; i < PER; ++i) {
              db[e + i] = to_f(raw[e + i]);
              if (OUT) dc[e + i] = to_f(raw[TT * NP + e + i]);
            }
        } else {
#pragma unroll 4
          for (int e = tid; e < TT * NP; e += kLanes) {
            const int r = t0 + e / NP, i = e % NP;
            const bool use = r < hi && i < p.n;
            uint32_t vb = 0, vc = 0;
            if (use) vb = load_bits(pb + r * p.b_row_stride + i);
            if (OUT && use) vc = load_bits(pc + r * p.c_row_stride + i);
            db[e] = from_bits<T>(vb);
            if (OUT) dc[e] = from_bits<T>(vc);
          }
        }
      };
      auto finish = [&](int k) GAM_INLINE {                     // skip and gate, and out
        const int t = lo + k * TT + tt;
        if (!mine || t >= hi) return;
        const Octet<T, WIDE> x = octet(k, 0, px + t * p.x_row_stride);
        Octet<T, WIDE> z;
        if (pz) z = octet(k, 2, pz + t * p.z_row_stride);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i] = fmaf(s_skip[o8 * 8 + i], x.get(i), s_y[k & 1][tt][o8 * 8 + i]);
          if (sizeof(T) == 2 && pz) o[i] *= swish_f<T>(z.get(i));
        }
        if (sizeof(T) == 4 && pz) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 g = unpack2(swish2(pack2(z.get(2 * i), z.get(2 * i + 1))));
            o[2 * i] *= g.x, o[2 * i + 1] *= g.y;
          }
        }
        T* dst = py + t * p.y_row_stride;
        if constexpr (WIDE) {
          store8(dst, o);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < left) dst[i] = from_f<T>(o[i]);
        }
      };
    auto zeros = [&] {                               // frames behind the end
      if (mine)
        for (int t = len + rank * TT + tt; t < p.t_max; t += R * TT) {
          T* dst = py + t * p.y_row_stride;
          if constexpr (WIDE) {
            store8(dst, {});
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < left) dst[i] = from_f<T>(0.f);
          }
        }
    };
    if (SPLIT && threadIdx.x >= kLanes) {
      // while the lanes run tile k: the y of the one before goes out, the one after is made ready
      auto pass = [&](auto out_tag, bool joined) GAM_INLINE {
        constexpr bool OUT = decltype(out_tag)::value;
        fetch(out_tag, 0);
        fetch(out_tag, 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (joined) __syncthreads();                 // the lanes have read the pieces' end states, whose place the tiles take
        if (tiles > 0) prepare(out_tag, 0);
        __syncthreads();
        for (int k = 0; k < tiles; ++k) {
          if (OUT && k > 0) finish(k - 1);
          fetch(out_tag, k + 2);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          if (k + 1 < tiles) prepare(out_tag, k + 1);
          __syncthreads();
        }
        if (OUT && tiles > 0) finish(tiles - 1);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      };
      if (R == 1 || rank == 0) pass(std::true_type(), false);
      else if (rank < R - 1) pass(std::false_type(), false);
      if (R > 1) {
        cluster.sync();
        cluster.sync();
        if (rank > 0) pass(std::true_type(), true);
      }
      zeros();
      return;
    }

  // ---- lanes: the recurrence ----
  const int part = tid % L, ch = tid / L;
  const int valid = p.n - part * S;                  // of this lane's states
  auto channel = [&](int j) { return min(c0 + ch + j * CT1, p.d - 1); };  // lanes past the last channel walk along
  auto rate = [](float v) { return finite_rate(v * kLog2e); };  // for 2^x
  u64 a[CH][S / 2], h[CH][S / 2];
  int col[CH];                                       // channel j's place in a row of s_in
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const float* pa = p.a + (int64_t)channel(j) * p.n;
    const float* st = rank == 0 && p.state_in ? p.state_in + ((int64_t)b * p.d + channel(j)) * p.n : nullptr;
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
      const int k = part * S + 2 * i;
      a[j][i] = pack2(k < p.n ? rate(pa[k]) : 0.f, k + 1 < p.n ? rate(pa[k + 1]) : 0.f);
      h[j][i] = pack2(st && k < p.n ? st[k] : 0.f, st && k + 1 < p.n ? st[k + 1] : 0.f);
    }
    const int c = ch + j * CT1;
    col[j] = (c / 8 * 4 + ((c % 8 / 2) ^ (c / 16 % 4))) * 2 + c % 2;
  }
  float sum_s[CH] = {};
  // The lanes' work on tile k; OUT: with outputs, else for the end state and the sum of s alone.
  auto run = [&](auto out_tag, int k) GAM_INLINE {
    constexpr bool OUT = decltype(out_tag)::value;
    const int buf = k & 1;
#pragma unroll 1
      for (int t4 = 0; t4 < TT; t4 += 4) {
        float v[CH][4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int t = t4 + f;
          u64 s2[CH], sx2[CH], y2[CH];
#pragma unroll
          for (int j = 0; j < CH; ++j) {
            const float2 in = s_in[buf][t][col[j]];
            s2[j] = both(in.x), sx2[j] = both(in.y);
            if (!OUT) sum_s[j] += in.x;
          }
#pragma unroll
          for (int i = 0; i < S / 4; ++i) {
            const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(&s_b[buf][t][part * S + 4 * i]);
            ulonglong2 cv;
            if (OUT) cv = *reinterpret_cast<const ulonglong2*>(&s_c[buf][t][part * S + 4 * i]);
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int j = 0; j < CH; ++j) {
                u64& hh = h[j][2 * i + q];
                const u64 decay = decay2<T>(s2[j], a[j][2 * i + q]);
                hh = fma2(decay, hh, mul2(sx2[j], q ? bv.y : bv.x));
                if constexpr (PAD) {
                  const float2 v = unpack2(hh);
                  hh = pack2(4 * i + 2 * q < valid ? v.x : 0.f, 4 * i + 2 * q + 1 < valid ? v.y : 0.f);
                }
                if (OUT) y2[j] = i + q ? fma2(q ? cv.y : cv.x, hh, y2[j]) : mul2(cv.x, hh);
              }
          }
          if (OUT)
#pragma unroll
            for (int j = 0; j < CH; ++j) {
              const float2 yy = unpack2(y2[j]);
              v[j][f] = L == 1 || valid > 0 ? yy.x + yy.y : 0.f;
            }
        }
        if constexpr (OUT) {
          // the lanes of a channel add their parts of 4 frames; with L >= 2 each ends with its own share of the frames
#pragma unroll
          for (int j = 0; j < CH; ++j) {
            const int c = ch + j * CT1;
            if constexpr (L == 1) {
#pragma unroll
              for (int f = 0; f < 4; ++f) s_y[buf][t4 + f][c] = v[j][f];
            } else {
              const bool up = part & 1;
              float w[2];
#pragma unroll
              for (int f = 0; f < 2; ++f)
                w[f] = (up ? v[j][f + 2] : v[j][f]) + __shfl_xor_sync(0xffffffffu, up ? v[j][f] : v[j][f + 2], 1);
              if constexpr (L == 2) {
#pragma unroll
                for (int f = 0; f < 2; ++f) s_y[buf][t4 + (up ? 2 : 0) + f][c] = w[f];
              } else {
                const bool up2 = part & 2;
                float q = (up2 ? w[1] : w[0]) + __shfl_xor_sync(0xffffffffu, up2 ? w[0] : w[1], 2);
#pragma unroll
                for (int o = 4; o < L; o <<= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
                if (part < 4) s_y[buf][t4 + (up ? 2 : 0) + (up2 ? 1 : 0)][c] = q;
              }
            }
          }
        }
      }
  };
  // One run over the piece.  Without producers a thread does both: it prepares the next tile before it
  // runs this one, so that one barrier a tile is enough and the warps of a CTA need not go in step.
  auto pass = [&](auto out_tag) GAM_INLINE {
    constexpr bool OUT = decltype(out_tag)::value;
    if constexpr (SPLIT) {
      __syncthreads();                               // the first tile is there
      for (int k = 0; k < tiles; ++k) {
        run(out_tag, k);
        __syncthreads();
      }
    } else {
      fetch(out_tag, 0);
      fetch(out_tag, 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      if (tiles > 0) prepare(out_tag, 0);
      __syncthreads();
      for (int k = 0; k < tiles; ++k) {
        fetch(out_tag, k + 2);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (k + 1 < tiles) prepare(out_tag, k + 1);
        run(out_tag, k);
        __syncthreads();
        if (OUT) finish(k);
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  };

  if (R > 1) {
    if (rank == 0) pass(std::true_type());    // the first piece knows its state
    else if (rank < R - 1) pass(std::false_type());
    cluster.sync();                                  // every CTA of the cluster has started: its shared memory is there
    // to every later piece (stores over the cluster need no answer; loads were ten times slower)
    for (int r = rank + 1; r < R; ++r) {
      float* to = cluster.map_shared_rank(s_join, r) + rank * JOIN;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int c = ch + j * CT1;
#pragma unroll
        for (int i = 0; i < S / 4; ++i)
          *reinterpret_cast<ulonglong2*>(to + c * NP + part * S + 4 * i) = make_ulonglong2(h[j][2 * i], h[j][2 * i + 1]);
        if (part == 0) to[CT * NP + c] = sum_s[j];
      }
    }
    cluster.sync();
    if (rank > 0) {
      // a piece without frames changes nothing, not even by a decay of 0 times an infinite or NaN rate
      for (int r = 0; r < rank && (r == 0 || r * piece < len); ++r) {
        const float* e = s_join + r * JOIN;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const int c = ch + j * CT1;
          const float q = e[CT * NP + c];
#pragma unroll
          for (int i = 0; i < S / 4; ++i) {
            const ulonglong2 end = *reinterpret_cast<const ulonglong2*>(e + c * NP + part * S + 4 * i);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              u64& hh = h[j][2 * i + k];
              // the first piece's end state is whole already
              hh = r ? fma2(both(1.f), carry2<T>(hh, q, a[j][2 * i + k]), k ? end.y : end.x) : (k ? end.y : end.x);
            }
          }
        }
      }
      __syncthreads();                               // the producers may put the first tile there now
      pass(std::true_type());
    }
  } else {
    pass(std::true_type());
  }

  if (!SPLIT) zeros();
  if (rank == R - 1 && p.state_out) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = c0 + ch + j * CT1;
      if (c >= p.d) continue;
      float* st = p.state_out + ((int64_t)b * p.d + c) * p.n;
#pragma unroll
      for (int i = 0; i < S / 2; ++i) {
        const int k = part * S + 2 * i;
        const float2 v = unpack2(h[j][i]);
        if (k < p.n) st[k] = v.x;
        if (k + 1 < p.n) st[k + 1] = v.y;
      }
    }
  }
}

// A few frames: L lanes of 4 states to a channel, neighbouring lanes on neighbouring memory;
// a thread has two channels on their way at a time, kStep / L apart.  CTAs of 128 threads even out the SMs' loads
// better than of 256 (one frame of 64 streams, 2048 channels of 16 states in bf16: 5.5 us, 5.7 with 256).
constexpr int kStep = 128;
template <typename T, int L, bool VEC, bool QUAD>
__global__ void __launch_bounds__(kStep) step_kernel(const gam_scan_args p) {
  constexpr int CT = kStep / L, CH = 2;
  const int cblocks = (p.d + CT * CH - 1) / (CT * CH);
  const int cb = blockIdx.x % cblocks, b = blockIdx.x / cblocks;
  const int part = threadIdx.x % L, c0 = cb * CT * CH + threadIdx.x / L;
  const int k0 = part * 4;
  const int len = length_of(p, b);
  // the channels whose outputs a lane finishes: of L lanes the even ones take the first, the odd ones the second
  constexpr int OWN = L > 1 ? 1 : CH;
  const bool up = part & 1;
  float a[CH][4], h[CH][4], bias[CH], skip[OWN];
  int ch[CH], own[OWN];
  bool live[OWN];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    ch[j] = min(c0 + j * CT, p.d - 1);               // lanes past the last channel walk along, for the shuffles
    const float* pa = p.a + (int64_t)ch[j] * p.n + k0;
    const float* ph = p.state_in ? p.state_in + ((int64_t)b * p.d + ch[j]) * p.n + k0 : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[j][i] = h[j][i] = 0.f;
    if constexpr (VEC) {                             // n a multiple of 4, 16-byte aligned
      if (k0 < p.n) {
        if (ph) {
          const float4 w = *reinterpret_cast<const float4*>(ph);
          h[j][0] = w.x, h[j][1] = w.y, h[j][2] = w.z, h[j][3] = w.w;
        }
        const float4 q = __ldg(reinterpret_cast<const float4*>(pa));
        a[j][0] = q.x, a[j][1] = q.y, a[j][2] = q.z, a[j][3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k0 + i < p.n) {
          if (ph) h[j][i] = ph[i];
          a[j][i] = __ldg(pa + i);
        }
    }
    bias[j] = p.dt_bias ? __ldg(p.dt_bias + ch[j]) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < OWN; ++j) {
    own[j] = L > 1 && up ? ch[CH - 1] : ch[j];
    live[j] = part < 2 && c0 + (L > 1 ? part : j) * CT < p.d;
    skip[j] = p.d_skip ? __ldg(p.d_skip + own[j]) : 0.f;
  }
  const T* px = (const T*)p.x + b * p.x_batch_stride;
  const T* pdt = (const T*)p.dt + b * p.dt_batch_stride;
  const T* pz = p.z ? (const T*)p.z + b * p.z_batch_stride : nullptr;
  const T* pb = (const T*)p.b + b * p.b_batch_stride + k0;
  const T* pc = (const T*)p.c + b * p.c_batch_stride + k0;
  T* y = (T*)p.y + b * p.y_batch_stride;
  for (int t = 0; t < len; ++t) {
    uint32_t ux[CH], ud[CH], uz[OWN], ub[4], uc[4];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      ud[j] = load_bits(pdt + t * p.dt_row_stride + ch[j]);
      ux[j] = load_bits(px + t * p.x_row_stride + ch[j]);
    }
#pragma unroll
    for (int j = 0; j < OWN; ++j) uz[j] = pz ? load_bits(pz + t * p.z_row_stride + own[j]) : 0;
    float bv[4] = {}, cv[4] = {};
    if constexpr (QUAD) {                            // rows of b and c in whole quads, n a multiple of 4
      if (k0 < p.n) {
        const Vec<T, 4> q = *reinterpret_cast<const Vec<T, 4>*>(pb + t * p.b_row_stride);
        const Vec<T, 4> r = *reinterpret_cast<const Vec<T, 4>*>(pc + t * p.c_row_stride);
#pragma unroll
        for (int i = 0; i < 4; ++i) bv[i] = to_f(q.v[i]), cv[i] = to_f(r.v[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ub[i] = uc[i] = 0;
        if (k0 + i < p.n) {
          ub[i] = load_bits(pb + t * p.b_row_stride + i);
          uc[i] = load_bits(pc + t * p.c_row_stride + i);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) bv[i] = from_bits<T>(ub[i]), cv[i] = from_bits<T>(uc[i]);
    }
    float2 s = make_float2(from_bits<T>(ud[0]) + bias[0], from_bits<T>(ud[1]) + bias[1]);
    if (p.dt_softplus) s = softplus2(s);
    float v[CH], xv[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      xv[j] = from_bits<T>(ux[j]);
      const float st = j ? s.y : s.x, sx = st * xv[j], e = st * kLog2e;
      v[j] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        // the rates are bounded here, not where they are loaded: the loads of the frame would wait for them (+0.5 us)
        const float2 decay = unpack2(decay2<T>(both(e), pack2(finite_rate(a[j][i]), finite_rate(a[j][i + 1]))));
        h[j][i] = fmaf(decay.x, h[j][i], sx * bv[i]);
        h[j][i + 1] = fmaf(decay.y, h[j][i + 1], sx * bv[i + 1]);
        if constexpr (!VEC) {                          // states past n stay 0 whatever s x is
          if (k0 + i >= p.n) h[j][i] = 0.f;
          if (k0 + i + 1 >= p.n) h[j][i + 1] = 0.f;
        }
        v[j] = fmaf(cv[i], h[j][i], v[j]);
        v[j] = fmaf(cv[i + 1], h[j][i + 1], v[j]);
      }
      if (VEC && k0 >= p.n) v[j] = 0.f;
    }
    if constexpr (L > 1) {
      v[0] = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 1);
#pragma unroll
      for (int o = 2; o < L; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
      xv[0] = up ? xv[1] : xv[0];
    }
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
      float q = fmaf(skip[j], xv[j], v[j]);
      if (pz) q *= swish_f<T>(from_bits<T>(uz[j]));
      if (live[j]) y[t * p.y_row_stride + own[j]] = from_f<T>(q);
    }
  }
#pragma unroll
  for (int j = 0; j < OWN; ++j)
    if (live[j])
      for (int t = len; t < p.t_max; ++t) y[t * p.y_row_stride + own[j]] = from_f<T>(0.f);
  if (!p.state_out) return;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    if (c0 + j * CT >= p.d) continue;
    float* ph = p.state_out + ((int64_t)b * p.d + ch[j]) * p.n + k0;
    if constexpr (VEC) {
      if (k0 < p.n) *reinterpret_cast<float4*>(ph) = make_float4(h[j][0], h[j][1], h[j][2], h[j][3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k0 + i < p.n) ph[i] = h[j][i];
    }
  }
}

template <typename T, int L>
gam_status launch_step(const gam_scan_args& p, cudaStream_t s) {
  const int64_t grid = (int64_t)((p.d + 2 * kStep / L - 1) / (2 * kStep / L)) * p.batch;
  if (grid > INT32_MAX) return op_fail(GAM_ERR_CAPACITY, "batch * d too large for one call");
  const unsigned g = (unsigned)grid;
  const bool vec = p.n % 4 == 0 && aligned(p.a, 16) && aligned(p.state_in, 16) && aligned(p.state_out, 16);
  constexpr size_t kQuad = 4 * sizeof(T);
  const bool quad = p.n % 4 == 0 && aligned(p.b, kQuad) && aligned(p.c, kQuad) && p.b_batch_stride % 4 == 0 &&
                    p.b_row_stride % 4 == 0 && p.c_batch_stride % 4 == 0 && p.c_row_stride % 4 == 0;
  auto kernel = vec && quad ? step_kernel<T, L, true, true> : vec ? step_kernel<T, L, true, false> : step_kernel<T, L, false, false>;
  return launch_status(launch_kernel(kernel, g, kStep, 0, s, p));
}

template <typename T, int S, int L, int CH>
gam_status launch_scan(const gam_scan_args& p, int sms, cudaStream_t s) {
  using Shape = ScanShape<T, S, L, CH>;
  constexpr int CT = Shape::CT, TT = Shape::TT;
  const int64_t ctas = (int64_t)((p.d + CT - 1) / CT) * p.batch;
  constexpr int V = 16 / sizeof(T);
  const bool wide = p.d % 8 == 0 && aligned(p.x, 16) && aligned(p.dt, 16) && aligned(p.z, 16) && aligned(p.y, 16) &&
                    p.x_batch_stride % V == 0 && p.x_row_stride % V == 0 && p.dt_batch_stride % V == 0 &&
                    p.dt_row_stride % V == 0 && p.z_batch_stride % V == 0 && p.z_row_stride % V == 0 &&
                    p.y_batch_stride % V == 0 && p.y_row_stride % V == 0;
  constexpr int PER = 4 / sizeof(T);
  const bool pair = aligned(p.b, 4) && aligned(p.c, 4) && p.b_batch_stride % PER == 0 && p.b_row_stride % PER == 0 &&
                    p.c_batch_stride % PER == 0 && p.c_row_stride % PER == 0;
  // Less than a CTA to an SM: split the time axis while the pieces keep two tiles and all CTAs are on the SMs at
  // once (6 to an SM, or what shared memory allows).  Pieces below 3 gain nothing over the twice as long work:
  // 1 x 749 frames of 1536 channels 33 us with 4, 29 us with 8; 3 x 517 of 1001 (189 CTAs) 48 us with 4, 38 with 1.
  int R = 1;
  if (CH == 1 && ctas <= sms)
    while (R < 8 && p.t_max >= R * 2 * 2 * TT &&
           ctas * R * 2 <= sms * std::min<int64_t>(6, 227 * 1024 / (Shape::bytes(wide, pair, R * 2) + CT * 8 + 1088)))
      R *= 2;
  if (R == 2) R = 1;
  if (ctas * R > INT32_MAX) return op_fail(GAM_ERR_CAPACITY, "batch * d too large for one call");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas * R));
  cfg.blockDim = dim3(Shape::THREADS);
  cfg.stream = s;
  cfg.dynamicSmemBytes = Shape::bytes(wide, pair, R);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = R;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = R > 1 ? 1 : 0;
  const bool pad = p.n % S != 0;
  auto kernel = wide ? (pad ? scan_kernel<T, S, L, CH, true, true> : scan_kernel<T, S, L, CH, true, false>)
                     : (pad ? scan_kernel<T, S, L, CH, false, true> : scan_kernel<T, S, L, CH, false, false>);
  if (cfg.dynamicSmemBytes + CT * 8 + 64 > 48 * 1024) {  // with the static part
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return launch_status(e);
  }
  return launch_status(cudaLaunchKernelEx(&cfg, kernel, p, sms, pair));
}

// Lanes with two channels of S states where that still gives every SM work, else
// lanes with one channel of S1 states, and a cluster over the time axis.
template <typename T, int S, int L, int S1, int L1>
gam_status launch_pair(const gam_scan_args& p, int sms, cudaStream_t s) {
  constexpr int CT = kLanes / L * 2;
  const int64_t ctas = (int64_t)((p.d + CT - 1) / CT) * p.batch;
  return ctas >= 4 * sms ? launch_scan<T, S, L, 2>(p, sms, s) : launch_scan<T, S1, L1, 1>(p, sms, s);
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
  if (p.n <= 4) return launch_scan<T, 4, 1, 1>(p, sms, s);
  if (p.n <= 8) return launch_pair<T, 8, 1, 4, 2>(p, sms, s);
  if (p.n <= 16) return launch_pair<T, 8, 2, 4, 4>(p, sms, s);
  if (p.n <= 32) return launch_pair<T, 8, 4, 4, 8>(p, sms, s);
  return launch_pair<T, 8, 8, 8, 8>(p, sms, s);
}

#undef GAM_INLINE

}  // namespace
}  // namespace ops
}  // namespace gam
