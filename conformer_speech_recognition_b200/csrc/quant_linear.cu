// Few-row linear layer on INT4-g64 weights: gam_quant_linear.
//
//   y[m, o] = act(bias[o] + sum_g scale[o, g] sum_{j in g} q[o, j] x[m, j])
//
// The floor is the weight stream (0.53 bytes per weight).  A warp owns 16 outputs:
// mma.m16n8k16 with the weights as the 16-row operand, dequantised in registers, and
// rows of x as 8-column tiles.  The integers are exact in both 16-bit types, so a
// group's sum is that of q x itself and is scaled in fp32 by the group's scale.
// Weights are read and dequantised once for every 8 rows (one tile of x) or 16 (two):
// once for up to 16 rows, four times for 64, and in fp32 once for every 8 rows above 16.
// (tcgen05 would take 128 outputs and all rows at once, with an accumulator of its own
// for every group's scale; not built.)
//
// What it measured: one row of 768 x 768 in 2.4 us (launch and one trip to memory); 16384 x 4096
// (36 MB of weights, 5.4 us at the copy rate): one row in 13.6 us, 16 in 19.6, 32 in 36, 64 in 62; in
// fp32 16 in 40, 32 in 128, 64 in 252.  No pipe bounds them (16 rows: 1.7 of 4 instructions a clock, ALU 38 %): it
// is the latency at 16 warps to an SM, as many as their registers allow, and the uneven last
// round of CTAs (512 at two to an SM; up to 8 rows 256, of which 108 SMs hold two and 40 one).
//
// Integers become floats through the mantissa of 1024 (fp16) or 128 (bf16), a published
// method.  The words' nibble order gives adjacent pairs by one shift and mask, and a lane's 16
// weights of a group are 16 consecutive k, so its fragments of x are 16 consecutive
// values of a row.  K is split over the warps of a CTA, and over a cluster of CTAs when
// there are few tiles; partial sums are added in a fixed order.
//
// fp32 x is held as three bf16 parts (8 + 8 + 8 bits: exact), each with its own MMA, whose
// fp32 sums within a group may truncate (2 u an addition; 1025 outputs of 1024 in all 2.8e-7
// off, an fp32 sum 1.8e-7).
#include <cooperative_groups.h>

#include <algorithm>

#include "stream_ops.cuh"

namespace gam {
namespace ops {
namespace {

namespace cg = cooperative_groups;

template <typename T>
struct Elem {                  // how x enters the MMA: type and number of parts
  using M = T;
  static constexpr int parts = 1;
};
template <>
struct Elem<float> {
  using M = bf16;
  static constexpr int parts = 3;
};

// c <- a b + (FIRST ? 0 : c)
#define GAM_MMA(T)                                                                                                    \
  if constexpr (FIRST)                                                                                                \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." T "." T ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "       \
                 "{%10,%10,%10,%10};"                                                                                 \
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])                                                     \
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));                           \
  else                                                                                                                \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." T "." T ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "       \
                 "{%0,%1,%2,%3};"                                                                                     \
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                                                     \
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1))
template <bool FIRST>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  GAM_MMA("f16");
}
template <bool FIRST>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bf16) {
  GAM_MMA("bf16");
}
#undef GAM_MMA

// (a & mask) | magic in one instruction: both constants stay in registers.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(magic));
  return r;
}
__device__ __forceinline__ uint32_t fma_pair(uint32_t a, uint32_t b, uint32_t c, __half) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t fma_pair(uint32_t a, uint32_t b, uint32_t c, bf16) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// The constants of unpack8 (made once: an instruction takes one as an immediate at most).
template <typename M>
struct UnpackConst;
template <>
struct UnpackConst<__half> {
  uint32_t lo, hi, magic, one, minus1032, sixteenth, minus72;
  __device__ __forceinline__ UnpackConst()
      : lo(0x000F000Fu), hi(0x00F000F0u), magic(0x64006400u), one(0x3C003C00u), minus1032(0xE408E408u),
        sixteenth(0x2C002C00u), minus72(0xD480D480u) {
    asm volatile("" : "+r"(lo), "+r"(hi), "+r"(magic));
  }
};
template <>
struct UnpackConst<bf16> {
  uint32_t lo, magic, scale, shift;  // 2^-9 and -136 * 2^-9
  __device__ __forceinline__ UnpackConst() : lo(0x000F000Fu), magic(0x43004300u), scale(0x3B003B00u), shift(0xBE88BE88u) {
    asm volatile("" : "+r"(lo), "+r"(magic));
  }
};
// The 8 weights of a word as four pairs.  fp16: 1024 + u and, from the nibbles left
// in place 4 bits up, 1024 + 16 u are exact, and so is the fused subtraction.
// bf16: 128 + u is exact; the pairs are 2^-9 q there, so that a group's sum of the
// largest finite x stays finite (64 * 7 < 2^9), and the last step takes 2^9 back.
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&p)[4], const UnpackConst<__half>& k) {
  const uint32_t w8 = w >> 8;
  p[0] = fma_pair(and_or(w, k.lo, k.magic), k.one, k.minus1032, __half());
  p[1] = fma_pair(and_or(w, k.hi, k.magic), k.sixteenth, k.minus72, __half());
  p[2] = fma_pair(and_or(w8, k.lo, k.magic), k.one, k.minus1032, __half());
  p[3] = fma_pair(and_or(w8, k.hi, k.magic), k.sixteenth, k.minus72, __half());
}
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&p)[4], const UnpackConst<bf16>& k) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = fma_pair(and_or(w >> (4 * i), k.lo, k.magic), k.scale, k.shift, bf16());
}
template <typename M>
constexpr float kUnpackScale = 1.f;
template <>
constexpr float kUnpackScale<bf16> = 512.f;

// x as parts of type M.  An infinity or NaN is its first part alone, since its
// difference from itself is NaN.
__device__ __forceinline__ void split(float v, bf16 (&p)[3]) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7F800000u) == 0x7F800000u) {
    p[0] = __float2bfloat16_rn(v);
    p[1] = p[2] = __float2bfloat16_rn(0.f);
    return;
  }
  const float a = __uint_as_float(u & 0xFFFF0000u), r = v - a;           // exact: the low 16 bits
  const float b = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
  p[0] = __float2bfloat16_rn(a);
  p[1] = __float2bfloat16_rn(b);
  p[2] = __float2bfloat16_rn(r - b);
}

struct LinearArgs {
  const void* x;
  const uint8_t* packed;
  const __half* scale;
  const float* bias;
  void* y;
  int64_t ldx, ldy;
  int act, rows, n, groups;   // groups = k / 64
  int wide;                   // x rows are 16-byte aligned
  int kw, per;                // staged form: warps that share a tile's K, groups of a stage
  int chunk;                  // shared and staged forms: groups of x held at a time
};

// ---- few rows or few weights ----
// One or two 8-column tiles of x make few enough fragments that a warp reads them where they lie (L2 holds
// x), so nothing is staged: a CTA of 8 warps takes NT tiles of 16 outputs and 8 MT rows, its warps every 8th
// group of K, each with the weights and x of its next groups on their way.  The call's time is then one trip
// to memory for a short K, and several CTAs to an SM keep the weight stream going for a long one.
constexpr int kThinWarps = 8;

template <typename T, int MT, int NT>
struct ThinGroup {               // a lane's part of a group, as it lies in memory
  uint2 w[NT][2];                // 16 weights of rows g and g + 8 of each tile
  uint32_t s[NT][2];             // their scales' bits
  uint32_t x[MT][16 * sizeof(T) / 4];
};

template <typename T, int MT, int NT>
__global__ void __launch_bounds__(kThinWarps * 32, NT > 1 ? 2 : 3) quant_linear_thin_kernel(const LinearArgs p) {
  using M = typename Elem<T>::M;
  constexpr int PARTS = Elem<T>::parts, U = MT == 1 && NT == 1 && PARTS == 1 ? 2 : 1;
  __shared__ float part[kThinWarps][8 * MT][NT * 16];
  extern __shared__ float join[];                        // [rank - 1][rows][NT 16], in a cluster
  cg::cluster_group cluster = cg::this_cluster();
  const int R = cluster.num_blocks(), rank = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int o0 = (blockIdx.x / R) * NT * 16, m0 = blockIdx.y * 8 * MT, rows = min(8 * MT, p.rows - m0);
  const int k_lo = p.groups * rank / R, k_hi = p.groups * (rank + 1) / R;
  const UnpackConst<M> consts;
  // bases of this lane's rows (past the last: another one, dropped below)
  const int64_t row_bytes = (int64_t)p.groups * 32;
  const uint8_t* w[NT][2];
  const __half* sc[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t o = min(o0 + i * 16 + h * 8 + g, p.n - 1);
      w[i][h] = p.packed + o * row_bytes + t * 8;
      sc[i][h] = p.scale + o * p.groups;
    }
  const T* x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) x[m] = (const T*)p.x + (m0 + (m * 8 + g < rows ? m * 8 + g : 0)) * p.ldx + t * 16;
  auto fetch = [&](ThinGroup<T, MT, NT>& q, int k) {
    k = min(k, k_hi - 1);                                // beyond the end the last group again, not used
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        q.w[i][h] = __ldg(reinterpret_cast<const uint2*>(w[i][h] + (int64_t)k * 32));
        q.s[i][h] = *reinterpret_cast<const unsigned short*>(sc[i][h] + k);
      }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const T* from = x[m] + (int64_t)k * 64;
      if (p.wide) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) {
          const uint4 v = reinterpret_cast<const uint4*>(from)[i];
          q.x[m][4 * i] = v.x, q.x[m][4 * i + 1] = v.y, q.x[m][4 * i + 2] = v.z, q.x[m][4 * i + 3] = v.w;
        }
      } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 16; ++i) q.x[m][i] = reinterpret_cast<const uint32_t*>(from)[i];
      } else {
        const unsigned short* u = reinterpret_cast<const unsigned short*>(from);
#pragma unroll
        for (int i = 0; i < 8; ++i) q.x[m][i] = u[2 * i] | (uint32_t)u[2 * i + 1] << 16;
      }
    }
  };
  float acc[NT][MT][4] = {};
  auto use = [&](const ThinGroup<T, MT, NT>& q) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t a[4][4];                                    // the group's four 16 x 16 pieces
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pa[4], pb[4];
        unpack8(h ? q.w[n][0].y : q.w[n][0].x, pa, consts);
        unpack8(h ? q.w[n][1].y : q.w[n][1].x, pb, consts);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          a[2 * h + i][0] = pa[2 * i], a[2 * h + i][1] = pb[2 * i], a[2 * h + i][2] = pa[2 * i + 1], a[2 * h + i][3] = pb[2 * i + 1];
    }
      const float fa = __half2float(__ushort_as_half((unsigned short)q.s[n][0]));
      const float fb = __half2float(__ushort_as_half((unsigned short)q.s[n][1]));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b[PARTS][2];                            // pairs of consecutive values in each part
          if constexpr (PARTS == 1) {
            b[0][0] = q.x[m][2 * i], b[0][1] = q.x[m][2 * i + 1];
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              bf16 lo[3], hi[3];
              split(__uint_as_float(q.x[m][4 * i + 2 * j]), lo);
              split(__uint_as_float(q.x[m][4 * i + 2 * j + 1]), hi);
#pragma unroll
              for (int h = 0; h < 3; ++h) {
                const __nv_bfloat162 v(lo[h], hi[h]);
                b[h][j] = *reinterpret_cast<const uint32_t*>(&v);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < PARTS; ++e) {
            if (i == 0 && e == 0) mma16816<true>(c, a[i], b[e][0], b[e][1], M());
            else mma16816<false>(c, a[i], b[e][0], b[e][1], M());
          }
        }
        acc[n][m][0] = fmaf(fa, c[0], acc[n][m][0]);
        acc[n][m][1] = fmaf(fa, c[1], acc[n][m][1]);
        acc[n][m][2] = fmaf(fb, c[2], acc[n][m][2]);
        acc[n][m][3] = fmaf(fb, c[3], acc[n][m][3]);
    }
    }
  };
  ThinGroup<T, MT, NT> now[U];
  int k = k_lo + warp;
  if (k < k_hi) {
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(now[u], k + u * kThinWarps);
  }
  while (k < k_hi) {
    ThinGroup<T, MT, NT> next[U];
    if (k + U * kThinWarps < k_hi) {
#pragma unroll
      for (int u = 0; u < U; ++u) fetch(next[u], k + (U + u) * kThinWarps);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k + u * kThinWarps < k_hi) use(now[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = next[u];
    k += U * kThinWarps;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[warp][m * 8 + 2 * t + (e & 1)][n * 16 + g + (e >> 1) * 8] = acc[n][m][e];
  __syncthreads();
  const int outs = rows * NT * 16;
  auto sum = [&](int i) {                                // over the warps, in order
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kThinWarps; ++q) v += (&part[q][0][0])[i];
    return v;
  };
  if (R > 1) {
    // to the first CTA, which adds the pieces of K in order
    cluster.sync();
    if (rank > 0) {
      float* to = cluster.map_shared_rank(join, 0) + (rank - 1) * outs;
      for (int i = threadIdx.x; i < outs; i += kThinWarps * 32) to[i] = sum(i);
    }
    cluster.sync();
    if (rank > 0) return;
  }
  for (int i = threadIdx.x; i < outs; i += kThinWarps * 32) {
    const int m = m0 + i / (NT * 16), o = o0 + i % (NT * 16);
    if (o >= p.n) continue;
    float v = sum(i);
    for (int q = 1; q < R; ++q) v += join[(q - 1) * outs + i];
    v *= kUnpackScale<M>;
    if (p.bias) v += p.bias[o];
    ((T*)p.y)[m * p.ldy + o] = from_f<T>(p.act == GAM_ACT_SWISH ? swish_f<T>(v) : v);
  }
}

template <typename T, int MT, int NT>
gam_status launch_thin(const LinearArgs& p, int sms, cudaStream_t s) {
  const int tiles = (p.n + NT * 16 - 1) / (NT * 16), blocks = (p.rows + 8 * MT - 1) / (8 * MT);
  // few tiles and a long K: K over a cluster of R CTAs too, while each warp keeps 2 groups
  int R = 1;
  while (R < 8 && tiles * blocks * R * 2 <= sms * 2 && p.groups >= R * 2 * kThinWarps * 2) R *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * R, blocks);
  cfg.blockDim = dim3(kThinWarps * 32);
  cfg.dynamicSmemBytes = (R - 1) * std::min(p.rows, 8 * MT) * NT * 16 * sizeof(float);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = R;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = R > 1 ? 1 : 0;
  return launch_status(cudaLaunchKernelEx(&cfg, quant_linear_thin_kernel<T, MT, NT>, p));
}

// ---- many weights, up to 8 rows, 16-bit ----
// A warp's loads of 8 rows touch 8 lines each, and that, not the bytes, was what the form above took its time
// for with many weights: the L1 moved lines 69 % of the time, for scales, weights and x.  Here loads from memory
// take whole 128-byte lines: a CTA of 8 warps takes 256 outputs, a warp 32 of them; weights reach it 4 groups
// (a run: 32 rows x 128 bytes) at a time by cp.async, the next run while it works on one, one scale load serves
// a run (lane t holds group t's, and hands it on by a shuffle), and x lies in shared memory for all warps.
// K is split over a cluster, whose CTAs exchange their sums.  1 x 16384 x 4096: 21 us above, 14 here
// (2.6 TB/s); three runs under way leave less room for x and took 16.5.
//
// The 32-byte slot of group G of row r is G ^ (r & 3) in a run, and rows of x lie 16 bytes beyond their length:
// fragment reads are free of bank conflicts.
constexpr int kMaxSmem = 227 * 1024;
constexpr int kSharedWarps = 8, kRunBytes = 32 * 128, kRuns = 2;
constexpr int kSharedSmem = 112 * 1024;  // two CTAs to an SM

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint2 lds8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kSharedWarps * 32, 2) quant_linear_shared_kernel(const LinearArgs p) {
  constexpr int NT = 2, kThreads = kSharedWarps * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int R = cluster.num_blocks(), rank = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int o0 = (blockIdx.x / R * kSharedWarps + warp) * NT * 16;
  const bool live = o0 < p.n;
  const int runs = (p.groups + 3) / 4;
  const int k_lo = (int)((int64_t)runs * rank / R) * 4, k_hi = min((int)((int64_t)runs * (rank + 1) / R) * 4, p.groups);
  const int64_t row_bytes = (int64_t)p.groups * 32;
  uint8_t* const xs = smem + kSharedWarps * kRuns * kRunBytes;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kRuns * kRunBytes;
  // a lane copies 16 bytes of rows 4 j + lane / 8
  const int cr = lane >> 3, cc = lane & 7;
  const uint32_t copy_to = ring + cr * 128 + ((((cc >> 1) ^ cr) << 1) | (cc & 1)) * 16;
  const uint32_t frag = ring + g * 128 + t * 8;
  // rows of x behind the last: row 0, dropped below
  const int xrow = p.chunk * 128 + 16;
  const uint32_t xf = (uint32_t)__cvta_generic_to_shared(xs) + (g < p.rows ? g : 0) * xrow + t * 32;
  const __half* sc[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) sc[i][h] = p.scale + (int64_t)min(o0 + i * 16 + h * 8 + g, p.n - 1) * p.groups + t;
  // rows past n are not copied: what lies there reaches only outputs that are dropped
  const uint8_t* src = p.packed + (o0 + cr) * row_bytes + (int64_t)k_lo * 32 + cc * 16;
  const UnpackConst<T> consts;

  uint32_t scales[kRuns - 1][NT][2] = {};                // of the runs on their way
  auto issue = [&](int k, int slot, uint32_t (&to)[NT][2]) {  // the run of group k
    if (live && k < k_hi) {
      const int ng = min(4, k_hi - k);
      const uint8_t* from = src;
      if ((cc >> 1) < ng) {
        if (o0 + NT * 16 <= p.n) {
#pragma unroll
          for (int j = 0; j < 8; ++j, from += 4 * row_bytes) cp_async16(copy_to + slot * kRunBytes + j * 512, from);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j, from += 4 * row_bytes)
            if (o0 + j * 4 + cr < p.n) cp_async16(copy_to + slot * kRunBytes + j * 512, from);
        }
      }
      src += 128;
      if (t < ng)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) to[i][h] = *reinterpret_cast<const unsigned short*>(sc[i][h] + k);
    }
    cp_commit();
  };
  u64 acc[NT][2] = {};                                   // pairs: outputs g (and g + 8) of rows 2 t and 2 t + 1
  auto group = [&](int G, uint32_t at_w, uint32_t at_x, const uint32_t (&s)[NT][2]) {
    const uint4 xv[2] = {lds16(xf + at_x), lds16(xf + at_x + 16)};
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint2 wa = lds8(at_w + i * 2048), wb = lds8(at_w + i * 2048 + 1024);
      float c[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pa[4], pb[4];
        unpack8(h ? wa.y : wa.x, pa, consts);
        unpack8(h ? wb.y : wb.x, pb, consts);
        const uint32_t a0[4] = {pa[0], pb[0], pa[1], pb[1]}, a1[4] = {pa[2], pb[2], pa[3], pb[3]};
        if (h == 0) mma16816<true>(c, a0, xv[h].x, xv[h].y, T());
        else mma16816<false>(c, a0, xv[h].x, xv[h].y, T());
        mma16816<false>(c, a1, xv[h].z, xv[h].w, T());
      }
      const uint32_t sa = __shfl_sync(0xffffffffu, s[i][0], (lane & 28) | G), sb = __shfl_sync(0xffffffffu, s[i][1], (lane & 28) | G);
      const float fa = __half2float(__ushort_as_half((unsigned short)sa)), fb = __half2float(__ushort_as_half((unsigned short)sb));
      acc[i][0] = fma2(both(fa), pack2(c[0], c[1]), acc[i][0]);
      acc[i][1] = fma2(both(fb), pack2(c[2], c[3]), acc[i][1]);
    }
  };

#pragma unroll
  for (int u = 0; u < kRuns - 1; ++u) issue(k_lo + 4 * u, u, scales[u]);
  int slot = 0;
  for (int c0 = k_lo; c0 < k_hi; c0 += p.chunk) {
    const int held = min(p.chunk, k_hi - c0), pieces = held * 8;
    if (c0 > k_lo) __syncthreads();                      // the chunk before is read
    const int per_row = p.rows == 1 ? kThreads : 32;      // threads of a row
    for (int r = threadIdx.x / per_row; r < p.rows; r += kThreads / per_row) {
      const T* from = (const T*)p.x + r * p.ldx + (int64_t)c0 * 64;
      uint8_t* to = xs + r * xrow;
      for (int c = threadIdx.x % per_row; c < pieces; c += per_row) {
        if (p.wide) {
          cp_async16((uint32_t)__cvta_generic_to_shared(to + c * 16), from + c * 8);
        } else {
          Vec<T, 8> v;
#pragma unroll
          for (int i = 0; i < 8; ++i) v.v[i] = from[c * 8 + i];
          *reinterpret_cast<Vec<T, 8>*>(to + c * 16) = v;
        }
      }
    }
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    for (int k = c0; k < c0 + held; k += 4) {
      uint32_t s[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s[i][h] = scales[0][i][h];
#pragma unroll
          for (int u = 0; u + 2 < kRuns; ++u) scales[u][i][h] = scales[u + 1][i][h];
        }
      // the new run's slot was read before the last __syncwarp
      issue(k + 4 * (kRuns - 1), slot == 0 ? kRuns - 1 : slot - 1, scales[kRuns - 2]);
      cp_wait<kRuns - 1>();
      __syncwarp();                                      // every lane's copies of this run are in
      const int ng = live ? min(4, k_hi - k) : 0;
      const uint32_t at = frag + slot * kRunBytes, at_x = (k - c0) * 128;
      if (ng == 4) {
#pragma unroll
        for (int G = 0; G < 4; ++G) group(G, at + (G ^ (g & 3)) * 32, at_x + G * 128, s);
      } else {
#pragma unroll 1
        for (int G = 0; G < ng; ++G) group(G, at + (G ^ (g & 3)) * 32, at_x + G * 128, s);
      }
      __syncwarp();
      slot = slot + 1 == kRuns ? 0 : slot + 1;
    }
  }
  cp_wait<0>();
  if (R > 1) {
    // warp w's sums are added up by CTA w % R of the cluster: [w / R][rank][sum][lane] over the idle ring
    u64* const join = reinterpret_cast<u64*>(smem);
    constexpr int SUMS = NT * 2;
    cluster.sync();
    u64* to = cluster.map_shared_rank(join, warp % R) + ((warp / R) * R + rank) * SUMS * 32 + lane;
#pragma unroll
    for (int i = 0; i < SUMS; ++i) to[i * 32] = (&acc[0][0])[i];
    cluster.sync();
    if (warp % R != rank) return;
#pragma unroll
    for (int i = 0; i < SUMS; ++i) {
      u64 v = 0;
      for (int q = 0; q < R; ++q) v = fma2(both(1.f), join[((warp / R) * R + q) * SUMS * 32 + i * 32 + lane], v);
      (&acc[0][0])[i] = v;
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int o = o0 + i * 16 + h * 8 + g;
      if (o >= p.n) continue;
      const float bias = p.bias ? p.bias[o] : 0.f;
      const float2 sums = unpack2(acc[i][h]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * t + e;
        const float v = (e ? sums.y : sums.x) * kUnpackScale<T> + bias;
        if (r < p.rows) ((T*)p.y)[r * p.ldy + o] = from_f<T>(p.act == GAM_ACT_SWISH ? swish_f<T>(v) : v);
      }
    }
}

template <typename T>
gam_status launch_shared(LinearArgs p, int sms, cudaStream_t s) {
  // K over a cluster of R CTAs while two CTAs to an SM hold them all at once and each has two runs
  const int ctas = (p.n + kSharedWarps * 32 - 1) / (kSharedWarps * 32);
  int R = 1;
  while (R < 8 && ctas * R <= sms && p.groups >= R * 2 * 4) R *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas * R);
  cfg.blockDim = dim3(kSharedWarps * 32);
  // of x: a CTA's share of K, or as many whole runs of it as fit
  constexpr int ring = kSharedWarps * kRuns * kRunBytes;
  p.chunk = std::min(((p.groups + 3) / 4 + R - 1) / R, ((kSharedSmem - ring) / p.rows - 16) / 512) * 4;
  cfg.dynamicSmemBytes = ring + p.rows * (p.chunk * 128 + 16);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = R;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = R > 1 ? 1 : 0;
  auto kernel = quant_linear_shared_kernel<T>;
  // The limit belongs to the kernel, not to the call: every call sets the same one, so that no thread lowers another's.
  static_assert(kSharedSmem - ring >= 8 * (512 + 16), "a run of 8 rows fits");
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedSmem);
  if (e != cudaSuccess) return launch_status(e);
  return launch_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

// ---- many weights, fp32 ----
// Splitting x into its parts takes more instructions than a tile's MMAs, so with many tiles it is done once per
// CTA: the parts lie in shared memory (in chunks of K, rows 16 bytes apart beyond their length, for the banks)
// and 16 warps read their fragments there.  Weights reach a warp through its own ring of cp.async stages (16 rows
// x 128 bytes, 4 groups): fully coalesced, no barrier between warps.  Inside a stage the 32-byte slot of group G
// of row r is G ^ (r & 3), which makes the 8-byte fragment reads free of bank conflicts.  K is split over KW warps
// (1 .. 16, a power of two) such that the tiles times KW about fill the GPU's SMs with 16 warps each.
constexpr int kWarps = 16, kStages = 3, kStageBytes = 2048;
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int kXBytes = kMaxSmem - kRingBytes;   // for x

// ke elements from k0 on of x's rows to shared memory in three bf16 parts.  The warps share the rows evenly.
__device__ __forceinline__ void stage_x(const LinearArgs& p, uint8_t* xs, int xrow, int64_t k0, int ke) {
  constexpr int U = 4;
  const int xpart = p.rows * xrow;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int per_row = 1;                                       // warps to a row
  while (per_row * 2 * p.rows <= kWarps) per_row *= 2;
  const int first = (warp % per_row) * 32 + lane, step = per_row * 32;
  // quads of values: the last one again beyond the end, with the same values
  const int quads = ke / 4;
  for (int r = warp / per_row; r < p.rows; r += kWarps / per_row) {
    const float* src = (const float*)p.x + r * p.ldx + k0;
    uint8_t* dst = xs + r * xrow;
    for (int v0 = first; v0 < quads; v0 += U * step) {
      float in[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* from = src + min(v0 + u * step, quads - 1) * 4;
        if (p.wide) {
          const float4 q = *reinterpret_cast<const float4*>(from);
          in[u][0] = q.x, in[u][1] = q.y, in[u][2] = q.z, in[u][3] = q.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) in[u][j] = from[j];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = min(v0 + u * step, quads - 1);
        bf16 q[4][3];
#pragma unroll
        for (int j = 0; j < 4; ++j) split(in[u][j], q[j]);
#pragma unroll
        for (int h = 0; h < 3; ++h) {
          Vec<bf16, 4> o;
#pragma unroll
          for (int j = 0; j < 4; ++j) o.v[j] = q[j][h];
          *reinterpret_cast<Vec<bf16, 4>*>(dst + h * xpart + v * 8) = o;
        }
      }
    }
  }
}

// MT: 8-row tiles of x
template <int MT>
__global__ void __launch_bounds__(kWarps * 32, 1) quant_linear_staged_kernel(const LinearArgs p) {
  using M = bf16;
  constexpr int PARTS = 3;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  uint8_t* xs = smem + kRingBytes;
  const int xrow = p.chunk * 128 + 16;                  // bytes of a row of one part
  const int xpart = p.rows * xrow;
  const int kw = p.kw, per_cta = kWarps / kw, wk = warp & (kw - 1), wt = warp / kw;
  const int64_t row_bytes = (int64_t)p.groups * 32;
  const int tiles = (p.n + 15) / 16;
  // a lane copies 16 bytes of rows i 4 + lane / 8 of a stage; chunk c of row r lies in slot (c / 2) ^ (r & 3)
  const int cr = lane >> 3, cc = lane & 7;
  const uint32_t copy_to = (uint32_t)__cvta_generic_to_shared(ring) + cr * 128 + ((((cc >> 1) ^ cr) << 1) | (cc & 1)) * 16;
  // columns of x behind the last row repeat row 0: they only reach outputs that are dropped
  uint32_t xf[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xf[m] = (uint32_t)__cvta_generic_to_shared(xs) + (m * 8 + g < p.rows ? m * 8 + g : 0) * xrow + t * 32;
  uint32_t frag[4];                                      // group G of the first stage
#pragma unroll
  for (int G = 0; G < 4; ++G) frag[G] = (uint32_t)__cvta_generic_to_shared(ring) + g * 128 + t * 8 + (G ^ (g & 3)) * 32;

  const UnpackConst<M> consts;
  bool staged = false;
  for (int tb = blockIdx.x * per_cta; tb < tiles; tb += gridDim.x * per_cta) {
    const int tile = tb + wt, o0 = tile * 16;
    const bool live = tile < tiles;
    const uint8_t* src[4];                               // rows past n are the last one again; dropped below
#pragma unroll
    for (int i = 0; i < 4; ++i) src[i] = p.packed + min(o0 + i * 4 + cr, p.n - 1) * row_bytes + cc * 16;
    const __half* sa = p.scale + (int64_t)min(o0 + g, p.n - 1) * p.groups + t;
    const __half* sb = p.scale + (int64_t)min(o0 + g + 8, p.n - 1) * p.groups + t;
    float acc[MT][4] = {};
    for (int c0 = 0; c0 < p.groups; c0 += p.chunk) {
      const int held = min(p.chunk, p.groups - c0);
      // stage st of this warp: groups (st kw + wk) per .. of the chunk, so that the warps go through K together
      const int per = p.per, round = kw * per, stages = (held + round - 1) / round;
      uint32_t sca[kStages], scb[kStages];               // scales of rows g and g + 8, group t of a stage (their bits)
      // stage by stage: the sources move on with it
      const uint8_t* from[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) from[i] = src[i] + (int64_t)(c0 + wk * per) * 32;
      const __half *from_a = sa + c0 + wk * per, *from_b = sb + c0 + wk * per;
      int todo = live ? held - wk * per : 0;             // groups from the next stage to issue on
      auto issue = [&](int slot, uint32_t& s_a, uint32_t& s_b) {
        const int ng = min(per, todo);
        if ((cc >> 1) < ng)
#pragma unroll
          for (int i = 0; i < 4; ++i) cp_async16(copy_to + slot * kStageBytes + i * 512, from[i]);
        if (t < ng) {
          s_a = *reinterpret_cast<const unsigned short*>(from_a);
          s_b = *reinterpret_cast<const unsigned short*>(from_b);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) from[i] += round * 32;
        from_a += round;
        from_b += round;
        todo -= round;
        cp_commit();                                     // an empty group keeps the count
      };
      if (!staged) __syncthreads();                      // the previous chunk of x is read
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) issue(i, sca[i], scb[i]);
      if (!staged) {
        stage_x(p, xs, xrow, (int64_t)c0 * 64, held * 64);
        __syncthreads();
        staged = p.chunk >= p.groups;                    // all of x stays for the following tiles
      }
      // group G of a stage: its weights from at_w on, its x at_x behind the rows' starts
      auto group = [&](uint32_t at_w, uint32_t at_x, int G, uint32_t s_a, uint32_t s_b) {
        const uint2 wa = lds8(at_w), wb = lds8(at_w + 8 * 128);
        s_a = __shfl_sync(0xffffffffu, s_a, (lane & 28) | G);
        s_b = __shfl_sync(0xffffffffu, s_b, (lane & 28) | G);
        float c[MT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pa[4], pb[4];
          unpack8(h ? wa.y : wa.x, pa, consts);
          unpack8(h ? wb.y : wb.x, pb, consts);
          const uint32_t a0[4] = {pa[0], pb[0], pa[1], pb[1]}, a1[4] = {pa[2], pb[2], pa[3], pb[3]};
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
              const uint4 b = lds16(xf[m] + at_x + q * xpart + h * 16);
              if (h == 0 && q == 0) mma16816<true>(c[m], a0, b.x, b.y, M());
              else mma16816<false>(c[m], a0, b.x, b.y, M());
              mma16816<false>(c[m], a1, b.z, b.w, M());
            }
        }
        const float fa = __half2float(__ushort_as_half((unsigned short)s_a)), fb = __half2float(__ushort_as_half((unsigned short)s_b));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[m][0] = fmaf(fa, c[m][0], acc[m][0]);
          acc[m][1] = fmaf(fa, c[m][1], acc[m][1]);
          acc[m][2] = fmaf(fb, c[m][2], acc[m][2]);
          acc[m][3] = fmaf(fb, c[m][3], acc[m][3]);
        }
      };
      for (int st0 = 0; st0 < stages; st0 += kStages) {
#pragma unroll
        for (int u = 0; u < kStages; ++u) {
          const int st = st0 + u;
          if (st >= stages) break;
          cp_wait<kStages - 2>();
          __syncwarp();                                  // every lane's copies of this stage are in; the slot before it is free
          const uint32_t s_a = sca[u], s_b = scb[u];
          constexpr int kNext = kStages - 1;
          issue((u + kNext) % kStages, sca[(u + kNext) % kStages], scb[(u + kNext) % kStages]);
          const int gl = st * round + wk * per, ng = live ? min(per, held - gl) : 0;
          if (ng == 4) {
#pragma unroll
            for (int G = 0; G < 4; ++G) group(frag[G] + u * kStageBytes, (gl + G) * 128, G, s_a, s_b);
          } else {
#pragma unroll
            for (int G = 0; G < 3; ++G)
              if (G < ng) group(frag[G] + u * kStageBytes, (gl + G) * 128, G, s_a, s_b);
          }
        }
      }
      cp_wait<0>();
      __syncwarp();
    }
    // partial sums [warp][x row][16 outputs] over the idle ring: 64 rows at most, 4 KB a warp
    float* part = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[(m * 8 + 2 * t + (e & 1)) * 16 + g + (e >> 1) * 8] = acc[m][e];
    __syncthreads();
    // output i: value i % 16 of tile i / 16 % per_cta of row m (per_cta is a power of two)
    const int outs = per_cta * 16 * p.rows, shift = __ffs(per_cta) + 3;
    auto sum = [&](int i) {                              // over the tile's warps, in order
      const int wi = (i >> 4) & (per_cta - 1), at = (i >> shift) * 16 + (i & 15);
      float v = 0.f;
      for (int k = 0; k < kw; ++k) v += reinterpret_cast<float*>(smem + (wi * kw + k) * kStages * kStageBytes)[at];
      return v;
    };
    for (int i = threadIdx.x; i < outs; i += kWarps * 32) {
      const int m = i >> shift, o = (tb * 16) + (i & (per_cta * 16 - 1));
      if (o >= p.n) continue;
      float v = sum(i);
      v *= kUnpackScale<M>;
      if (p.bias) v += p.bias[o];
      ((float*)p.y)[m * p.ldy + o] = p.act == GAM_ACT_SWISH ? swish_f<float>(v) : v;
    }
    __syncthreads();
  }
}

template <int MT>
gam_status launch_staged(LinearArgs p, int sms, cudaStream_t s) {
  constexpr int PARTS = 3;
  const int tiles = (p.n + 15) / 16;
  p.kw = 1;
  while (p.kw < kWarps && p.kw * 2 <= p.groups && (int64_t)tiles * p.kw * 2 <= (int64_t)sms * kWarps) p.kw *= 2;
  const int per_cta = kWarps / p.kw;
  p.per = p.groups >= 4 * p.kw ? 4 : p.groups >= 2 * p.kw ? 2 : 1;
  // all of x when it fits, else chunks of a multiple of 4 kw groups if possible, so that the warps' shares are even
  p.chunk = std::min(p.groups, (kXBytes / (p.rows * PARTS) - 16) / 128);
  if (p.chunk < p.groups && p.chunk > 4 * p.kw) p.chunk = p.chunk / (4 * p.kw) * (4 * p.kw);
  auto kernel = quant_linear_staged_kernel<MT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e != cudaSuccess) return launch_status(e);
  const int smem = kRingBytes + p.rows * PARTS * (p.chunk * 128 + 16);
  return launch_status(launch_kernel(kernel, std::min((tiles + per_cta - 1) / per_cta, sms), kWarps * 32, smem, s, p));
}

// Forms by size, measured in us (thin with one tile, thin with two, staged):
//   16-bit, 16 x 16384 x 4096: 27.2, 19.5, 19.3; 30 x 3712 x 5888: 17.7, 11.6, 20.8; 16 x 4096 x 1024: 3.6, 3.5, 3.4
//   16-bit, 2 x 4745 x 4224: 7.5, -, 9.4; 1 x 768 x 768: 2.4, -, 5.0
//   16-bit, up to 8 rows (thin, shared): 8 x 16384 x 4096: 23.5, 13.9; 8 x 8192 x 8192: 26.8, 14.1; 1 x 5120 x 8192:
//     14.3, 13.0; 1 and 8 x 6144 x 4096: 8.7, 9.0 and 9.4, 8.8; 8 x 4096 x 8192: 11.6, 12.3; 8 x 8192 x 1024: 4.9, 5.6
//   fp32, 2 x 15083 x 3904: 36.7, 37.1, 20.3; 16 x 16384 x 4096: 77.7, 68.0, 43.1; 64 x 4096 x 4096: 76.2, 66.1, 173
//   fp32, 7 x 6272 x 2496: 13.5, 14.9, 12.1; 5 x 1025 x 1024: 3.8, 4.9, 5.2
template <typename T>
gam_status launch(const LinearArgs& p, int sms, cudaStream_t s) {
  const int64_t weights = (int64_t)p.n * p.groups * 64;
  if constexpr (Elem<T>::parts == 1) {
    if (p.rows <= 8) return p.n > 4096 && weights >= (24 << 20) ? launch_shared<T>(p, sms, s) : launch_thin<T, 1, 1>(p, sms, s);
    return p.n < 2048 ? launch_thin<T, 2, 1>(p, sms, s) : launch_thin<T, 2, 2>(p, sms, s);
  } else {
    if (weights <= (8 << 20)) return launch_thin<T, 1, 1>(p, sms, s);
    if (p.rows <= 8) return launch_staged<1>(p, sms, s);
    if (p.rows <= 16) return launch_staged<2>(p, sms, s);
    return launch_thin<T, 1, 2>(p, sms, s);
  }
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
    if (n > kMaxDim || k > kMaxDim) return op_fail(GAM_ERR_CAPACITY, "n and k up to 2^30");
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
    const LinearArgs p{x,   packed, static_cast<const __half*>(scale), bias, y, ldx, ldy, act, rows, n, k / 64,
                       aligned(x, 16) && (rows == 1 || ldx % (16 / es) == 0), 1, 4, 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == GAM_DTYPE_F32) return launch<float>(p, sms, s);
    if (dtype == GAM_DTYPE_F16) return launch<__half>(p, sms, s);
    return launch<bf16>(p, sms, s);
  });
}
