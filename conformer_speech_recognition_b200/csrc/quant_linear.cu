// Few-row linear layer on INT4-g64 weights: gam_quant_linear.
//
//   y[m, o] = act(bias[o] + sum_g scale[o, g] sum_{j in g} q[o, j] x[m, j])
//
// The weights are read once and the rows are few, so the bound is the weight
// stream (0.53 bytes per weight) and, close behind it, the instructions that turn
// integers into an MMA operand.  A warp owns 16 outputs: mma.m16n8k16 with the
// weights as the 16-row operand and up to 64 rows of x as 8-column tiles.  The
// integers are exact in both 16-bit types, so a group's sum is that of q x itself
// and is scaled in fp32 by the group's scale.
//
// Weights reach a warp through its own ring of cp.async stages (16 rows x 128
// bytes, 4 groups): fully coalesced, no barrier between warps, and enough bytes in
// flight per SM to cover the memory's latency.  Inside a stage the 32-byte slot of
// group G of row r is G ^ (r & 3), which makes the 8-byte fragment reads free of
// bank conflicts.  The words' nibble order gives adjacent pairs by one shift and
// mask.  A lane's 16 weights of a group are 16 consecutive k, so its fragments of x
// are two 16-byte reads of a row in shared memory; rows are 16 bytes apart beyond
// their length, again for the banks.
//
// K is split over KW warps of a CTA (1 .. 16, a power of two) such that the tiles
// times KW about fill the GPU's SMs with 16 warps each; the partial sums meet in
// shared memory and are added in a fixed order.
//
// fp32 x is held as three bf16 parts (8 + 8 + 8 bits: exact), each with its own MMA.
#include <algorithm>

#include "stream_ops.cuh"

namespace gam {
namespace ops {
namespace {

constexpr int kWarps = 16, kStages = 3, kStageBytes = 2048;
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int kMaxSmem = 227 * 1024;
constexpr int kXBytes = kMaxSmem - kRingBytes;   // for x

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

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bf16) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8 weights of a word as four pairs.  fp16: 1024 + u and, from the nibbles left
// in place 4 bits up, 1024 + 16 u are exact, and so is the fused subtraction.
// bf16: 128 + u is exact; the pairs are 2^-9 q there, so that a group's sum of the
// largest finite x stays finite (64 * 7 < 2^9), and the scale takes 2^9 back.
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&p)[4], __half) {
  const uint32_t w8 = w >> 8;
  const uint32_t r[4] = {(w & 0x000F000Fu) | 0x64006400u, (w & 0x00F000F0u) | 0x64006400u,
                         (w8 & 0x000F000Fu) | 0x64006400u, (w8 & 0x00F000F0u) | 0x64006400u};
  const __half2 one = __float2half2_rn(1.f), lo = __float2half2_rn(-1032.f);
  const __half2 six = __float2half2_rn(0.0625f), hi = __float2half2_rn(-72.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = *reinterpret_cast<const __half2*>(&r[i]);
    const __half2 q = (i & 1) ? __hfma2(v, six, hi) : __hfma2(v, one, lo);
    p[i] = *reinterpret_cast<const uint32_t*>(&q);
  }
}
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&p)[4], bf16) {
  const __nv_bfloat162 f = __float2bfloat162_rn(0.001953125f), c = __float2bfloat162_rn(-136.f * 0.001953125f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 q = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&r), f, c);
    p[i] = *reinterpret_cast<const uint32_t*>(&q);
  }
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

struct LinearArgs {
  const void* x;
  const uint8_t* packed;
  const __half* scale;
  const float* bias;
  void* y;
  int64_t ldx, ldy;
  int act, rows, n, groups;   // groups = k / 64
  int kw;                     // warps that share a tile's K
  int chunk;                  // groups of x held in shared memory at a time
  int wide;                   // x rows are 16-byte aligned
};

// MT: 8-row tiles of x
template <typename T, int MT>
__global__ void __launch_bounds__(kWarps * 32, 1) quant_linear_kernel(const LinearArgs p) {
  using M = typename Elem<T>::M;
  constexpr int PARTS = Elem<T>::parts;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_u = (uint32_t)__cvta_generic_to_shared(ring);
  uint8_t* xs = smem + kRingBytes;
  const int xrow = p.chunk * 128 + 16;                  // bytes of a row of one part
  const int xpart = p.rows * xrow;
  const int kw = p.kw, per_cta = kWarps / kw, wk = warp & (kw - 1), wt = warp / kw;
  const int64_t row_bytes = (int64_t)p.groups * 32;
  const int tiles = (p.n + 15) / 16;
  const T* x = (const T*)p.x;
  bool staged = false;

  for (int tb = blockIdx.x * per_cta; tb < tiles; tb += gridDim.x * per_cta) {
    const int tile = tb + wt, o0 = tile * 16;
    const bool live = tile < tiles;
    float acc[MT][4] = {};
    for (int c0 = 0; c0 < p.groups; c0 += p.chunk) {
      const int cg = min(p.chunk, p.groups - c0);
      const int s0 = cg * wk / kw, s1 = live ? cg * (wk + 1) / kw : s0;   // this warp's groups of the chunk
      const int stages = (s1 - s0 + 3) >> 2;
      uint32_t sc[kStages];                              // scales of rows g and g + 8, group t of a stage
      auto issue = [&](int st, uint32_t& sreg) {
        if (st < stages) {
          const int gb = c0 + s0 + st * 4, ng = min(4, s1 - s0 - st * 4);
          const uint32_t dst = ring_u + (st % kStages) * kStageBytes;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 4 + (lane >> 3), c = lane & 7;
            if ((c >> 1) < ng)
              cp_async16(dst + r * 128 + ((((c >> 1) ^ (r & 3)) << 1) | (c & 1)) * 16,
                         p.packed + min(o0 + r, p.n - 1) * row_bytes + (int64_t)gb * 32 + c * 16);
          }
          const int gt = gb + min(t, ng - 1);
          const __half a = p.scale[(int64_t)min(o0 + g, p.n - 1) * p.groups + gt];
          const __half b = p.scale[(int64_t)min(o0 + g + 8, p.n - 1) * p.groups + gt];
          const __half2 ab = __halves2half2(a, b);
          sreg = *reinterpret_cast<const uint32_t*>(&ab);
        }
        cp_commit();                                     // an empty group keeps the count
      };
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) issue(i, sc[i]);
      if (!staged) {
        __syncthreads();                                 // the previous chunk of x is read
        const int ke = cg * 64;                          // elements of a row in this chunk
        if (p.wide) {
          constexpr int V = 16 / sizeof(T);
          const int vecs = ke / V;
          for (int i = threadIdx.x; i < p.rows * vecs; i += kWarps * 32) {
            const int r = i / vecs, v = i % vecs;
            const Vec<T, V> in = *reinterpret_cast<const Vec<T, V>*>(x + r * p.ldx + (int64_t)c0 * 64 + v * V);
            if constexpr (PARTS == 1) {
              *reinterpret_cast<Vec<T, V>*>(xs + r * xrow + v * 16) = in;
            } else {
              Vec<bf16, V> o[3];
#pragma unroll
              for (int j = 0; j < V; ++j) {
                bf16 q[3];
                split(in.v[j], q);
                o[0].v[j] = q[0], o[1].v[j] = q[1], o[2].v[j] = q[2];
              }
#pragma unroll
              for (int q = 0; q < 3; ++q) *reinterpret_cast<Vec<bf16, V>*>(xs + q * xpart + r * xrow + v * V * 2) = o[q];
            }
          }
        } else {
          for (int i = threadIdx.x; i < p.rows * ke; i += kWarps * 32) {
            const int r = i / ke, v = i % ke;
            const T in = x[r * p.ldx + (int64_t)c0 * 64 + v];
            if constexpr (PARTS == 1) {
              *reinterpret_cast<T*>(xs + r * xrow + v * 2) = in;
            } else {
              bf16 q[3];
              split(in, q);
#pragma unroll
              for (int j = 0; j < 3; ++j) *reinterpret_cast<bf16*>(xs + j * xpart + r * xrow + v * 2) = q[j];
            }
          }
        }
        __syncthreads();
        staged = p.chunk >= p.groups;                    // all of x stays for the following tiles
      }
      // columns of x behind the last row repeat row 0: they only reach outputs that are dropped
      const uint8_t* xf[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) xf[m] = xs + (m * 8 + g < p.rows ? m * 8 + g : 0) * xrow + t * 32;
      for (int st0 = 0; st0 < stages; st0 += kStages) {
#pragma unroll
        for (int u = 0; u < kStages; ++u) {
          const int st = st0 + u;
          if (st >= stages) break;
          cp_wait<kStages - 2>();
          __syncwarp();                                  // every lane's copies of this stage are in; the slot before it is free
          const uint32_t scales = sc[u];
          issue(st + kStages - 1, sc[(u + kStages - 1) % kStages]);
          const uint8_t* sw = ring + u * kStageBytes + g * 128 + t * 8;
          const int gl = s0 + st * 4, ng = min(4, s1 - gl);
#pragma unroll
          for (int G = 0; G < 4; ++G) {
            if (G >= ng) break;
            const uint2 wa = *reinterpret_cast<const uint2*>(sw + ((G ^ (g & 3)) * 32));
            const uint2 wb = *reinterpret_cast<const uint2*>(sw + 8 * 128 + ((G ^ (g & 3)) * 32));
            const uint32_t s2 = __shfl_sync(0xffffffffu, scales, (lane & 28) | G);
            const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&s2));
            const float sa = s.x * kUnpackScale<M>, sb = s.y * kUnpackScale<M>;
            float c[MT][4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pa[4], pb[4];
              unpack8(h ? wa.y : wa.x, pa, M());
              unpack8(h ? wb.y : wb.x, pb, M());
              const uint32_t a0[4] = {pa[0], pb[0], pa[1], pb[1]}, a1[4] = {pa[2], pb[2], pa[3], pb[3]};
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int q = 0; q < PARTS; ++q) {
                  const uint4 b = *reinterpret_cast<const uint4*>(xf[m] + q * xpart + (gl + G) * 128 + h * 16);
                  mma16816(c[m], a0, b.x, b.y, M());
                  mma16816(c[m], a1, b.z, b.w, M());
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              acc[m][0] = fmaf(sa, c[m][0], acc[m][0]);
              acc[m][1] = fmaf(sa, c[m][1], acc[m][1]);
              acc[m][2] = fmaf(sb, c[m][2], acc[m][2]);
              acc[m][3] = fmaf(sb, c[m][3], acc[m][3]);
            }
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
    const int outs = p.rows * 16;
    for (int i = threadIdx.x; i < per_cta * outs; i += kWarps * 32) {
      const int wi = i / outs, r = i % outs, m = r >> 4, o = (tb + wi) * 16 + (r & 15);
      if (o >= p.n) continue;
      float v = 0.f;
      for (int k = 0; k < kw; ++k) v += reinterpret_cast<float*>(smem + (wi * kw + k) * kStages * kStageBytes)[r];
      if (p.bias) v += p.bias[o];
      ((T*)p.y)[m * p.ldy + o] = from_f<T>(p.act == GAM_ACT_SWISH ? swish_f(v) : v);
    }
    __syncthreads();
  }
}

template <typename T, int MT>
gam_status launch_mt(LinearArgs p, int sms, cudaStream_t s) {
  constexpr int PARTS = Elem<T>::parts;
  const int tiles = (p.n + 15) / 16;
  p.kw = 1;
  while (p.kw < kWarps && p.kw * 2 <= p.groups && (int64_t)tiles * p.kw * 2 <= (int64_t)sms * kWarps) p.kw *= 2;
  // all of x when it fits, else chunks of a multiple of 4 kw groups if possible, so that the warps' shares are even
  const int most = (kXBytes / (p.rows * PARTS) - 16) / 128;
  p.chunk = std::min(p.groups, most);
  if (p.chunk < p.groups && p.chunk > 4 * p.kw) p.chunk = p.chunk / (4 * p.kw) * (4 * p.kw);
  const int smem = kRingBytes + p.rows * PARTS * (p.chunk * 128 + 16);
  auto kernel = quant_linear_kernel<T, MT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e != cudaSuccess) return launch_status(e);
  const int per_cta = kWarps / p.kw;
  const int grid = std::min((tiles + per_cta - 1) / per_cta, sms);
  kernel<<<grid, kWarps * 32, smem, s>>>(p);
  return launch_status(cudaGetLastError());
}

template <typename T>
gam_status launch(const LinearArgs& p, int sms, cudaStream_t s) {
  if (p.rows <= 8) return launch_mt<T, 1>(p, sms, s);
  if (p.rows <= 16) return launch_mt<T, 2>(p, sms, s);
  if (p.rows <= 32) return launch_mt<T, 4>(p, sms, s);
  return launch_mt<T, 8>(p, sms, s);
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
    const LinearArgs p{x,   packed, static_cast<const __half*>(scale), bias, y, ldx, ldy, act, rows, n, k / 64, 1, 0,
                       aligned(x, 16) && (rows == 1 || ldx % (16 / es) == 0)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == GAM_DTYPE_F32) return launch<float>(p, sms, s);
    if (dtype == GAM_DTYPE_F16) return launch<__half>(p, sms, s);
    return launch<bf16>(p, sms, s);
  });
}
