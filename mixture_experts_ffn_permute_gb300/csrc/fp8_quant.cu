// Quantisation to E4M3 with a scale per block of 128 (moe_fp8_quantize_* of
// include/moe_experts.h).
//
// HBM bound: every value is read once and its code written once.  T=8192 H=7168 bf16
// 29.4 us (6.05 TB/s, 0.89 of the copy rate), SwiGLU T=8192 H=14336 95.2 us (0.91), weights
// E=8 N=4096 K=14336 with transposed codes 272 us (1.01).  Codes of products with the rounded
// reciprocal in place of quotients took 28.9, 92.4 and 267.
//
// Rows.  A thread takes 16 consecutive values (one or two 32-byte loads, one
// 16-byte store), eight threads a block, whose maximum goes through three shuffles;
// with SwiGLU it takes 16 gate and the 16 up values that belong to them.
// Threads walk the blocks of all rows.
//
// Weights.  A CTA takes one 128 x 128 block into registers (64 values a thread,
// bf16 ones in pairs), finds its maximum, and writes the codes; transposed ones
// through shared memory, so that both sides are written in whole 128-byte rows.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_experts.h"
#include "internal.h"
#include "lowprec.cuh"
#include "ptx.cuh"
#include "rowwise.cuh"

namespace moe {
namespace {

constexpr int kBlock = 128;
constexpr int kPer = 16;                   // values of a thread
constexpr int kThreadsPer = kBlock / kPer; // of a block
constexpr float kE4m3Max = 448.f;
constexpr float kDown = 0x1p-80f;

// max(|a|, |b|), NaN where one is
__device__ __forceinline__ float amax(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

__device__ __forceinline__ float scale_of(float m) {
  // (a NaN stays)
  return m == 0.f ? 1.f : m / kE4m3Max < 0x1p-126f ? 0x1p-126f : m / kE4m3Max;
}

// Sixteen values of a row, as loaded.
template <typename T, bool kWide>
struct Values;
template <bool kWide>
struct Values<Bf16, kWide> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const Bf16* p) {
    if (kWide) {
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                     "=r"(w[6]), "=r"(w[7])
                   : "l"(p)
                   : "memory");
    } else {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
      const uint4 b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    return (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
  }
};
template <bool kWide>
struct Values<float, kWide> {
  float f[16];
  __device__ __forceinline__ void load(const float* p) {
    if (kWide) {
      float a[8], b[8];
      load_stream32(a, p);
      load_stream32(b, p + 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = a[i], f[8 + i] = b[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p) + i);
        f[4 * i] = a.x, f[4 * i + 1] = a.y, f[4 * i + 2] = a.z, f[4 * i + 3] = a.w;
      }
    }
  }
  __device__ __forceinline__ float get(int i) const { return f[i]; }
};

// x / (1 + exp(-x)) by the exponential of -|x|, which is at most 1.  The fast
// forms are off by about |x| 2^-24, far below a code's 2^-4, and without them the
// arithmetic takes longer than the bytes.  (The divisor is 1 to 2: its reciprocal needs no
// care for sizes.)
__device__ __forceinline__ float silu(float x) {
  const float e = __expf(-fabsf(x));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return (x < 0.f ? x * e : x) * r;
}

// The reciprocal of a scale in two parts, 1 / s = y + y2.
struct Inverse {
  float y, y2;
  bool big;  // y2 would be subnormal: those of kDown s, for kDown v
};
__device__ __forceinline__ Inverse inverse_of(float scale) {
  Inverse r;
  r.big = !(scale < 0x1p100f);  // (or the scale is NaN)
  const float s = r.big ? scale * kDown : scale;
  r.y = 1.f / s;
  const float e = __fmaf_rn(-s, r.y, 1.f), d = e * r.y;
  r.y2 = s < INFINITY ? __fmaf_rn(__fmaf_rn(-d, s, e), r.y, d) : 0.f;  // e / s (Markstein 1990)
  return r;
}

// The codes of v / s in fp32.  A product with the rounded reciprocal is two roundings, and a
// quotient that lies on the border of two codes (of bf16 values one in some 2000) would fall to
// either side; v y + v y2 has one that counts.  Every value and scale whose result could lie on
// another side of a border than their quotient in fp32 were gone through: none does.  (v y2 is
// rounded down, as a sum with -0, so that a zero keeps its sign.)
__device__ __forceinline__ uint4 codes_of(float (&v)[kPer], const Inverse& r) {
  if (r.big) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] *= kDown;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = __fmaf_rn(v[i], r.y, __fmaf_rd(v[i], r.y2, -0.f));
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = f32x2_to_e4m3x2(v[4 * i], v[4 * i + 1]) | f32x2_to_e4m3x2(v[4 * i + 2], v[4 * i + 3]) << 16;
  return make_uint4(c[0], c[1], c[2], c[3]);
}

struct RowParams {
  const void* src;
  uint4* codes;
  float* scales;
  int T, H, blocks;  // blocks per row
  long ld;
  int interleave;    // SwiGLU: H where the halves lie apart
  float clamp;       // 0: none
};

template <typename T, bool kGlu, bool kWide>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const RowParams p) {
  pdl_enter();
  const uint32_t total = static_cast<uint32_t>(p.T) * p.blocks;  // below 2^31
  const uint32_t stride = gridDim.x * (256 / kThreadsPer);
  const int sub = threadIdx.x % kThreadsPer;
  // (whole warps run the loop together: the shuffles below)
  for (uint32_t q0 = blockIdx.x * (256 / kThreadsPer); q0 < total; q0 += stride) {
    const uint32_t q = q0 + threadIdx.x / kThreadsPer;
    const long t = q / static_cast<uint32_t>(p.blocks);
    const int b = static_cast<int>(q % static_cast<uint32_t>(p.blocks));
    const int c = b * kBlock + sub * kPer;
    const bool in = q < total && c < p.H;
    float v[kPer];
    if (in) {
      const T* row = static_cast<const T*>(p.src) + t * p.ld;
      if (kGlu) {
        const int at = p.interleave == p.H ? c : c / p.interleave * (2 * p.interleave) + c % p.interleave;
        Values<T, kWide> g, u;
        g.load(row + at);
        u.load(row + at + p.interleave);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          float x = g.get(i), y = u.get(i);
          if (p.clamp > 0.f) {  // (a NaN stays)
            x = x > p.clamp ? p.clamp : x;
            y = y > p.clamp ? p.clamp : y < -p.clamp ? -p.clamp : y;
          }
          v[i] = silu(x) * y;
        }
      } else {
        Values<T, kWide> x;
        x.load(row + c);
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = x.get(i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = 0.f;
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = amax(m, v[i]);
#pragma unroll
    for (int o = 1; o < kThreadsPer; o *= 2) m = amax(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float scale = scale_of(m);
    if (in) {
      p.codes[(t * p.H + c) / kPer] = codes_of(v, inverse_of(scale));
      if (sub == 0) p.scales[q] = scale;
    }
  }
}

struct WeightParams {
  const void* src;
  uint8_t *codes, *codes_t;
  float *scales, *scales_t;
  int N, K, n_blocks, k_blocks;
};

// Columns of four rows: w[r] holds four codes of row r, out[c] the four rows'
// codes of column c.
__device__ __forceinline__ void transpose4(const uint32_t (&w)[4], uint32_t (&out)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
  out[0] = __byte_perm(a, b, 0x5410);
  out[1] = __byte_perm(a, b, 0x7632);
  out[2] = __byte_perm(c, d, 0x5410);
  out[3] = __byte_perm(c, d, 0x7632);
}

// One CTA per 128 x 128 block: thread i has the rows 4 (i / 8) .. + 3, the columns
// 16 (i % 8) .. + 15.
// (bf16: 80 registers, three CTAs to an SM; a form of 127 registers took 329 us for the 272 above)
template <typename T, bool kWide, bool kTransposed>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) quantize_weights_kernel(const WeightParams p) {
  __shared__ float s_max[8];
  // codes by column, in words of four rows; the words of column k change places
  // by k / 16, so that a warp's words lie in 32 banks
  __shared__ __align__(16) uint32_t s_codes[kTransposed ? kBlock * kBlock / 4 : 4];
  pdl_enter();
  const uint32_t blk = blockIdx.x;
  const uint32_t per = static_cast<uint32_t>(p.n_blocks) * p.k_blocks;
  const long e = blk / per;
  const int in_e = static_cast<int>(blk % per);
  const int bn = in_e / p.k_blocks, bk = in_e - bn * p.k_blocks;
  const int sub = threadIdx.x % 8, quad = threadIdx.x / 8;
  const int row = bn * kBlock + 4 * quad, col = bk * kBlock + sub * kPer;
  const T* src = static_cast<const T*>(p.src) + (e * p.N + row) * p.K + col;
  Values<T, kWide> x[4];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (row + i < p.N && col < p.K) x[i].load(src + static_cast<long>(i) * p.K);
    else x[i] = Values<T, kWide>{};
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) m = amax(m, x[i].get(j));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = amax(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = amax(m, s_max[w]);
  const float scale = scale_of(m);
  const Inverse inv = inverse_of(scale);
  if (threadIdx.x == 0) {
    p.scales[blk] = scale;
    if (kTransposed) p.scales_t[(e * p.k_blocks + bk) * p.n_blocks + bn] = scale;
  }
  uint4 c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = x[i].get(j);
    c[i] = codes_of(v, inv);
    if (row + i < p.N && col < p.K)
      *reinterpret_cast<uint4*>(p.codes + (e * p.N + row + i) * p.K + col) = c[i];
  }
  if (kTransposed) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {  // columns 4 g .. + 3 of this thread's 16
      auto word = [&](const uint4& q) { return g == 0 ? q.x : g == 1 ? q.y : g == 2 ? q.z : q.w; };
      const uint32_t w[4] = {word(c[0]), word(c[1]), word(c[2]), word(c[3])};
      uint32_t out[4];
      transpose4(w, out);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s_codes[(sub * kPer + 4 * g + j) * (kBlock / 4) + (quad ^ sub * 4)] = out[j];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = quad + 32 * i, n = bn * kBlock + sub * 16;
      if (bk * kBlock + k < p.K && n < p.N)
        *reinterpret_cast<uint4*>(p.codes_t + (e * p.K + bk * kBlock + k) * p.N + n) =
            *reinterpret_cast<const uint4*>(s_codes + k * (kBlock / 4) + (sub ^ (k / 16)) * 4);
    }
  }
}

bool off(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

template <typename T>
cudaError_t launch_rows(const RowParams& p, bool glu, bool wide, cudaStream_t s) {
  const long blocks = (static_cast<long>(p.T) * p.blocks + 31) / 32;
  const dim3 grid(static_cast<unsigned>(std::min<long>(blocks, 16L * num_sms()))), block(256);
  auto kern = glu ? (wide ? quantize_rows_kernel<T, true, true> : quantize_rows_kernel<T, true, false>)
                  : (wide ? quantize_rows_kernel<T, false, true> : quantize_rows_kernel<T, false, false>);
  return launch_kernel(kern, grid, block, 0, s, 1, p);
}

template <typename T>
cudaError_t launch_weights(const WeightParams& p, long blocks, bool wide, cudaStream_t s) {
  auto kern = p.codes_t ? (wide ? quantize_weights_kernel<T, true, true>
                                : quantize_weights_kernel<T, false, true>)
                        : (wide ? quantize_weights_kernel<T, true, false>
                                : quantize_weights_kernel<T, false, false>);
  return launch_kernel(kern, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, 1, p);
}

int check_rows(const moe_quant_problem* p) {
  if (!p || p->T < 0 || p->H < 1) return MOE_ERR_INVALID_ARG;
  if (p->src_dtype != MOE_DTYPE_BF16 && p->src_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (p->H % 16 != 0 || p->H > (1 << 28)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (p->glu_interleave < 0) return MOE_ERR_INVALID_ARG;
  if (p->swiglu && p->glu_interleave != 0 &&
      (p->glu_interleave % 16 != 0 || p->H % p->glu_interleave != 0))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  const int64_t width = p->swiglu ? 2LL * p->H : p->H;
  if (p->ld_src != 0 && p->ld_src < width) return MOE_ERR_INVALID_ARG;
  if (p->ld_src % 8 != 0 || p->ld_src > (1LL << 40) ||
      static_cast<int64_t>(p->T) * ceil_div(p->H, kBlock) >= (1LL << 31) - (1 << 24))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_fp8_quantize_rows(const moe_quant_problem* p, const void* src, void* codes,
                                     float* scales, void* stream) {
  const int rc = check_rows(p);
  if (rc != MOE_OK) return rc;
  set_last_launch_count(0);
  if (p->T == 0) return MOE_OK;
  if (!src || !codes || !scales) return MOE_ERR_INVALID_ARG;
  if (off(src, 16) || off(codes, 16) || off(scales, 4)) return MOE_ERR_MISALIGNED;
  RowParams r{};
  r.src = src;
  r.codes = static_cast<uint4*>(codes);
  r.scales = scales;
  r.T = p->T;
  r.H = p->H;
  r.blocks = ceil_div(p->H, kBlock);
  r.ld = p->ld_src ? p->ld_src : (p->swiglu ? 2L : 1L) * p->H;
  r.interleave = p->glu_interleave ? p->glu_interleave : p->H;
  const float c = p->swiglu_clamp;
  r.clamp = c > 0.f && std::isfinite(c) ? c : 0.f;
  const int size = p->src_dtype == MOE_DTYPE_F32 ? 4 : 2;
  const bool wide = !off(src, 32) && r.ld * size % 32 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t err = size == 4 ? launch_rows<float>(r, p->swiglu != 0, wide, s)
                                    : launch_rows<Bf16>(r, p->swiglu != 0, wide, s);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  set_last_launch_count(1);
  return MOE_OK;
}

extern "C" int moe_fp8_quantize_weights(const moe_quant_weights_problem* p, const void* src,
                                        void* codes, float* scales, void* codes_t, float* scales_t,
                                        void* stream) {
  if (!p || p->E < 0 || p->N < 1 || p->K < 1) return MOE_ERR_INVALID_ARG;
  if (p->src_dtype != MOE_DTYPE_BF16 && p->src_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  const long n_blocks = ceil_div(p->N, kBlock), k_blocks = ceil_div(p->K, kBlock);
  if (p->K % 16 != 0 || n_blocks * k_blocks >= (1L << 31) ||
      p->E * n_blocks * k_blocks >= (1L << 31))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!codes_t != !scales_t) return MOE_ERR_INVALID_ARG;
  if (codes_t && p->N % 16 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  set_last_launch_count(0);
  if (p->E == 0) return MOE_OK;
  if (!src || !codes || !scales) return MOE_ERR_INVALID_ARG;
  if (off(src, 16) || off(codes, 16) || off(codes_t, 16) || off(scales, 4) || off(scales_t, 4))
    return MOE_ERR_MISALIGNED;
  WeightParams w{};
  w.src = src;
  w.codes = static_cast<uint8_t*>(codes);
  w.codes_t = static_cast<uint8_t*>(codes_t);
  w.scales = scales;
  w.scales_t = scales_t;
  w.N = p->N;
  w.K = p->K;
  w.n_blocks = static_cast<int>(n_blocks);
  w.k_blocks = static_cast<int>(k_blocks);
  const bool wide = !off(src, 32);  // rows are whole 32 bytes: K is a multiple of 16
  const long blocks = p->E * n_blocks * k_blocks;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t err = p->src_dtype == MOE_DTYPE_F32 ? launch_weights<float>(w, blocks, wide, s)
                                                        : launch_weights<Bf16>(w, blocks, wide, s);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  set_last_launch_count(1);
  return MOE_OK;
}
