// Global L2 norm of many gradient tensors and their clipping
// (moe_clip_grad_norm, include/moe_block.h).
//
// Two launches.  The first reads every tensor in chunks of 32 KB and leaves
// one fp64 sum of squares per block; the second adds those in a fixed order
// (every block for itself: a few KB from L2) and writes grad * factor, taking
// the chunks in the opposite order, so that it starts on what the first read
// last and still is in L2.  HBM bound: the norm is needed before the first
// output, so the tensors are read twice beyond what L2 keeps (129 MB).
//
// The tensors' table travels in the kernel parameters (no copy to the device,
// nothing to go stale in a captured graph).  Chunks start at 16-byte
// boundaries of the gradient: a tensor's leading elements before the first
// boundary belong to its first chunk.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_block.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowwise.cuh"

namespace moe {
namespace {

constexpr int kChunkBytes = 32768;
constexpr int kClipThreads = 256;
constexpr int kClipUnroll = 4;       // 16-byte loads in flight per thread
constexpr int kClipBlocksPerSm = 8;  // 2048 threads
constexpr int kMaxClipBlocks = 2048; // per launch; bounds the workspace
constexpr size_t kClipHeader = 256;
// Tables by capacity: parameters are copied with every launch, so a short list
// takes a short table.
constexpr int kSmallTable = 64, kMiddleTable = 256, kLargeTable = 1024;

template <int kCap>
struct GradTable {
  int n;
  int chunk0[kCap + 1];  // first chunk of each tensor
  const void* grad[kCap];
  void* out[kCap];
  long numel[kCap];      // sign bit: fp32
};
static_assert(sizeof(GradTable<kLargeTable>) <= 32000, "kernel parameters");

struct Chunk {
  const uint8_t* grad;  // first element
  uint8_t* out;
  long n;      // elements
  int lead;    // elements before the first 16-byte boundary
  bool f32, first;
};

template <int kCap>
__device__ __forceinline__ Chunk chunk_at(const GradTable<kCap>& t, int c) {
  int lo = 0, hi = t.n - 1;  // the last tensor whose first chunk is <= c
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.chunk0[mid] <= c) lo = mid; else hi = mid - 1;
  }
  Chunk k;
  k.f32 = t.numel[lo] < 0;
  const long numel = t.numel[lo] & 0x7fffffffffffffffL;
  const int size = k.f32 ? 4 : 2;
  const uint8_t* g = static_cast<const uint8_t*>(t.grad[lo]);
  const long lead = min(static_cast<long>((16 - (reinterpret_cast<uintptr_t>(g) & 15)) & 15) / size,
                        numel);
  const int i = c - t.chunk0[lo];
  const long per = kChunkBytes / size;
  const long from = i == 0 ? 0 : lead + i * per;
  k.n = min(numel, lead + (i + 1) * per) - from;
  k.lead = i == 0 ? static_cast<int>(lead) : 0;
  k.grad = g + from * size;
  k.out = t.out[lo] ? static_cast<uint8_t*>(t.out[lo]) + from * size : nullptr;
  return k;
}

__device__ __forceinline__ uint4 load16(const void* p) {
  return *static_cast<const uint4*>(p);
}

template <bool kF32>
__device__ __forceinline__ float square16(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kF32) {
      s = fmaf(__uint_as_float(w[i]), __uint_as_float(w[i]), s);
    } else {
      s = fmaf(bf16_lo(w[i]), bf16_lo(w[i]), s);
      s = fmaf(bf16_hi(w[i]), bf16_hi(w[i]), s);
    }
  }
  return s;
}

template <bool kF32>
__device__ __forceinline__ double square16_f64(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  double s = 0.;
  for (int i = 0; i < 4; ++i) {
    const double a = kF32 ? __uint_as_float(w[i]) : bf16_lo(w[i]);
    const double b = kF32 ? 0.f : bf16_hi(w[i]);
    s += a * a + b * b;
  }
  return s;
}

// This thread's part of a chunk's sum of squares.
template <bool kF32>
__device__ __forceinline__ double chunk_squares(const Chunk& c) {
  using T = typename std::conditional<kF32, float, Bf16>::type;
  constexpr int kPer = 16 / sizeof(T);
  const T* g = reinterpret_cast<const T*>(c.grad);
  const long vecs = (c.n - c.lead) / kPer;
  const uint4* v = reinterpret_cast<const uint4*>(g + c.lead);
  const long tail = c.lead + vecs * kPer;
  float s = 0.f;
  long i = threadIdx.x;
  for (; i + (kClipUnroll - 1) * kClipThreads < vecs; i += kClipUnroll * kClipThreads) {
    uint4 x[kClipUnroll];
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) x[u] = load16(v + i + u * kClipThreads);
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) s += square16<kF32>(x[u]);
  }
  for (; i < vecs; i += kClipThreads) s += square16<kF32>(load16(v + i));
  // the elements round the vectors: fewer than 8 on either side
  float e = 0.f;
  if (threadIdx.x < c.lead) e = to_float(g[threadIdx.x]);
  else if (threadIdx.x >= 32 && tail + (threadIdx.x - 32) < c.n)
    e = to_float(g[tail + threadIdx.x - 32]);
  s = fmaf(e, e, s);
  if (s == 0.f || (s >= 0x1p-80f && s < __int_as_float(0x7f800000))) return s;
  double d = static_cast<double>(e) * e;  // out of fp32's comfortable range: again in fp64
  for (i = threadIdx.x; i < vecs; i += kClipThreads) d += square16_f64<kF32>(load16(v + i));
  return d;
}

__device__ __forceinline__ double block_sum(double x, double* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.;
#pragma unroll
  for (int i = 0; i < kClipThreads / 32; ++i) x += s[i];
  return x;
}

template <int kCap>
__global__ void __launch_bounds__(kClipThreads)
grad_norm_kernel(const __grid_constant__ GradTable<kCap> t, double* __restrict__ part) {
  pdl_enter();
  __shared__ double s[kClipThreads / 32];
  const int chunks = t.chunk0[t.n];
  double sum = 0.;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Chunk k = chunk_at(t, c);
    sum += k.f32 ? chunk_squares<true>(k) : chunk_squares<false>(k);
  }
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <bool kF32>
__device__ __forceinline__ uint4 scale16(uint4 v, float f) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = kF32 ? __float_as_uint(__uint_as_float(w[i]) * f)
                : pack_bf16(bf16_lo(w[i]) * f, bf16_hi(w[i]) * f);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool kF32>
__device__ __forceinline__ void chunk_scale(const Chunk& c, float f) {
  using T = typename std::conditional<kF32, float, Bf16>::type;
  constexpr int kPer = 16 / sizeof(T);
  const T* g = reinterpret_cast<const T*>(c.grad);
  T* o = reinterpret_cast<T*>(c.out);
  if (((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(o)) & 15) != 0) {
    // the output's boundaries lie elsewhere: element by element
    for (long i = threadIdx.x; i < c.n; i += kClipThreads) from_float(o[i], to_float(g[i]) * f);
    return;
  }
  const long vecs = (c.n - c.lead) / kPer;
  const uint4* v = reinterpret_cast<const uint4*>(g + c.lead);
  uint4* w = reinterpret_cast<uint4*>(o + c.lead);
  const long tail = c.lead + vecs * kPer;
  long i = threadIdx.x;
  for (; i + (kClipUnroll - 1) * kClipThreads < vecs; i += kClipUnroll * kClipThreads) {
    uint4 x[kClipUnroll];
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) x[u] = load16(v + i + u * kClipThreads);
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) __stcs(w + i + u * kClipThreads, scale16<kF32>(x[u], f));
  }
  for (; i < vecs; i += kClipThreads) __stcs(w + i, scale16<kF32>(load16(v + i), f));
  if (threadIdx.x < c.lead) from_float(o[threadIdx.x], to_float(g[threadIdx.x]) * f);
  else if (threadIdx.x >= 32 && tail + (threadIdx.x - 32) < c.n)
    from_float(o[tail + threadIdx.x - 32], to_float(g[tail + threadIdx.x - 32]) * f);
}

template <int kCap>
__global__ void __launch_bounds__(kClipThreads)
grad_scale_kernel(const __grid_constant__ GradTable<kCap> t, const double* __restrict__ part,
                  int n_part, float grad_scale, float max_norm, float eps, float* norm_out) {
  pdl_enter();
  __shared__ double s[kClipThreads / 32];
  double sum = 0.;
  for (int i = threadIdx.x; i < n_part; i += kClipThreads) sum += part[i];
  sum = block_sum(sum, s);
  const float norm = static_cast<float>(fabs(static_cast<double>(grad_scale)) * sqrt(sum));
  float coef = max_norm / (norm + eps);
  if (coef >= 1.f) coef = 1.f;  // a NaN stays
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) {
    norm_out[0] = norm;
    norm_out[1] = coef;
  }
  const float f = grad_scale * coef;
  const int chunks = t.chunk0[t.n];
  for (int c = chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const Chunk k = chunk_at(t, c);
    if (!k.out || (f == 1.f && k.out == k.grad)) continue;
    if (k.f32) chunk_scale<true>(k, f);
    else chunk_scale<false>(k, f);
  }
}

// Fills the table with tensors[0 .. n); false if a tensor is too large.
template <int kCap>
void fill_table(GradTable<kCap>& t, const moe_grad_tensor* g, int n) {
  t.n = n;
  int chunks = 0;
  for (int i = 0; i < n; ++i) {
    const int size = g[i].dtype == MOE_DTYPE_F32 ? 4 : 2;
    const uintptr_t a = reinterpret_cast<uintptr_t>(g[i].grad);
    const int64_t lead = std::min<int64_t>(((16 - (a & 15)) & 15) / size, g[i].numel);
    const int64_t per = kChunkBytes / size;
    t.chunk0[i] = chunks;
    t.grad[i] = g[i].grad;
    t.out[i] = g[i].out;
    t.numel[i] = g[i].numel | (size == 4 ? INT64_MIN : 0);
    // the first chunk also takes the leading elements
    chunks += g[i].numel == 0 ? 0
                              : static_cast<int>(std::max<int64_t>(
                                    1, (g[i].numel - lead + per - 1) / per));
  }
  t.chunk0[n] = chunks;
}

int clip_blocks(int chunks) {
  return std::max(1, std::min({chunks, num_sms() * kClipBlocksPerSm, kMaxClipBlocks}));
}

template <int kCap>
int run_clip(int n, const moe_grad_tensor* g, float grad_scale, float max_norm, float eps,
             float* norm_out, double* part, cudaStream_t s) {
  GradTable<kCap> t;
  fill_table(t, g, 0);
  int launches = 0, n_part = 0;
  for (int i = 0; i < n; i += kCap) {
    fill_table(t, g + i, std::min(kCap, n - i));
    const int blocks = clip_blocks(t.chunk0[t.n]);
    if (launch_kernel(grad_norm_kernel<kCap>, dim3(blocks), dim3(kClipThreads), 0, s, 1, t,
                      part + n_part) != cudaSuccess)
      return MOE_ERR_CUDA;
    n_part += blocks;
    ++launches;
  }
  // the last table first: its tensors were read last.  One launch at least,
  // for the norm.
  for (int i = n ? (n - 1) / kCap * kCap : 0; i >= 0; i -= kCap) {
    if (n > kCap) fill_table(t, g + i, std::min(kCap, n - i));  // else it still holds them
    if (launch_kernel(grad_scale_kernel<kCap>, dim3(clip_blocks(t.chunk0[t.n])),
                      dim3(kClipThreads), 0, s, 1, t, static_cast<const double*>(part), n_part,
                      grad_scale, max_norm, eps, launches == (n + kCap - 1) / kCap ? norm_out
                                                                                    : nullptr) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    ++launches;
  }
  set_last_launch_count(launches);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_clip_workspace_size(int32_t n) {
  if (n < 0 || n > MOE_MAX_GRAD_TENSORS) return 0;
  const int tables = std::max(1, ceil_div(n, kLargeTable));
  return kClipHeader + sizeof(double) * kMaxClipBlocks * static_cast<size_t>(tables);
}

extern "C" int moe_clip_grad_norm(int32_t n, const moe_grad_tensor* tensors, float grad_scale,
                                  float max_norm, float eps, float* norm_out, void* ws,
                                  size_t ws_bytes, void* stream) {
  if (n < 0 || (n > 0 && !tensors) || !norm_out || !ws) return MOE_ERR_INVALID_ARG;
  if (n > MOE_MAX_GRAD_TENSORS) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!(max_norm >= 0.f) || !(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(grad_scale))
    return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0 || (reinterpret_cast<uintptr_t>(norm_out) & 3))
    return MOE_ERR_MISALIGNED;
  if (ws_bytes < moe_clip_workspace_size(n)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    const moe_grad_tensor& g = tensors[i];
    if (g.dtype != MOE_DTYPE_BF16 && g.dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
    if (g.numel < 0 || (g.numel > 0 && !g.grad)) return MOE_ERR_INVALID_ARG;
    const int size = g.dtype == MOE_DTYPE_F32 ? 4 : 2;
    if ((reinterpret_cast<uintptr_t>(g.grad) % size) || (reinterpret_cast<uintptr_t>(g.out) % size))
      return MOE_ERR_MISALIGNED;
    // chunk indices are 32-bit
    if (g.numel > (1LL << 42) || (total += g.numel / (kChunkBytes / 4) + 2) >= (1LL << 30))
      return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  double* part = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + kClipHeader);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return n <= kSmallTable
             ? run_clip<kSmallTable>(n, tensors, grad_scale, max_norm, eps, norm_out, part, s)
         : n <= kMiddleTable
             ? run_clip<kMiddleTable>(n, tensors, grad_scale, max_norm, eps, norm_out, part, s)
             : run_clip<kLargeTable>(n, tensors, grad_scale, max_norm, eps, norm_out, part, s);
}
