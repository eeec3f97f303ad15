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
// For few bytes the launches' latencies count: the second kernel reads its first
// chunk before it waits for the first kernel (the gradients were complete
// before that one began), and a chunk's tensor is found by a hint.  150 tensors
// of 5 MB take 6.9 us in a captured graph; with a binary search over the table,
// whose dependent misses in the constant cache cost most, no early read and
// fp64 in every thread they took 14.3.  1.2 GB of bf16 gradients take 0.55 ms:
// the norm at 6.9 TB/s, the scaling (read and write) at 6.5.
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
constexpr int kClipVecs = kChunkBytes / 16 / kClipThreads;  // per thread and chunk, all in flight
constexpr int kClipBlocksPerSm = 8;  // 2048 threads
constexpr int kMaxClipBlocks = 2048; // per launch; bounds the workspace
constexpr size_t kClipHeader = 256;
// Tables by capacity: parameters are copied with every launch, so a short list
// takes a short table.
constexpr int kSmallTable = 64, kMiddleTable = 256, kLargeTable = 1024;

constexpr int kHints = 256;
template <int kCap>
struct GradTable {
  int n;
  int hint_shift;
  uint16_t hint[kHints];  // the tensor of chunk i << hint_shift
  int chunk0[kCap + 1];   // first chunk of each tensor
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
  int lo = t.hint[c >> t.hint_shift];  // at or before the last tensor whose first chunk is <= c
  while (t.chunk0[lo + 1] <= c) ++lo;
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

// 0 exactly if every element is a zero of either sign.
template <bool kF32>
__device__ __forceinline__ uint32_t magnitude16(uint4 v) {
  return (v.x | v.y | v.z | v.w) & (kF32 ? 0x7fffffffu : 0x7fff7fffu);
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

// What a thread takes of a chunk: every kClipThreads-th 16-byte vector behind
// the leading elements, and one of the few elements round the vectors.
struct Part {
  uint4 x[kClipVecs];
  int vecs;    // of the chunk
  int single;  // index of the element, or -1
  __device__ __forceinline__ void load(const Chunk& c) {
    const int size = c.f32 ? 4 : 2, per = 16 / size;
    vecs = static_cast<int>((c.n - c.lead) / per);
    const uint4* v = reinterpret_cast<const uint4*>(c.grad + static_cast<long>(c.lead) * size);
#pragma unroll
    for (int u = 0; u < kClipVecs; ++u) {
      const int i = u * kClipThreads + threadIdx.x;
      if (i < vecs) x[u] = v[i];
    }
    const int tail = c.lead + vecs * per + static_cast<int>(threadIdx.x) - 32;
    single = static_cast<int>(threadIdx.x) < c.lead       ? static_cast<int>(threadIdx.x)
             : threadIdx.x >= 32 && tail < c.n ? tail
                                               : -1;
  }
};

// This thread's part of a chunk's sum of squares.
template <bool kF32>
__device__ __forceinline__ double part_squares(const Chunk& c, const Part& p) {
  using T = typename std::conditional<kF32, float, Bf16>::type;
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < kClipVecs; ++u)
    if (u * kClipThreads + static_cast<int>(threadIdx.x) < p.vecs) s += square16<kF32>(p.x[u]);
  const float e = p.single >= 0 ? to_float(reinterpret_cast<const T*>(c.grad)[p.single]) : 0.f;
  s = fmaf(e, e, s);
  if (s == 0.f) {  // zeros, or squares that are all below fp32's smallest number
    uint32_t bits = __float_as_uint(e) << 1;
#pragma unroll
    for (int u = 0; u < kClipVecs; ++u)
      if (u * kClipThreads + static_cast<int>(threadIdx.x) < p.vecs)
        bits |= magnitude16<kF32>(p.x[u]);
    if (bits == 0) return 0.;
  } else if (s >= 0x1p-80f && s < __int_as_float(0x7f800000)) {
    return s;
  }
  double d = static_cast<double>(e) * e;  // out of fp32's comfortable range: again in fp64
#pragma unroll 1
  for (int i = threadIdx.x; i < p.vecs; i += kClipThreads)
    d += square16_f64<kF32>(reinterpret_cast<const uint4*>(
        c.grad + static_cast<long>(c.lead) * sizeof(T))[i]);
  return d;
}

// The block's sum, in thread 0 (fp64 is slow here: no thread does more of it
// than it has to).
__device__ __forceinline__ double block_sum(double x, double* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x < 32) {
    x = threadIdx.x < kClipThreads / 32 ? s[threadIdx.x] : 0.;
#pragma unroll
    for (int o = kClipThreads / 64; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  }
  return x;
}

template <int kCap>
__global__ void __launch_bounds__(kClipThreads)
grad_norm_kernel(const __grid_constant__ GradTable<kCap> t, double* __restrict__ part) {
  __shared__ double s[kClipThreads / 32];
  const int chunks = t.chunk0[t.n];
  double sum = 0.;
  int c = blockIdx.x;
  Chunk k;
  if (c < chunks) k = chunk_at(t, c);  // parameters only
  pdl_enter();
  for (; c < chunks; c += gridDim.x) {
    if (c != static_cast<int>(blockIdx.x)) k = chunk_at(t, c);
    Part x;
    x.load(k);
    sum += k.f32 ? part_squares<true>(k, x) : part_squares<false>(k, x);
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
__device__ __forceinline__ void part_scale(const Chunk& c, const Part& p, float f) {
  using T = typename std::conditional<kF32, float, Bf16>::type;
  const T* g = reinterpret_cast<const T*>(c.grad);
  T* o = reinterpret_cast<T*>(c.out);
  if (((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(o)) & 15) != 0) {
    // the output's boundaries lie elsewhere: element by element
    for (long i = threadIdx.x; i < c.n; i += kClipThreads) from_float(o[i], to_float(g[i]) * f);
    return;
  }
  uint4* w = reinterpret_cast<uint4*>(o + c.lead);
#pragma unroll
  for (int u = 0; u < kClipVecs; ++u) {
    const int i = u * kClipThreads + threadIdx.x;
    if (i < p.vecs) __stcs(w + i, scale16<kF32>(p.x[u], f));
  }
  if (p.single >= 0) from_float(o[p.single], to_float(g[p.single]) * f);
}

template <int kCap>
__global__ void __launch_bounds__(kClipThreads)
grad_scale_kernel(const __grid_constant__ GradTable<kCap> t, const double* __restrict__ part,
                  int n_part, float grad_scale, float max_norm, float eps, float* norm_out) {
  __shared__ double s[kClipThreads / 32];
  __shared__ float s_factor;
  const int chunks = t.chunk0[t.n];
  int c = chunks - 1 - static_cast<int>(blockIdx.x);
  Chunk k;
  Part x;
  // The first chunk ahead of the wait: the kernel before this one only read
  // the gradients, and began when whatever wrote them was complete.
  if (c >= 0) {
    k = chunk_at(t, c);
    x.load(k);
  }
  pdl_enter();
  double sum = 0.;
  for (int i = threadIdx.x; i < n_part; i += kClipThreads) sum += part[i];
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) {
    const float norm = static_cast<float>(fabs(static_cast<double>(grad_scale)) * sqrt(sum));
    float coef = max_norm / (norm + eps);
    // a NaN stays, unless there is no limit
    if (coef >= 1.f || max_norm == __int_as_float(0x7f800000)) coef = 1.f;
    if (norm_out && blockIdx.x == 0) {
      norm_out[0] = norm;
      norm_out[1] = coef;
    }
    s_factor = grad_scale * coef;
  }
  __syncthreads();
  const float f = s_factor;
  while (c >= 0) {
    if (k.out && !(f == 1.f && k.out == k.grad)) {
      if (k.f32) part_scale<true>(k, x, f);
      else part_scale<false>(k, x, f);
    }
    c -= gridDim.x;
    if (c >= 0) {
      k = chunk_at(t, c);
      x.load(k);
    }
  }
}

// Fills the table with tensors[0 .. n).
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
  t.hint_shift = 0;
  while ((chunks >> t.hint_shift) >= kHints) ++t.hint_shift;
  int owner = 0;
  for (int i = 0; i < kHints; ++i) {
    const long c = static_cast<long>(i) << t.hint_shift;
    if (c >= chunks) break;
    while (t.chunk0[owner + 1] <= c) ++owner;
    t.hint[i] = static_cast<uint16_t>(owner);
  }
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
