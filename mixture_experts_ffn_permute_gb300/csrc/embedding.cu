// Token embedding and its gradient (moe_embedding_* of include/moe_block.h).
//
// Forward: a gather of rows, one warp per 512 columns of a token's row.
//
// Backward: d_table[v] is a sum over the tokens of id v, taken in token order,
// in three launches:
//   1. sort.  Every block owns a range of the vocabulary and scans all T ids
//      (4 T bytes from L2) in token order: it counts the ids below its range
//      (the base of its part of the sorted list) and those inside, per warp
//      and id, then places its tokens by a second scan.  A stable counting
//      sort without a global histogram or any pass over another block's
//      counts.
//   2. rows.  One warp per (id, 512 columns) sums the id's tokens and writes
//      the row: zeros where there is none, which for a large vocabulary is
//      most of the bytes.  Ids with more than 64 tokens ("heavy") are left
//      out here; their runs are cut at multiples of 64 sorted positions and
//      each piece is one warp's item, so that a frequent token does not keep
//      one warp busy.  The pieces' fp32 sums go to the workspace.
//   3. join.  Heavy ids: the pieces are added in order.
// HBM bound: T rows read, V rows written.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/moe_block.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowwise.cuh"

namespace moe {
namespace {

constexpr int kSteps = 2;           // octets of a row per lane
constexpr int kSlice = 32 * 8 * kSteps;
constexpr int kWarps = 8;           // per block of the row kernels
constexpr int kPiece = 64;          // tokens of a heavy id per item
constexpr int kSortWarps = 32;
constexpr int kMaxRange = 1024;     // ids per sort block (counters in shared memory)
constexpr size_t kEmbedHeader = 256;

// ------------------------------------------------------------------ forward
template <typename TT, typename TO, bool kWide>
__global__ void __launch_bounds__(32 * kWarps)
embed_fwd_kernel(const int32_t* __restrict__ ids, const TT* __restrict__ table,
                 TO* __restrict__ out, int T, int V, int H, int slices, float scale,
                 uint32_t* status) {
  pdl_enter();
  const long item = static_cast<long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long t = item / slices;
  const int slice = static_cast<int>(item - t * slices);
  if (t >= T) return;
  const int id = ids[t];
  const bool ok = id >= 0 && id < V;
  if (id >= V && slice == 0 && lane == 0) record_status(status, kStatusIndex);
  const int c0 = slice * kSlice, n = min(kSlice, H - c0);
  const TT* src = table + static_cast<long>(ok ? id : 0) * H + c0;
  TO* dst = out + t * H + c0;
  Oct<TT> x[kSteps];
#pragma unroll
  for (int v = 0; v < kSteps; ++v)
    if (ok) load_oct<kWide>(x[v], src, v, lane, 32, n);
#pragma unroll
  for (int v = 0; v < kSteps; ++v) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = ok ? scale * x[v].get(j) : 0.f;
    store_oct<kWide>(y, dst, v, lane, 32, n);
  }
}

// ------------------------------------------------------------------ sort
// Block b: ids [b * range, (b + 1) * range).  Warp w takes the tokens
// [w * per, (w + 1) * per) in both scans, so its placements keep token order.
// count [kSortWarps][range] in shared memory.
__global__ void __launch_bounds__(32 * kSortWarps)
embed_sort_kernel(const int32_t* __restrict__ ids, int T, int V, int range,
                  int32_t* __restrict__ order, int32_t* __restrict__ start, uint32_t* status) {
  pdl_enter();
  extern __shared__ int32_t s_count[];
  __shared__ int32_t s_warp[kSortWarps];
  __shared__ int32_t s_below[kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int v0 = blockIdx.x * range, v1 = min(V, v0 + range), nv = v1 - v0;
  for (int i = threadIdx.x; i < kSortWarps * range; i += 32 * kSortWarps) s_count[i] = 0;
  __syncthreads();
  const int per = ((T + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const long t0 = min(static_cast<long>(T), static_cast<long>(warp) * per);
  const long t1 = min(static_cast<long>(T), t0 + per);
  int32_t* mine = s_count + warp * range;
  int below = 0;
  bool bad = false;
#pragma unroll 4
  for (long t = t0 + lane; t < t1; t += 32) {
    const int id = __ldg(ids + t);
    below += id >= 0 && id < v0;
    bad |= id >= V;
    if (id >= v0 && id < v1) atomicAdd(&mine[id - v0], 1);  // integers: any order
  }
  if (blockIdx.x == 0 && bad) record_status(status, kStatusIndex);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
  if (lane == 0) s_below[warp] = below;
  __syncthreads();
  // thread v: total of its id, exclusive scan over the ids, then over the warps
  int total = 0;
  if (threadIdx.x < nv)
    for (int w = 0; w < kSortWarps; ++w) total += s_count[w * range + threadIdx.x];
  int incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int base = incl - total;
  for (int w = 0; w < kSortWarps; ++w) {
    base += s_below[w];
    if (w < warp) base += s_warp[w];
  }
  if (threadIdx.x < nv) {
    start[v0 + threadIdx.x] = base;
    if (v0 + static_cast<int>(threadIdx.x) == V - 1) start[V] = base + total;
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = s_count[w * range + threadIdx.x];
      s_count[w * range + threadIdx.x] = base;
      base += c;
    }
  }
  __syncthreads();
  for (long tb = t0; tb < t1; tb += 32) {  // the whole warp stays together
    const long t = tb + lane;
    const int id = t < t1 ? __ldg(ids + t) : -1;
    const bool hit = id >= v0 && id < v1;
    const unsigned hits = __ballot_sync(0xffffffffu, hit);
    if (!hits) continue;
    if (hit) {
      const unsigned same = __match_any_sync(hits, id);
      const int rank = __popc(same & ((1u << lane) - 1));
      const int at = mine[id - v0];
      __syncwarp(hits);
      if (rank == 0) mine[id - v0] = at + __popc(same);
      order[at + rank] = static_cast<int32_t>(t);
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------------ rows
// Adds the rows of the sorted positions [p0, p1) to acc, in order.
template <typename TO, bool kWide>
__device__ __forceinline__ void sum_tokens(float (&acc)[kSteps][8], const int32_t* order, long p0,
                                           long p1, const TO* d_out, int H, int c0, int n,
                                           int lane) {
  for (long p = p0; p < p1; p += 32) {
    const int m = static_cast<int>(min(32L, p1 - p));
    const int mine = lane < m ? order[p + lane] : 0;
#pragma unroll 4
    for (int i = 0; i < m; ++i) {
      const long t = __shfl_sync(0xffffffffu, mine, i);
      const TO* row = d_out + t * H + c0;
      Oct<TO> x[kSteps];
#pragma unroll
      for (int v = 0; v < kSteps; ++v) load_oct<kWide>(x[v], row, v, lane, 32, n);
#pragma unroll
      for (int v = 0; v < kSteps; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[v][j] += x[v].get(j);
    }
  }
}

// Items [0, pieces * slices): pieces of heavy ids; then V * slices rows.
template <typename TT, typename TO, bool kWide>
__global__ void __launch_bounds__(32 * kWarps)
embed_rows_kernel(const int32_t* __restrict__ ids, const int32_t* __restrict__ order,
                  const int32_t* __restrict__ start, const TO* __restrict__ d_out,
                  TT* __restrict__ d_table, float* __restrict__ part, int V, int H, int pieces,
                  int slices, float scale) {
  pdl_enter();
  long item = static_cast<long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long q = item / slices;
  const int c0 = static_cast<int>(item - q * slices) * kSlice, n = min(kSlice, H - c0);
  if (q < pieces) {
    // the piece [64 q, 64 q + 64) of the sorted positions touches at most two
    // heavy ids: the one at its first position (sum in slot 2 q) and another
    // that starts inside and goes on beyond its end (slot 2 q + 1)
    const long total = start[V], p0 = q * kPiece, p1 = min(total, p0 + kPiece);
    if (p0 >= total) return;
    const int va = ids[order[p0]], vb = ids[order[p1 - 1]];
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const int v = h ? vb : va;
      if (h && vb == va) break;
      const long s0 = start[v], s1 = start[v + 1];
      if (s1 - s0 <= kPiece) continue;
      float acc[kSteps][8] = {};
      sum_tokens<TO, kWide>(acc, order, max(s0, p0), min(s1, p1), d_out, H, c0, n, lane);
      float* dst = part + (2 * q + h) * H + c0;
#pragma unroll
      for (int u = 0; u < kSteps; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = oct_col<kWide>(u, j, lane, 32);
          if (c < n) dst[c] = acc[u][j];
        }
    }
    return;
  }
  const long v = q - pieces;
  if (v >= V) return;
  const long s0 = start[v], s1 = start[v + 1];
  if (s1 - s0 > kPiece) return;
  float acc[kSteps][8] = {};
  sum_tokens<TO, kWide>(acc, order, s0, s1, d_out, H, c0, n, lane);
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[u][j] *= scale;
    store_oct<kWide>(acc[u], d_table + v * H + c0, u, lane, 32, n);
  }
}

// Piece q: the heavy id that starts in it, if any (there is at most one).
template <typename TT, bool kWide>
__global__ void __launch_bounds__(32 * kWarps)
embed_join_kernel(const int32_t* __restrict__ ids, const int32_t* __restrict__ order,
                  const int32_t* __restrict__ start, const float* __restrict__ part,
                  TT* __restrict__ d_table, int V, int H, int pieces, int slices, float scale) {
  pdl_enter();
  const long item = static_cast<long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long q = item / slices;
  const int c0 = static_cast<int>(item - q * slices) * kSlice, n = min(kSlice, H - c0);
  if (q >= pieces) return;
  const long total = start[V], p0 = q * kPiece, p1 = min(total, p0 + kPiece);
  if (p0 >= total) return;
  const long v = ids[order[p1 - 1]];
  const long s0 = start[v], s1 = start[v + 1];
  if (s1 - s0 <= kPiece || s0 < p0) return;
  float acc[kSteps][8] = {};
#pragma unroll 4
  for (long i = q; i * kPiece < s1; ++i) {
    // in its first piece the id is at the first position, or it starts inside
    const float* src = part + (2 * i + (i == q && s0 > p0 ? 1 : 0)) * H + c0;
    Oct<float> x[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) load_oct<kWide>(x[u], src, u, lane, 32, n);
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[u][j] += x[u].get(j);
  }
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[u][j] *= scale;
    store_oct<kWide>(acc[u], d_table + v * H + c0, u, lane, 32, n);
  }
}

// ------------------------------------------------------------------ host
int elt(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
bool dtype_ok(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }

int check_embed(const moe_embed_problem* p) {
  if (!p || p->T < 0 || p->V < 1 || p->H < 1) return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(p->table_dtype) || !dtype_ok(p->out_dtype)) return MOE_ERR_INVALID_ARG;
  const long long slices = (p->H + kSlice - 1) / kSlice;
  // block indices: (rows + pieces) * slices / 8 warps
  if (p->T > (1 << 28) || p->V > (1 << 28) || p->H > (1 << 20) ||
      (static_cast<long long>(p->V) + p->T) * slices / kWarps >= (1LL << 31) - 2)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// Ids per sort block: as many blocks as SMs while the counters fit.
int sort_range(int V) { return std::min(kMaxRange, std::max(32, ceil_div(V, num_sms()))); }
int pieces_of(int T) { return ceil_div(T, kPiece); }

struct EmbedLayout {
  size_t order, start, part, total;
};
EmbedLayout embed_layout(const moe_embed_problem* p) {
  EmbedLayout L;
  size_t o = kEmbedHeader;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  L.order = take(sizeof(int32_t) * static_cast<size_t>(p->T));
  L.start = take(sizeof(int32_t) * (static_cast<size_t>(p->V) + 1));
  L.part = take(sizeof(float) * 2 * static_cast<size_t>(pieces_of(p->T)) * p->H);
  L.total = o;
  return L;
}

bool aligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

unsigned blocks_of(long items) { return static_cast<unsigned>((items + kWarps - 1) / kWarps); }

template <typename F>
cudaError_t by_types(const moe_embed_problem* p, bool wide, F&& f) {
  auto go = [&](auto t, auto o) {
    return wide ? f(t, o, std::true_type{}) : f(t, o, std::false_type{});
  };
  const bool tb = p->table_dtype == MOE_DTYPE_BF16, ob = p->out_dtype == MOE_DTYPE_BF16;
  if (tb) return ob ? go(Bf16{}, Bf16{}) : go(Bf16{}, float{});
  return ob ? go(float{}, Bf16{}) : go(float{}, float{});
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_embedding_forward(const moe_embed_problem* p, const int32_t* ids,
                                     const void* table, void* out, void* ws, void* stream) {
  const int rc = check_embed(p);
  if (rc != MOE_OK) return rc;
  set_last_launch_count(0);
  if (p->T == 0) return MOE_OK;
  if (!ids || !table || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned(ids, 4) || !aligned(table, elt(p->table_dtype)) ||
      !aligned(out, elt(p->out_dtype)) || !aligned(ws, 256))
    return MOE_ERR_MISALIGNED;
  const bool wide = p->H % 8 == 0 && aligned(table, 8 * elt(p->table_dtype)) &&
                    aligned(out, 8 * elt(p->out_dtype));
  const int slices = ceil_div(p->H, kSlice);
  const cudaError_t err = by_types(p, wide, [&](auto t, auto o, auto w) {
    using TT = decltype(t);
    using TO = decltype(o);
    return launch_kernel(embed_fwd_kernel<TT, TO, decltype(w)::value>,
                         dim3(blocks_of(static_cast<long>(p->T) * slices)), dim3(32 * kWarps), 0,
                         static_cast<cudaStream_t>(stream), 1, ids, static_cast<const TT*>(table),
                         static_cast<TO*>(out), p->T, p->V, p->H, slices, p->scale,
                         static_cast<uint32_t*>(ws));
  });
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  set_last_launch_count(1);
  return MOE_OK;
}

extern "C" size_t moe_embedding_workspace_size(const moe_embed_problem* p) {
  return check_embed(p) == MOE_OK ? embed_layout(p).total : 0;
}

extern "C" int moe_embedding_backward(const moe_embed_problem* p, const int32_t* ids,
                                      const void* d_out, void* d_table, void* ws, size_t ws_bytes,
                                      void* stream) {
  const int rc = check_embed(p);
  if (rc != MOE_OK) return rc;
  if (!d_table || !ws || (p->T > 0 && (!ids || !d_out))) return MOE_ERR_INVALID_ARG;
  if (!aligned(ids, 4) || !aligned(d_table, elt(p->table_dtype)) ||
      !aligned(d_out, elt(p->out_dtype)) || !aligned(ws, 256))
    return MOE_ERR_MISALIGNED;
  const EmbedLayout L = embed_layout(p);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* base = static_cast<uint8_t*>(ws);
  int32_t* order = reinterpret_cast<int32_t*>(base + L.order);
  int32_t* start = reinterpret_cast<int32_t*>(base + L.start);
  float* part = reinterpret_cast<float*>(base + L.part);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = p->H % 8 == 0 && aligned(d_table, 8 * elt(p->table_dtype)) &&
                    aligned(d_out, 8 * elt(p->out_dtype));
  const int slices = ceil_div(p->H, kSlice), pieces = pieces_of(p->T);
  const int range = sort_range(p->V);
  const size_t smem = sizeof(int32_t) * kSortWarps * range;
  set_last_launch_count(0);
  if (cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(sizeof(int32_t) * kSortWarps * kMaxRange)) !=
          cudaSuccess ||
      launch_kernel(embed_sort_kernel, dim3(ceil_div(p->V, range)), dim3(32 * kSortWarps), smem, s,
                    1, ids, p->T, p->V, range, order, start, static_cast<uint32_t*>(ws)) !=
          cudaSuccess)
    return MOE_ERR_CUDA;
  int launches = 1;
  const cudaError_t err = by_types(p, wide, [&](auto t, auto o, auto w) {
    using TT = decltype(t);
    using TO = decltype(o);
    constexpr bool kWide = decltype(w)::value;
    cudaError_t e = launch_kernel(
        embed_rows_kernel<TT, TO, kWide>,
        dim3(blocks_of((static_cast<long>(p->V) + pieces) * slices)), dim3(32 * kWarps), 0, s, 1,
        ids, static_cast<const int32_t*>(order), static_cast<const int32_t*>(start),
        static_cast<const TO*>(d_out), static_cast<TT*>(d_table), part, p->V, p->H, pieces, slices,
        p->scale);
    if (e != cudaSuccess) return e;
    ++launches;
    if (pieces < 2) return e;  // an id has more than 64 tokens only if there are more
    ++launches;
    return launch_kernel(embed_join_kernel<TT, kWide>,
                         dim3(blocks_of(static_cast<long>(pieces) * slices)), dim3(32 * kWarps), 0,
                         s, 1, ids, static_cast<const int32_t*>(order),
                         static_cast<const int32_t*>(start), static_cast<const float*>(part),
                         static_cast<TT*>(d_table), p->V, p->H, pieces, slices, p->scale);
  });
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  set_last_launch_count(launches);
  return MOE_OK;
}
