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
//   2. rows.  The sorted list is cut into pieces of 8 to 32 tokens, whatever their
//      ids, one group of threads (8 columns a thread) per piece and 2048
//      columns: every group has the same work, however the ids are
//      distributed.  A row whose tokens all lie in the piece is written; the
//      sums of an id that goes on before or behind it go to the workspace in
//      fp32.  Among these blocks are those that fill the rows of ids without
//      a token, run by run (for a large vocabulary most of the bytes): they
//      keep HBM busy while the others wait for their loads.
//   3. join.  Ids of several pieces: the pieces' sums are added in order.
// Two forms of 2 that gave ids to warps or groups took 100 and 142 us at
// T=16384 V=32000 H=4096 bf16 with word frequencies: the latencies of a few
// tokens an id do not overlap.
// HBM bound: T rows read, V rows written.  T=16384 V=32000 H=4096 bf16 with word
// frequencies: 85 us (396 MB; 58 at HBM rate), of which the sort takes 10 and
// the join 10; T=3001 V=50021 H=1001 fp32 45 us (212 MB; 31).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/moe_block.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowwise.cuh"

namespace moe {
namespace {

constexpr int kSteps = 2;           // forward: octets of a row per lane
constexpr int kSlice = 32 * 8 * kSteps;
constexpr int kWarps = 8;           // forward: warps per block
constexpr int kMinPiece = 8, kMaxPiece = 32;  // sorted positions per piece
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
// The ids of a lane's next kSortBatch tokens (32 apart; -1 past the end), all
// under way at once.
constexpr int kSortBatch = 8;
__device__ __forceinline__ void load_ids(int (&id)[kSortBatch], const int32_t* ids, long t,
                                         long end) {
#pragma unroll
  for (int u = 0; u < kSortBatch; ++u) id[u] = t + 32 * u < end ? __ldg(ids + t + 32 * u) : -1;
}

// Block b: ids [b * range, (b + 1) * range).  Warp w takes the tokens
// [w * per, (w + 1) * per) in both scans, so its placements keep token order.
// count [kSortWarps][range] in shared memory.
__global__ void __launch_bounds__(32 * kSortWarps)
embed_sort_kernel(const int32_t* __restrict__ ids, int T, int V, int range,
                  int32_t* __restrict__ order, int32_t* __restrict__ sorted_id,
                  int32_t* __restrict__ start, uint32_t* status) {
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
  for (long tb = t0; tb < t1; tb += 32 * kSortBatch) {
    int id[kSortBatch];
    load_ids(id, ids, tb + lane, t1);
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u) {
      below += id[u] >= 0 && id[u] < v0;
      bad |= id[u] >= V;
      if (id[u] >= v0 && id[u] < v1) atomicAdd(&mine[id[u] - v0], 1);  // integers: any order
    }
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
  for (long tb = t0; tb < t1; tb += 32 * kSortBatch) {  // the whole warp stays together
    int id[kSortBatch];
    load_ids(id, ids, tb + lane, t1);
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u) {
      const bool hit = id[u] >= v0 && id[u] < v1;
      const unsigned hits = __ballot_sync(0xffffffffu, hit);
      if (!hits) continue;
      if (hit) {
        const unsigned same = __match_any_sync(hits, id[u]);
        const int rank = __popc(same & ((1u << lane) - 1));
        const int at = mine[id[u] - v0];
        __syncwarp(hits);
        if (rank == 0) mine[id[u] - v0] = at + __popc(same);
        order[at + rank] = static_cast<int32_t>(tb + 32 * u + lane);
        sorted_id[at + rank] = id[u];
      }
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ rows
constexpr int kRowThreads = 256;
constexpr int kRowCols = kRowThreads * 8;  // columns of a block that is one group

// A group's threads: n of them (32 .. 256), 8 columns each from column c0 on.
struct Group {
  int index, tid, n, c0, cols;
  __device__ __forceinline__ Group(int H, int n_) {
    n = n_;
    index = threadIdx.x / n;
    tid = threadIdx.x - index * n;
    c0 = blockIdx.y * kRowCols;
    cols = min(kRowCols, H - c0);
  }
};

// Tokens in flight per thread (single elements take eight loads a token).
template <typename TO, bool kWide>
__host__ __device__ constexpr int batch_of() { return !kWide ? 2 : sizeof(TO) == 2 ? 8 : 4; }

template <typename T>
__device__ __forceinline__ void add_oct(float (&acc)[8], const Oct<T>& x) {
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] += x.get(j);
}

// Zeros to the n elements from `at` on, by one warp.
template <typename T>
__device__ __forceinline__ void fill_zero(T* at, long n, int lane) {
  constexpr int kPer = 16 / sizeof(T);
  const long lead = min(
      n, static_cast<long>(((16 - (reinterpret_cast<uintptr_t>(at) & 15)) & 15) / sizeof(T)));
  const long vecs = (n - lead) / kPer, tail = lead + vecs * kPer;
  uint4* v = reinterpret_cast<uint4*>(at + lead);
  for (long i = lane; i < vecs; i += 32) v[i] = make_uint4(0, 0, 0, 0);
  if (lane < lead) at[lane] = T{};  // fewer than 8 elements on either side
  if (tail + lane < n) at[tail + lane] = T{};
}

// The rows of the ids [v0, v0 + kFillIds) that have no token, by one warp.
constexpr int kFillIds = 8;
template <typename TT>
__device__ __forceinline__ void fill_rows(const int32_t* start, TT* d_table, long v0, int V, int H,
                                          int lane) {
  const int n = static_cast<int>(max(0L, min(static_cast<long>(kFillIds), V - v0)));
  const bool empty = lane < n && __ldg(start + v0 + lane) == __ldg(start + v0 + lane + 1);
  unsigned mask = __ballot_sync(0xffffffffu, empty);
  while (mask) {
    const int i = __ffs(mask) - 1, len = __ffs(~(mask >> i)) - 1;
    fill_zero(d_table + (v0 + i) * H, static_cast<long>(len) * H, lane);
    mask &= ~(((1u << len) - 1) << i);
  }
}

// Piece q of the sorted list.  Its first id may have begun before it and its
// last may go on behind it: their sums go to the slots 2 q (begun before,
// whether it ends here or not) and 2 q + 1.  Of the grid's columns of
// blocks, piece_blocks take pieces and the others fill.
template <typename TT, typename TO, bool kWide>
__global__ void __launch_bounds__(kRowThreads, 3)
embed_rows_kernel(const int32_t* __restrict__ order, const int32_t* __restrict__ sorted_id,
                  const int32_t* __restrict__ start, const TO* __restrict__ d_out,
                  TT* __restrict__ d_table, float* __restrict__ part, int V, int H, int pieces,
                  int piece, int group_threads, int piece_blocks, float scale) {
  pdl_enter();
  constexpr int kBatch = batch_of<TO, kWide>();
  const int lane = threadIdx.x & 31;
  // the two kinds of blocks in proportion, so that both are under way throughout
  const long pb = static_cast<long>(blockIdx.x) * piece_blocks / gridDim.x;
  if (static_cast<long>(blockIdx.x + 1) * piece_blocks / gridDim.x == pb) {
    const long b = (blockIdx.x - pb) * gridDim.y + blockIdx.y;
    fill_rows(start, d_table, (b * (kRowThreads / 32) + (threadIdx.x >> 5)) * kFillIds, V, H, lane);
    return;
  }
  const Group g(H, group_threads);
  const long q = pb * (kRowThreads / group_threads) + g.index;
  const long total = start[V], p0 = q * piece;
  if (q >= pieces || p0 >= total) return;  // whole warps
  const int m = static_cast<int>(min(static_cast<long>(piece), total - p0));
  const int my_t = lane < m ? __ldg(order + p0 + lane) : 0;
  const int my_v = lane < m ? __ldg(sorted_id + p0 + lane) : -1;
  const int before = p0 > 0 ? __ldg(sorted_id + p0 - 1) : -1;
  const int behind = p0 + m < total ? __ldg(sorted_id + p0 + m) : -1;
  int cur = __shfl_sync(0xffffffffu, my_v, 0);
  bool begun = before == cur;  // the present id began in an earlier piece
  float acc[8] = {};
  auto flush = [&](bool goes_on) {
    if (begun || goes_on) {
      float* dst = part + (2 * q + (begun ? 0 : 1)) * H + g.c0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = oct_col<kWide>(0, j, g.tid, g.n);
        if (c < g.cols) dst[c] = acc[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] *= scale;
      store_oct<kWide>(acc, d_table + static_cast<long>(cur) * H + g.c0, 0, g.tid, g.n, g.cols);
    }
  };
#pragma unroll 1
  for (int i = 0; i < m; i += kBatch) {
    Oct<TO> x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const long t = __shfl_sync(0xffffffffu, my_t, (i + u) & 31);
      if (i + u < m) load_oct<kWide>(x[u], d_out + t * H + g.c0, 0, g.tid, g.n, g.cols);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int v = __shfl_sync(0xffffffffu, my_v, (i + u) & 31);
      if (i + u < m) {
        if (v != cur) {
          flush(false);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = 0.f;
          cur = v;
          begun = false;
        }
        add_oct(acc, x[u]);
      }
    }
  }
  flush(behind == cur);
}

// The id that starts in piece q and goes on behind it, if there is one.  64
// threads take 512 columns; the four of them in a block take a quarter of the
// id's pieces each, so that a frequent id's are not one chain of loads.
constexpr int kJoinCols = 512, kJoinRuns = 4;
template <typename TT, bool kWide>
__global__ void __launch_bounds__(64 * kJoinRuns)
embed_join_kernel(const int32_t* __restrict__ sorted_id, const int32_t* __restrict__ start,
                  const float* __restrict__ part, TT* __restrict__ d_table, int V, int H,
                  int piece, float scale) {
  pdl_enter();
  __shared__ float s_sum[kJoinRuns - 1][8][64];
  const long q = blockIdx.x;
  const int c0 = blockIdx.y * kJoinCols, cols = min(kJoinCols, H - c0);
  const int run = threadIdx.x / 64, tid = threadIdx.x & 63;
  const long total = start[V], p0 = q * piece, p1 = p0 + piece;
  if (p1 >= total) return;
  const long v = __ldg(sorted_id + p1 - 1);
  if (__ldg(sorted_id + p1) != v || (p0 > 0 && __ldg(sorted_id + p0 - 1) == v)) return;
  const long n = (start[v + 1] - 1) / piece - q + 1;  // its pieces
  const long i1 = q + n * (run + 1) / kJoinRuns;
  float acc[8] = {};
#pragma unroll 4
  for (long i = q + n * run / kJoinRuns; i < i1; ++i) {
    Oct<float> x;
    load_oct<kWide>(x, part + (2 * i + (i == q ? 1 : 0)) * H + c0, 0, tid, 64, cols);
    add_oct(acc, x);
  }
  if (run) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s_sum[run - 1][j][tid] = acc[j];
  }
  __syncthreads();
  if (run) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    for (int r = 0; r < kJoinRuns - 1; ++r) acc[j] += s_sum[r][j][tid];
    acc[j] *= scale;
  }
  store_oct<kWide>(acc, d_table + v * H + c0, 0, tid, 64, cols);
}

// ------------------------------------------------------------------ host
int elt(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
bool dtype_ok(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }

int check_embed(const moe_embed_problem* p) {
  if (!p || p->T < 0 || p->V < 1 || p->H < 1) return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(p->table_dtype) || !dtype_ok(p->out_dtype)) return MOE_ERR_INVALID_ARG;
  const long long slices = (p->H + kSlice - 1) / kSlice;
  // a table no GPU holds; block indices of the forward: tokens * slices / 8 warps
  if (p->T > (1 << 28) || p->V > (1 << 28) || p->H > (1 << 20) ||
      static_cast<long long>(p->V) * p->H > (1LL << 42) ||
      p->T * slices / kWarps >= (1LL << 31) - 2)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// A group's threads: 8 columns each, a power of two of warps.
int group_threads(int H) {
  int n = 32;
  while (n < kRowThreads && n * 8 < H) n *= 2;
  return n;
}

// Ids per sort block: as many blocks as SMs while the counters fit.
int sort_range(int V) { return std::min(kMaxRange, std::max(32, ceil_div(V, num_sms()))); }
// Tokens per piece: the most (fewer sums through the workspace) that still
// gives every SM four blocks.  T=3001 H=1001 fp32: rows 20 us with 32.
int piece_of(int T, int H) {
  const int groups = kRowThreads / group_threads(H);
  int piece = kMaxPiece;
  while (piece > kMinPiece && static_cast<long>(ceil_div(T, static_cast<long>(piece) * groups)) *
                                      ceil_div(H, kRowCols) <
                                  4L * num_sms())
    piece /= 2;
  return piece;
}

struct EmbedLayout {
  size_t order, sorted_id, start, part, total;
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
  L.sorted_id = take(sizeof(int32_t) * static_cast<size_t>(p->T));
  L.start = take(sizeof(int32_t) * (static_cast<size_t>(p->V) + 1));
  L.part = take(sizeof(float) * 2 * static_cast<size_t>(ceil_div(p->T, piece_of(p->T, p->H))) * p->H);
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
  int32_t* sorted_id = reinterpret_cast<int32_t*>(base + L.sorted_id);
  int32_t* start = reinterpret_cast<int32_t*>(base + L.start);
  float* part = reinterpret_cast<float*>(base + L.part);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = p->H % 8 == 0 && aligned(d_table, 8 * elt(p->table_dtype)) &&
                    aligned(d_out, 8 * elt(p->out_dtype));
  const int group = group_threads(p->H), piece = piece_of(p->T, p->H);
  const int pieces = ceil_div(p->T, piece);
  const int range = sort_range(p->V);
  const size_t smem = sizeof(int32_t) * kSortWarps * range;
  set_last_launch_count(0);
  int launches = 0;
  const cudaError_t err = by_types(p, wide, [&](auto t, auto o, auto w) {
    using TT = decltype(t);
    using TO = decltype(o);
    constexpr bool kWide = decltype(w)::value;
    cudaError_t e = cudaFuncSetAttribute(
        embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        static_cast<int>(sizeof(int32_t) * kSortWarps * kMaxRange));
    if (e != cudaSuccess) return e;
    e = launch_kernel(embed_sort_kernel, dim3(ceil_div(p->V, range)), dim3(32 * kSortWarps), smem,
                      s, 1, ids, p->T, p->V, range, order, sorted_id, start,
                      static_cast<uint32_t*>(ws));
    if (e != cudaSuccess) return e;
    ++launches;
    const int piece_blocks = ceil_div(pieces, kRowThreads / group);
    const int col_blocks = ceil_div(p->H, kRowCols);
    const int fill_blocks = ceil_div(p->V, static_cast<long>(kRowThreads / 32 * kFillIds));
    e = launch_kernel(embed_rows_kernel<TT, TO, kWide>,
                      dim3(piece_blocks + ceil_div(fill_blocks, col_blocks), col_blocks),
                      dim3(kRowThreads), 0, s, 1, static_cast<const int32_t*>(order),
                      static_cast<const int32_t*>(sorted_id), static_cast<const int32_t*>(start),
                      static_cast<const TO*>(d_out), static_cast<TT*>(d_table), part, p->V, p->H,
                      pieces, piece, group, piece_blocks, p->scale);
    if (e != cudaSuccess) return e;
    ++launches;
    if (pieces <= 1) return e;  // nothing goes on into another piece
    ++launches;
    return launch_kernel(embed_join_kernel<TT, kWide>, dim3(pieces, ceil_div(p->H, kJoinCols)),
                         dim3(64 * kJoinRuns), 0, s, 1, static_cast<const int32_t*>(sorted_id),
                         static_cast<const int32_t*>(start), static_cast<const float*>(part),
                         static_cast<TT*>(d_table), p->V, p->H, piece, p->scale);
  });
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  set_last_launch_count(launches);
  return MOE_OK;
}
