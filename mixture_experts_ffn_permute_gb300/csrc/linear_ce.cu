// Softmax cross entropy of a linear layer, z = scale x W^T, on the sm_103a
// tensor cores, without keeping the logits (moe_linear_ce_* of
// include/moe_block.h).
//
// Forward.  One persistent GEMM over (256 tokens x N vocabulary rows) tiles of
// CTA pairs (tcgen05.mma.cta_group::2, fp32 accumulators in TMEM) whose
// epilogue keeps, per token and tile, the running maximum and the sum of
// exponentials (log2 units) and picks out the label's logit; a small kernel
// joins a token's tiles in order.  Per token and vocabulary tile 8 bytes leave
// the kernel instead of 2 N of logits.
//
// Backward, in pieces of the vocabulary whose logit gradients (bf16) fit in
// L2:
//   G  = a exp(z - lse) - b [v = label]  the forward's GEMM with another
//                                        epilogue, [T, piece] to the workspace
//   dx += G W_piece    A = G K-major, B = W_piece read MN-major (as stored)
//   dW_piece = G^T x   A = G, B = x, both read MN-major (as stored)
// with a = scale (d_loss + d_lse), b = scale d_loss.  The two products are
// tiles of one launch.  dx is kept in fp32 in the workspace from piece to
// piece (each element is one thread's in every piece, so the order of its sum
// is fixed) and rounded once by the last; with one piece it is written
// directly.
//
// Warp roles (192 threads, one CTA per SM, tiles round-robin over the pairs):
//   warp 0     TMA producer: 6 stages of 16 KB of A and up to 16 KB of B per CTA
//   warp 1     TMEM allocation, MMA issue (the leader CTA's)
//   warps 2-5  epilogue, thread = token (or vocabulary) row of the tile; two
//              accumulators of 256 columns, so it overlaps the next mainloop;
//              bf16 tiles leave through swizzled staging and bulk-tensor stores
// Every wait is bounded (ptx.cuh).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_block.h"
#include "internal.h"
#include "pair_tiles.cuh"
#include "ptx.cuh"
#include "rowwise.cuh"

namespace moe {
namespace {

constexpr int kTileM = 256;  // rows of a pair tile, 128 per CTA
constexpr int kTileN = 256;  // columns at most
constexpr int kTileK = 64;
constexpr int kStagesCe = 6;
constexpr uint32_t kABytesCe = 128 * kTileK * 2;     // 16 KB
constexpr uint32_t kBBytesCe = kTileN / 2 * kTileK * 2;
constexpr uint32_t kStageCe = kABytesCe + kBBytesCe;
constexpr uint32_t kBoxCe = 64 * 64 * 2;             // MN-major box: 64 columns x 64 rows
constexpr uint32_t kStagingBox = 32 * 128;           // 32 rows x 64 bf16
constexpr int kStagingBuffers = 2;
constexpr uint32_t kStagingCe = 4 * kStagingBuffers * kStagingBox;
constexpr size_t kSmemCe = 1024 + kStagesCe * kStageCe + kStagingCe + 256;
static_assert(kSmemCe <= 232448, "shared memory budget");
constexpr int kGroupM = 8;  // m-tiles whose sweep over the n-tiles shares B tiles in L2
constexpr int kThreadsCe = 192;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One GEMM: C[M, N] = A B^T over K, by pair tiles.
struct Gemm {
  int m_tiles, n_tiles, ksteps;
  int n_step;                 // columns per tile (a multiple of 32, <= 256)
  int M, N;                   // extents (rows and columns beyond are not written)
  bool a_mn, b_mn;            // operand stored [K, M] (resp. [K, N]): read MN-major
  bool add, keep;             // fp32 accumulation over launches: add acc, keep it in acc
  __host__ __device__ int tiles() const { return m_tiles * n_tiles; }
};

enum class CeMode : int { kLse = 0, kGrad = 1, kProducts = 2 };

struct CeParams {
  Gemm g[2];            // kProducts: dx then dW; otherwise g[0]
  const int32_t* labels;
  int v0, V;            // first vocabulary row of the piece; vocabulary
  float scale;
  float2* part;         // kLse: [n_tiles][T] (max, sum) in log2 units
  float* label_logit;   // kLse: [T]
  const float* lse;     // kGrad
  const float* d_loss;
  const float* d_lse;   // or NULL
  float* acc;           // kProducts: dx in fp32 [T, N]
  uint32_t* status;
};

struct CeMaps {
  CUtensorMap a, b, out;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Descriptor of an MN-major operand: boxes of 64 columns x 64 K rows with the
// 128-byte swizzle; leading offset = the next 64 columns (one box), stride
// offset = 8 K rows.
__device__ __forceinline__ uint64_t mn_desc(uint32_t smem_addr) {
  return sw128_kmajor_desc(smem_addr) ^ (static_cast<uint64_t>(1u) << 16) ^
         (static_cast<uint64_t>(kBoxCe >> 4) << 16);
}

__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Tile `i` of a GEMM: groups of kGroupM m-tiles sweep the n-tiles.
__device__ __forceinline__ void tile_of(const Gemm& g, int i, int& m, int& n) {
  const int per = kGroupM * g.n_tiles;
  const int grp = i / per, within = i - grp * per;
  const int size = min(kGroupM, g.m_tiles - grp * kGroupM);
  n = within / size;
  m = grp * kGroupM + (within - n * size);
}

template <CeMode kMode>
__global__ void __launch_bounds__(kThreadsCe, 1)
linear_ce_kernel(const __grid_constant__ CeMaps m0, const __grid_constant__ CeMaps m1,
                 const __grid_constant__ CeParams p) {
  pdl_enter();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sA = smem;
  uint8_t* sB = sA + kStagesCe * kABytesCe;
  uint8_t* s_out = sB + kStagesCe * kBBytesCe;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_out + kStagingCe);
  uint64_t* empty = full + kStagesCe;
  uint64_t* tfull = empty + kStagesCe;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStagesCe; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * 128);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&m0.a);
    prefetch_tensormap(&m0.b);
  }
  if (warp == 1) pair::tmem_alloc2<512>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before anything signals them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int tiles0 = p.g[0].tiles();
  const int total = tiles0 + (kMode == CeMode::kProducts ? p.g[1].tiles() : 0);
  const int first = static_cast<int>(blockIdx.x >> 1), stride = static_cast<int>(gridDim.x >> 1);
  auto second = [&](int tile) { return kMode == CeMode::kProducts && tile >= tiles0; };

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      for (int tile = first; tile < total; tile += stride) {
        if (*abort_flag) break;
        const bool two = second(tile);
        const Gemm& g = p.g[two];
        const CeMaps& maps = two ? m1 : m0;
        int m, n;
        tile_of(g, two ? tile - tiles0 : tile, m, n);
        const int row0 = m * kTileM + static_cast<int>(rank) * 128;
        const int half = g.n_step / 2;
        const int col0 = n * g.n_step + static_cast<int>(rank) * half;
        const uint32_t bytes = 2 * (kABytesCe + static_cast<uint32_t>(half) * kTileK * 2);
        bool ok = true;
        for (int kb = 0; kb < g.ksteps; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, p.status)) { ok = false; break; }
          if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
          const uint32_t bar = pair::mapa(smem_u32(&full[stage]), 0);
          uint8_t* a = sA + stage * kABytesCe;
          uint8_t* b = sB + stage * kBBytesCe;
          const int k0 = kb * kTileK;
          if (g.a_mn) {
            pair::tma_load(a, &maps.a, row0, k0, bar, pol);
            pair::tma_load(a + kBoxCe, &maps.a, row0 + 64, k0, bar, pol);
          } else {
            pair::tma_load(a, &maps.a, k0, row0, bar, pol);
          }
          if (g.b_mn) {  // 128 columns: n_step is 256
            pair::tma_load(b, &maps.b, col0, k0, bar, pol);
            pair::tma_load(b + kBoxCe, &maps.b, col0 + 64, k0, bar, pol);
          } else {
            pair::tma_load(b, &maps.b, k0, col0, bar, pol);
          }
          ++issued;
          if (++stage == kStagesCe) { stage = 0; phase ^= 1; }
        }
        if (!ok) { *abort_flag = 1; break; }
      }
      // no bulk copy left in flight: the last fill of every stage has landed
      // (a pair's copies complete on the leader's barriers; the final cluster
      // barrier keeps the peer's shared memory until then)
      for (int i = 1; leader && i <= kStagesCe && i <= issued; ++i) {
        int s = stage - i;
        uint32_t ph = phase;
        if (s < 0) { s += kStagesCe; ph ^= 1; }
        mbar_wait(&full[s], ph, p.status);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (leader && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;
      for (int tile = first; tile < total; tile += stride, ++local) {
        if (*abort_flag) break;
        const bool two = second(tile);
        const Gemm& g = p.g[two];
        const bool a_mn = g.a_mn, b_mn = g.b_mn;
        const int ksteps = g.ksteps;
        const uint32_t idesc = idesc_bf16_f32(kTileM, static_cast<uint32_t>(g.n_step)) |
                               (static_cast<uint32_t>(a_mn) << 15) |
                               (static_cast<uint32_t>(b_mn) << 16);
        const int buf = local & 1;
        const uint32_t tph = (local >> 1) & 1;
        if (!mbar_wait(&tempty[buf], tph ^ 1, p.status)) { *abort_flag = 1; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + buf * kTileN;
        bool ok = true;
        for (int kb = 0; kb < ksteps; ++kb) {
          if (!mbar_wait(&full[stage], phase, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a = smem_u32(sA + stage * kABytesCe);
          const uint32_t b = smem_u32(sB + stage * kBBytesCe);
          // a K=16 step is 32 bytes along a K-major row, 16 rows of 128 bytes
          // of an MN-major box
          const uint64_t ad = a_mn ? mn_desc(a) : sw128_kmajor_desc(a);
          const uint64_t bd = b_mn ? mn_desc(b) : sw128_kmajor_desc(b);
          const uint32_t as = a_mn ? 128 : 2, bs = b_mn ? 128 : 2;  // in 16 bytes
#pragma unroll
          for (int kk = 0; kk < kTileK / 16; ++kk)
            pair::mma(d_tmem, ad + kk * as, bd + kk * bs, idesc, (kb | kk) != 0);
          pair::commit_both(&empty[stage]);
          if (++stage == kStagesCe) { stage = 0; phase ^= 1; }
        }
        if (!ok) { *abort_flag = 1; break; }
        pair::commit_both(&tfull[buf]);
      }
      pair::commit_local(drain);  // every MMA done before TMEM is released
      mbar_wait(drain, 0, p.status);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue
    const int quad = warp & 3;  // the TMEM lanes this warp may access
    uint8_t* staging = s_out + (warp - 2) * kStagingBuffers * kStagingBox;
    const int rsw = lane & 7;
    int local = 0, n_stores = 0;
    for (int tile = first; tile < total; tile += stride, ++local) {
      if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
      const bool two = second(tile);
      const Gemm& g = p.g[two];
      int m, n;
      tile_of(g, two ? tile - tiles0 : tile, m, n);
      const int buf = local & 1;
      const uint32_t tph = (local >> 1) & 1;
      const int wrow0 = m * kTileM + static_cast<int>(rank) * 128 + quad * 32;
      const int row = wrow0 + lane;
      const bool row_ok = row < g.M;
      const int col0 = n * g.n_step;
      const int ncols = min(g.n_step, g.N - col0);
      int label = -1;
      float lse2 = 0.f, ga = 0.f, gb = 0.f;
      if (kMode != CeMode::kProducts && row_ok) {
        label = __ldg(p.labels + row);
        if (label >= p.V) label = -1;
        label = label >= 0 ? label - p.v0 - col0 : -1;  // column of this tile, if it is one
      }
      if (kMode == CeMode::kGrad && row_ok) {
        const int id = __ldg(p.labels + row);
        const float dl = id >= 0 && id < p.V ? __ldg(p.d_loss + row) : 0.f;
        ga = p.scale * (dl + (p.d_lse ? __ldg(p.d_lse + row) : 0.f));
        gb = p.scale * dl;
        lse2 = __ldg(p.lse + row) * kLog2e;
      }
      const bool ok = __all_sync(0xffffffffu, mbar_wait(&tfull[buf], tph, p.status));
      if (!ok) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t t_lane =
          tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + buf * kTileN;
      const float c2 = p.scale * kLog2e;

      if (kMode == CeMode::kLse) {
        float mx = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int c = 0; c < ncols; c += 32) {
          __syncwarp();
          uint32_t a[32];
          tmem_ld_32x32b_x32(t_lane + c, a);
          tmem_ld_wait();
          const int left = ncols - c;
          if (label >= c && label < c + 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c + i == label) p.label_logit[row] = p.scale * __uint_as_float(a[i]);
          }
          float z[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            z[i] = i < left ? c2 * __uint_as_float(a[i]) : -INFINITY;
          float cm = mx;
#pragma unroll
          for (int i = 0; i < 32; ++i) cm = fmaxf(cm, z[i]);
          if (cm != -INFINITY) {  // all -inf so far: the sum stays 0
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) s += ex2(z[i] - cm);
            sum = fmaf(sum, ex2(mx - cm), s);
            mx = cm;
          }
        }
        if (row_ok) p.part[static_cast<long>(n) * g.M + row] = make_float2(mx, sum);
      } else {
        const bool f32_only = kMode == CeMode::kProducts && g.keep;
        float* acc = nullptr;
        if (kMode == CeMode::kProducts && (g.add || g.keep))
          acc = p.acc + static_cast<long>(row) * g.N + col0;
#pragma unroll 1
        for (int c = 0; c < kTileN; c += 64) {
          if (c >= ncols) break;
          uint8_t* box = staging + (n_stores % kStagingBuffers) * kStagingBox;
          if (!f32_only) {
            if (lane == 0) bulk_wait_group_read<kStagingBuffers - 1>();
            __syncwarp();
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int cc = c + 32 * h;
            __syncwarp();
            uint32_t a[32];
            tmem_ld_32x32b_x32(t_lane + cc, a);
            tmem_ld_wait();
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(a[i]);
            if (kMode == CeMode::kGrad) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                v[i] = ga * ex2(fmaf(v[i], c2, -lse2));
                if (cc + i == label) v[i] -= gb;
              }
            } else if (acc && row_ok) {
              // the width is a multiple of 8: whole float4 pairs
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                if (cc + i < ncols) {
                  float4* q = reinterpret_cast<float4*>(acc + cc + i);
                  if (g.add) {
                    const float4 o = *q;
                    v[i] += o.x, v[i + 1] += o.y, v[i + 2] += o.z, v[i + 3] += o.w;
                  }
                  if (g.keep) *q = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
              }
            }
            if (!f32_only) {
              uint8_t* srow = box + lane * 128;
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4*>(srow + (((4 * h + q) ^ rsw) << 4)) = make_uint4(
                    pack_bf16(v[8 * q], v[8 * q + 1]), pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                    pack_bf16(v[8 * q + 4], v[8 * q + 5]), pack_bf16(v[8 * q + 6], v[8 * q + 7]));
            }
          }
          if (!f32_only) {
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
              // rows and columns beyond the matrix are clipped by the map; a
              // box with no row inside is not stored at all
              if (wrow0 < g.M)
                tma_store_2d(two ? &m1.out : &m0.out, box, col0 + c, wrow0);
              bulk_commit_group();
            }
            ++n_stores;
          }
        }
      }
      tc_fence_before();
      pair::arrive_remote(pair::mapa(smem_u32(&tempty[buf]), 0));  // the leader's
    }
    if (kMode != CeMode::kLse && lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA frees TMEM or exits while the other may still signal its
  // barriers or the leader's MMAs may still write its TMEM
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    pair::tmem_dealloc2<512>(tmem_base);
  }
}

// lse and loss of every token from its tiles' (max, sum), in tile order: 32
// tokens x 8 runs of tiles per block.
__global__ void __launch_bounds__(256)
ce_join_kernel(const float2* __restrict__ part, const float* __restrict__ label_logit,
               const int32_t* __restrict__ labels, int T, int V, int tiles,
               float* __restrict__ loss, float* __restrict__ lse, uint32_t* status) {
  pdl_enter();
  __shared__ float2 s[8][32];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int t = blockIdx.x * 32 + lane;
  float m = -INFINITY, sum = 0.f;
  auto add = [&](float2 x) {
    const float cm = fmaxf(m, x.x);
    if (cm == -INFINITY) return;
    sum = sum * ex2(m - cm) + x.y * ex2(x.x - cm);
    m = cm;
  };
  if (t < T) {
    const int per = (tiles + 7) / 8, i1 = min(tiles, (q + 1) * per);
#pragma unroll 8
    for (int i = q * per; i < i1; ++i) add(part[static_cast<long>(i) * T + t]);
  }
  s[q][lane] = make_float2(m, sum);
  __syncthreads();
  if (q || t >= T) return;
  m = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) add(s[i][lane]);
  const float l = (m + log2f(sum)) * kLn2;
  lse[t] = l;
  const int id = labels[t];
  if (id >= V) record_status(status, kStatusIndex);
  loss[t] = id >= 0 && id < V ? l - label_logit[t] : 0.f;
}

// ------------------------------------------------------------------ host

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<EncodeFn>(ptr);
  }();
  return fn;
}

// bf16 [rows, cols] with rows ld elements apart; boxes of 64 columns x
// box_rows rows with the 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* base, long rows, long cols, long ld, int box_rows) {
  const EncodeFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Columns per tile: with the waves that 256-column tiles would take over the
// CTA pairs, the narrowest tile (a multiple of `unit`) that needs no more
// waves, so that the last wave is as full as the others.  The unit is what
// the epilogue takes at a time: 32 columns, or 64 where it stores them.
constexpr int kUnitLse = 32, kUnitGrad = 64;
int tile_columns(int m_tiles, int N, int unit) {
  const int pairs = std::max(1, num_sms() / 2);
  const long waves = ceil_div(static_cast<long>(m_tiles) * ceil_div(N, kTileN), pairs);
  int n = kTileN;
  while (n > unit && static_cast<long>(m_tiles) * ceil_div(N, n - unit) <= waves * pairs) n -= unit;
  return n;
}

Gemm make_gemm(long M, long N, long K, int n_step, bool a_mn, bool b_mn) {
  Gemm g{};
  g.M = static_cast<int>(M);
  g.N = static_cast<int>(N);
  g.m_tiles = ceil_div(M, kTileM);
  g.n_tiles = ceil_div(N, n_step);
  g.ksteps = ceil_div(K, kTileK);
  g.n_step = n_step;
  g.a_mn = a_mn;
  g.b_mn = b_mn;
  return g;
}

template <CeMode kMode>
cudaError_t launch_ce(const CeMaps& m0, const CeMaps& m1, const CeParams& p, cudaStream_t s) {
  auto kern = linear_ce_kernel<kMode>;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kSmemCe));
  if (err != cudaSuccess) return err;
  const long tiles = static_cast<long>(p.g[0].tiles()) +
                     (kMode == CeMode::kProducts ? p.g[1].tiles() : 0);
  const int pairs = static_cast<int>(std::max(1L, std::min<long>(num_sms() / 2, tiles)));
  return launch_kernel(kern, dim3(2 * pairs), dim3(kThreadsCe), kSmemCe, s, 2, m0, m1, p);
}

constexpr size_t kCeHeader = 256;
// Bytes of a piece's logit gradients: about half of L2, so that both products
// read them there.
constexpr size_t kPieceBytes = 64u << 20;

int check_ce(const moe_ce_problem* p) {
  if (!p || p->T < 0 || p->H < 1 || p->V < 1 || !std::isfinite(p->logit_scale))
    return MOE_ERR_INVALID_ARG;
  if (p->H % 8 != 0 || p->H > (1 << 20) || p->V > (1 << 26) || p->T > (1 << 26))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  // tile counts are 32-bit
  if (static_cast<long long>(ceil_div(p->T, kTileM)) * ceil_div(p->V, 32) >= (1LL << 30) ||
      static_cast<long long>(ceil_div(p->V, kTileM) + ceil_div(p->T, kTileM)) *
              ceil_div(p->H, kTileN) >=
          (1LL << 30))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

size_t ce_forward_bytes(const moe_ce_problem* p) {
  const int n = tile_columns(ceil_div(p->T, kTileM), p->V, kUnitLse);
  const size_t T = static_cast<size_t>(p->T);
  return kCeHeader + up(sizeof(float2) * T * ceil_div(p->V, n)) + up(sizeof(float) * T);
}

// Vocabulary rows per piece (a multiple of the tile), pieces of equal size.
int piece_rows(const moe_ce_problem* p) {
  const long most = std::max<long>(
      kTileM, static_cast<long>(kPieceBytes / 2 / std::max(1, p->T)) / kTileM * kTileM);
  const int pieces = ceil_div(p->V, most);
  return ceil_div(ceil_div(p->V, pieces), kTileM) * kTileM;
}

size_t ce_backward_bytes(const moe_ce_problem* p) {
  const size_t T = static_cast<size_t>(p->T);
  const int rows = piece_rows(p);
  return kCeHeader + up(2 * T * rows) + (rows < p->V ? up(sizeof(float) * T * p->H) : 0);
}

bool aligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

int check_ce_tensors(const void* x, const void* w, const int32_t* labels, const float* lse,
                     const float* loss, void* ws) {
  if (!ws) return MOE_ERR_INVALID_ARG;
  if (!x || !w || !labels || !lse || !loss) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(labels, 4) || !aligned(lse, 4) ||
      !aligned(loss, 4) || !aligned(ws, 256))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_linear_ce_workspace_size(const moe_ce_problem* p) {
  return check_ce(p) == MOE_OK ? ce_forward_bytes(p) : 0;
}

extern "C" size_t moe_linear_ce_backward_workspace_size(const moe_ce_problem* p) {
  return check_ce(p) == MOE_OK ? std::max(ce_forward_bytes(p), ce_backward_bytes(p)) : 0;
}

extern "C" int moe_linear_ce_forward(const moe_ce_problem* p, const void* x, const void* w,
                                     const int32_t* labels, float* loss, float* lse, void* ws,
                                     size_t ws_bytes, void* stream) {
  int rc = check_ce(p);
  if (rc != MOE_OK) return rc;
  set_last_launch_count(0);
  if (p->T == 0) return MOE_OK;
  rc = check_ce_tensors(x, w, labels, lse, loss, ws);
  if (rc != MOE_OK) return rc;
  if (ws_bytes < ce_forward_bytes(p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const int n_step = tile_columns(ceil_div(p->T, kTileM), p->V, kUnitLse);
  uint8_t* base = static_cast<uint8_t*>(ws) + kCeHeader;
  CeParams k{};
  k.g[0] = make_gemm(p->T, p->V, p->H, n_step, false, false);
  k.labels = labels;
  k.V = p->V;
  k.scale = p->logit_scale;
  k.part = reinterpret_cast<float2*>(base);
  k.label_logit = reinterpret_cast<float*>(
      base + up(sizeof(float2) * static_cast<size_t>(p->T) * k.g[0].n_tiles));
  k.status = static_cast<uint32_t*>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CeMaps m{};
  if (!make_map(&m.a, x, p->T, p->H, p->H, 128) || !make_map(&m.b, w, p->V, p->H, p->H, n_step / 2))
    return MOE_ERR_CUDA;
  if (launch_ce<CeMode::kLse>(m, m, k, s) != cudaSuccess) return MOE_ERR_CUDA;
  if (launch_kernel(ce_join_kernel, dim3(ceil_div(p->T, 32)), dim3(256), 0, s, 1,
                    static_cast<const float2*>(k.part), static_cast<const float*>(k.label_logit),
                    labels, p->T, p->V, k.g[0].n_tiles, loss, lse, k.status) != cudaSuccess)
    return MOE_ERR_CUDA;
  set_last_launch_count(2);
  return MOE_OK;
}

extern "C" int moe_linear_ce_backward(const moe_ce_problem* p, const void* x, const void* w,
                                      const int32_t* labels, const float* lse, const float* d_loss,
                                      const float* d_lse, void* dx, void* dw, void* ws,
                                      size_t ws_bytes, void* stream) {
  int rc = check_ce(p);
  if (rc != MOE_OK) return rc;
  if (!dw) return MOE_ERR_INVALID_ARG;
  if (!aligned(dw, 16)) return MOE_ERR_MISALIGNED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int launches = 0;
  set_last_launch_count(0);
  if (p->T == 0) {  // no tokens: the weights' gradient is zero
    if (cudaMemsetAsync(dw, 0, 2 * static_cast<size_t>(p->V) * p->H, s) != cudaSuccess)
      return MOE_ERR_CUDA;
    set_last_launch_count(1);
    return MOE_OK;
  }
  rc = check_ce_tensors(x, w, labels, lse, d_loss, ws);
  if (rc != MOE_OK) return rc;
  if (!dx) return MOE_ERR_INVALID_ARG;
  if (!aligned(dx, 16) || !aligned(d_lse, 4)) return MOE_ERR_MISALIGNED;
  if (ws_bytes < ce_backward_bytes(p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const int rows = piece_rows(p);
  const int pieces = ceil_div(p->V, rows);
  uint8_t* base = static_cast<uint8_t*>(ws) + kCeHeader;
  void* grad = base;  // [T, rows] bf16
  CeParams k{};
  k.labels = labels;
  k.V = p->V;
  k.scale = p->logit_scale;
  k.lse = lse;
  k.d_loss = d_loss;
  k.d_lse = d_lse;
  k.acc = reinterpret_cast<float*>(base + up(2 * static_cast<size_t>(p->T) * rows));
  k.status = static_cast<uint32_t*>(ws);
  for (int i = 0; i < pieces; ++i) {
    const int v0 = i * rows, nv = std::min(rows, p->V - v0);
    const uint8_t* wp = static_cast<const uint8_t*>(w) + 2 * static_cast<size_t>(v0) * p->H;
    uint8_t* dwp = static_cast<uint8_t*>(dw) + 2 * static_cast<size_t>(v0) * p->H;
    k.v0 = v0;
    const int n_step = tile_columns(ceil_div(p->T, kTileM), nv, kUnitGrad);
    k.g[0] = make_gemm(p->T, nv, p->H, n_step, false, false);
    CeMaps m{}, m1{};
    if (!make_map(&m.a, x, p->T, p->H, p->H, 128) || !make_map(&m.b, wp, nv, p->H, p->H, n_step / 2) ||
        !make_map(&m.out, grad, p->T, nv, rows, 32))
      return MOE_ERR_CUDA;
    if (launch_ce<CeMode::kGrad>(m, m, k, s) != cudaSuccess) return MOE_ERR_CUDA;
    k.g[0] = make_gemm(p->T, p->H, nv, kTileN, false, true);
    k.g[0].add = i > 0;
    k.g[0].keep = i + 1 < pieces;
    k.g[1] = make_gemm(nv, p->H, p->T, kTileN, true, true);
    if (!make_map(&m.a, grad, p->T, nv, rows, 128) || !make_map(&m.b, wp, nv, p->H, p->H, 64) ||
        !make_map(&m.out, dx, p->T, p->H, p->H, 32) || !make_map(&m1.a, grad, p->T, nv, rows, 64) ||
        !make_map(&m1.b, x, p->T, p->H, p->H, 64) || !make_map(&m1.out, dwp, nv, p->H, p->H, 32))
      return MOE_ERR_CUDA;
    if (launch_ce<CeMode::kProducts>(m, m1, k, s) != cudaSuccess) return MOE_ERR_CUDA;
    launches += 2;
  }
  set_last_launch_count(launches);
  return MOE_OK;
}
