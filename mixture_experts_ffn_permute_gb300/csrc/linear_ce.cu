// Softmax cross entropy of a linear layer, z = scale x W^T, on the sm_103a
// tensor cores, without keeping the logits (moe_linear_ce_* of
// include/moe_block.h).
//
// Forward.  One persistent GEMM over (256 tokens x N vocabulary rows) tiles of
// CTA pairs (tcgen05.mma.cta_group::2, fp32 accumulators in TMEM) whose
// epilogue keeps, per token and tile, the running maximum and the sum of
// exponentials (log2 units) and picks out the label's logit; a small kernel
// joins a token's tiles in order.  Up to 128 tokens: tiles of (128 x 128) of
// single CTAs (one_cta).  Per token and vocabulary tile 8 bytes leave
// the kernel instead of 2 N of logits.
//
// Backward, in pieces of the vocabulary whose logit gradients (bf16) take 128 MB
// (about what L2 holds; W and x pass through it too, and W and G are read about
// twice from HBM):
//   G  = a exp(z - lse) - b [v = label]  the forward's GEMM with another
//                                        epilogue, [T, piece] to the workspace
//   dx += S G W_piece    A = G K-major, B = W_piece read MN-major (as stored)
//   dW_piece = S G^T x   A = G, B = x, both read MN-major (as stored)
// with a = (d_loss + d_lse) / s, b = d_loss / s, S = scale s and s the largest
// finite |d_loss|.  G is rounded to bf16: under a mean, where every token has
// the same d_loss, its largest entries, the labels', are then -(1 - p) and not
// all rounded by the same amount (which would scale both gradients by up to
// 1 + 2^-8).  S multiplies the fp32 results.  The two products are tiles of
// one launch.  dx is kept in fp32 in the workspace from piece to
// piece (each element is one thread's in every piece, so the order of its sum
// is fixed) and rounded once by the last; with one piece it is written
// directly.
//
// Operands move in stages of 128 along K.  Where a matrix's row length is a
// multiple of 64 one bulk-tensor copy brings a stage of an operand as two
// 64-column planes, every row one 256-byte segment; otherwise two copies of
// 128-byte rows do (they zero-fill past the row's end, which planes cannot).
//
// The tensor core's fp32 accumulator loses a little at every step, always
// toward zero, which does not average out over a row of logits: at K = 4096 lse
// was 1e-6 of its value too small.  The forward therefore takes the
// accumulator out every 1024 of K and adds the parts in registers (128
// columns a thread, eight epilogue warps), while the tensor core fills the
// other accumulator.  The backward's logits keep all of K there: their exponents
// are off by that much from the forward's, a thousandth of the rounding of G to
// bf16 for logits of order one.
//
// Warp roles (one CTA per SM, tiles dealt to the pairs in a fixed order):
//   warp 0     TMA producer: 3 stages of 32 KB of A and 32 KB of B per CTA, up to 8
//              where few rows or narrow tiles make them smaller
//   warp 1     TMEM allocation, MMA issue (the leader CTA's)
//   warps 2..  epilogue, thread = row of the tile; two accumulators of 256
//              columns, so it overlaps the next mainloop; bf16 tiles leave
//              through swizzled staging and bulk-tensor stores
// Every wait is bounded (ptx.cuh).
//
// Measured (one GB300): T=4096 H=4096 V=32000, runs of 20 of one direction:
// forward 0.56 ms (1920 TFLOP/s), backward 1.79 ms (1800, its three products);
// both in turn, where the board's power cap counts, 2.5 to 2.65 ms (1620 to 1720
// for the four products; a plain library GEMM sustains 1695).  With few tokens
// the forward streams W: T=4 H=2048 V=32000 29 us with the join (131 MB, 19 us at
// HBM rate; 250 tiles on 152 CTAs, so that some take 256 rows of W where an even
// share is 210; launches, set-up and the join are the rest), T=4 H=4096 V=128000
// 165 us (6.4 TB/s).
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
constexpr int kTileK = 128;  // one stage
constexpr int kMaxStages = 8;
constexpr uint32_t kPlane = 128 * 64 * 2;            // 128 rows x 64 columns, 16 KB
constexpr uint32_t kRingCe = 3 * 4 * kPlane;         // 3 full stages, more of smaller ones
constexpr int kPromote = 8;  // forward: stages per accumulation in TMEM (K = 1024)
constexpr uint32_t kStagingBox = 32 * 128;           // 32 rows x 64 bf16
constexpr int kStagingBuffers = 2;
constexpr uint32_t kStagingCe = 4 * kStagingBuffers * kStagingBox;
constexpr size_t kSmemCe = 1024 + kRingCe + kStagingCe + 256;
static_assert(kSmemCe <= 232448, "shared memory budget");
static_assert((2 * kMaxStages + 5) * 8 + 8 + 4 * 4 <= 256, "barrier area");
constexpr int kGroupM = 8;  // m-tiles whose sweep over the n-tiles shares B tiles in L2
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One GEMM: C[M, N] = A B^T over K, by pair tiles.
struct Gemm {
  int m_tiles, n_tiles, ksteps;  // ksteps: stages of k_step
  int k_step;                 // 128, or (both operands MN-major) K's even share
  int n_step;                 // columns per tile (a multiple of 32, <= 256)
  int M, N;                   // extents (rows and columns beyond are not written)
  bool a_mn, b_mn;            // operand stored [K, M] (resp. [K, N]): read MN-major
  bool a_planes, b_planes;    // one copy per stage (row length a multiple of 64)
  int a_rows;                 // K-major A: rows per CTA that are loaded (128, fewer for small M)
  int splits;                 // of K: each is a tile of its own with its own sums in acc
  bool add, keep;             // fp32 sums: add to acc, leave them in acc (else bf16 out)
  float* acc;                 // [splits][M][N]
  __host__ __device__ int tiles() const { return m_tiles * n_tiles * splits; }
  // first stage of a split (splits are at most twice the CTA pairs: no overflow)
  __host__ __device__ int k_begin(int split) const {
    return splits == 1 ? split * ksteps : ksteps * split / splits;
  }
};

enum class CeMode : int { kLse = 0, kGrad = 1, kProducts = 2 };
// Epilogue warps: one per TMEM lane quadrant, two in the forward (each half
// of the columns)
template <CeMode kMode>
__host__ __device__ constexpr int epi_warps() { return kMode == CeMode::kLse ? 8 : 4; }
template <CeMode kMode>
__host__ __device__ constexpr int threads_ce() { return 64 + 32 * epi_warps<kMode>(); }

struct CeParams {
  Gemm g[2];            // kProducts: dx then dW; otherwise g[0]
  const int32_t* labels;
  int v0, V;            // first vocabulary row of the piece; vocabulary
  float scale;
  float2* part;         // kLse: [2 n_tiles][T] (max, sum) of a tile's halves in log2 units
  float* label_logit;   // kLse: [T]
  const float* lse;     // kGrad
  const float* d_loss;
  const float* d_lse;   // or NULL
  float* unit;          // s, the unit of G: kGrad finds and writes it
  int T;
  uint32_t* status;
  int stages;               // of the ring
  uint32_t a_stage, b_stage;  // bytes of a stage's operands in one CTA
};

struct CeMaps {
  CUtensorMap a, b, out;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A running softmax (maximum m, sum of 2^(v - m)): what the exponents are taken
// against.  It is finite also where m is not, so that the sum stays what the
// formula has: 0 while every logit is -inf, infinite once one is +inf, and NaN
// once one is NaN, which a maximum (fmaxf) does not show.
__device__ __forceinline__ float sum_unit(float m) { return fabsf(m) < INFINITY ? m : 0.f; }

// Descriptor of an MN-major operand: planes of 64 columns x k_step K rows with
// the 128-byte swizzle; leading offset = the next 64 columns (one plane),
// stride offset = 8 K rows.
__device__ __forceinline__ uint64_t mn_desc(uint32_t smem_addr, int k_step) {
  return sw128_kmajor_desc(smem_addr) ^ (static_cast<uint64_t>(1u) << 16) ^
         (static_cast<uint64_t>(k_step * 8) << 16);
}

__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Tile `i` of a GEMM: split by split, groups of kGroupM m-tiles sweep the
// n-tiles.
__device__ __forceinline__ void tile_of(const Gemm& g, int i, int& m, int& n, int& split) {
  split = 0;
  if (g.splits > 1) {
    split = i / (g.m_tiles * g.n_tiles);
    i -= split * (g.m_tiles * g.n_tiles);
  }
  if (g.m_tiles == 1) {
    m = 0;
    n = i;
    return;
  }
  const int per = kGroupM * g.n_tiles;
  const int grp = i / per, within = i - grp * per;
  const int size = min(kGroupM, g.m_tiles - grp * kGroupM);
  n = within / size;
  m = grp * kGroupM + (within - n * size);
}

// The tiles of one CTA pair of `pairs`, in order: g[0]'s round-robin, then
// g[1]'s so that the pairs whose share of g[0] was one tile shorter take their
// first `lead` tiles of g[1] while the others finish, the rest round-robin.
struct Deal {
  int pair, pairs, mine0, rem, tiles0, tiles1, lead;
  __device__ __forceinline__ Deal(const CeParams& p, int pair_, int pairs_, bool both) {
    pair = pair_;
    pairs = pairs_;
    tiles0 = p.g[0].tiles();
    tiles1 = both ? p.g[1].tiles() : 0;
    rem = tiles0 % pairs;
    mine0 = tiles0 / pairs + (pair < rem ? 1 : 0);
    lead = 0;
    if (!both) return;
    const int k0 = p.g[0].ksteps / max(1, p.g[0].splits);
    const int k1 = max(1, p.g[1].ksteps / max(1, p.g[1].splits));
    if (rem) lead = (k0 + k1 / 2) / k1;
  }
  // tile number `i` of this pair: false past the last; `second`: of g[1]
  __device__ __forceinline__ bool at(int i, int& tile, bool& second) const {
    second = i >= mine0;
    if (!second) {
      tile = i * pairs + pair;
      return true;
    }
    if (tiles1 == 0) return false;
    int j = i - mine0;
    if (pair >= rem) {
      if (j < lead) {
        tile = j * (pairs - rem) + (pair - rem);
        return tile < tiles1;
      }
      j -= lead;
    }
    tile = lead * (pairs - rem) + j * pairs + pair;
    return tile < tiles1;
  }
};

// The tensor core's operations of a CTA pair (cta_group::2) or of one CTA.
template <bool kPair>
struct Core {
  static __device__ __forceinline__ uint32_t rank() { return kPair ? cluster_ctarank() : 0; }
  static __device__ __forceinline__ void sync() {
    if (kPair) cluster_sync();
  }
  static __device__ __forceinline__ void load(void* dst, const CUtensorMap* map, bool planes,
                                              int c, int r, uint32_t plane, uint64_t* bar,
                                              uint64_t pol) {
    uint8_t* second = static_cast<uint8_t*>(dst) + plane;
    if (kPair) {  // a pair's loads complete on the leader's barrier
      const uint32_t b = pair::mapa(smem_u32(bar), 0);
      if (planes) {
        pair::tma_load_3d(dst, map, 0, r, c / 64, b, pol);
      } else {
        pair::tma_load(dst, map, c, r, b, pol);
        pair::tma_load(second, map, c + 64, r, b, pol);
      }
    } else if (planes) {
      tma_load_3d(dst, map, 0, r, c / 64, bar, pol);
    } else {
      tma_load_2d(dst, map, c, r, bar, pol);
      tma_load_2d(second, map, c + 64, r, bar, pol);
    }
  }
  static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             bool accumulate) {
    if (kPair) pair::mma(d, a, b, idesc, accumulate);
    else mma_bf16_ss(d, a, b, idesc, accumulate);
  }
  static __device__ __forceinline__ void commit(uint64_t* bar) {  // in both CTAs
    if (kPair) pair::commit_both(bar);
    else mma_commit(bar);
  }
  static __device__ __forceinline__ void commit_here(uint64_t* bar) {
    if (kPair) pair::commit_local(bar);
    else mma_commit(bar);
  }
};

// kPair: 256-row tiles of CTA pairs.  Otherwise (forward and logit gradients of at
// most 128 tokens: one_cta) every CTA takes 128-row tiles of its own: in a pair
// the second CTA would have no rows, and half of the epilogues nothing to do.
template <CeMode kMode, bool kPair>
__global__ void __launch_bounds__(threads_ce<kMode>(), 1)
linear_ce_kernel(const __grid_constant__ CeMaps m0, const __grid_constant__ CeMaps m1,
                 const __grid_constant__ CeParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sA = smem;
  uint8_t* sB = sA + p.stages * p.a_stage;
  uint8_t* s_out = smem + kRingCe;
  const int n_stages = p.stages;
  const uint32_t a_stage = p.a_stage, b_stage = p.b_stage;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_out + kStagingCe);  // past the forward's ring
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* s_unit = reinterpret_cast<float*>(tmem_slot + 2);  // one per epilogue warp (kGrad)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  using C = Core<kPair>;
  constexpr int kCtas = kPair ? 2 : 1;
  const uint32_t rank = C::rank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < n_stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kCtas * epi_warps<kMode>());  // one arrival per epilogue warp
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&m0.a);
    prefetch_tensormap(&m0.b);
  }
  if (warp == 1) {
    if (kPair) pair::tmem_alloc2<512>(tmem_slot);
    else tmem_alloc<512>(tmem_slot);
  }
  tc_fence_before();
  __syncthreads();
  C::sync();  // both CTAs' barriers exist before anything signals them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // nothing above touches global memory
  pdl_enter();
  const Deal deal(p, static_cast<int>(blockIdx.x) / kCtas, static_cast<int>(gridDim.x) / kCtas,
                  kMode == CeMode::kProducts);
  int tile, m, n, split;
  bool two;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      for (int i = 0; deal.at(i, tile, two); ++i) {
        if (*abort_flag) break;
        const Gemm& g = p.g[two];
        const CeMaps& maps = two ? m1 : m0;
        tile_of(g, tile, m, n, split);
        const int row0 = m * (128 * kCtas) + static_cast<int>(rank) * 128;
        const int half = g.n_step / kCtas;  // this CTA's columns of B
        const int col0 = n * g.n_step + static_cast<int>(rank) * half;
        const bool a_mn = g.a_mn, b_mn = g.b_mn, a_planes = g.a_planes, b_planes = g.b_planes;
        const uint32_t a_plane = static_cast<uint32_t>(a_mn ? g.k_step : g.a_rows) * 128;
        const uint32_t b_plane = static_cast<uint32_t>(b_mn ? g.k_step : half) * 128;
        // one CTA's rows may hold the whole of a small M (the MMA then reads
        // whatever the shared memory behind them holds: rows of the
        // accumulator that nobody reads)
        const bool a_load = rank == 0 || g.M > 128;
        const uint32_t bytes = (g.M > 128 ? 4 : 2) * a_plane + 2 * kCtas * b_plane;
        const int k_first = g.k_begin(split), k_last = g.k_begin(split + 1);
        // with one m-tile every pair reads the same A: each starts elsewhere in
        // K, so that they do not all ask for the same lines at once
        int kb = k_first;
        if (g.m_tiles == 1) kb += deal.pair % (k_last - k_first);
        bool ok = true;
        for (int j = k_first; j < k_last; ++j) {
          if (!mbar_wait(&empty[stage], phase ^ 1, p.status)) { ok = false; break; }
          if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
          const int k0 = kb * g.k_step;
          if (a_load)
            C::load(sA + stage * a_stage, &maps.a, a_planes, a_mn ? row0 : k0, a_mn ? k0 : row0,
                    a_plane, &full[stage], pol);
          C::load(sB + stage * b_stage, &maps.b, b_planes, b_mn ? col0 : k0, b_mn ? k0 : col0,
                  b_plane, &full[stage], pol);
          ++issued;
          if (++kb == k_last) kb = k_first;
          if (++stage == n_stages) { stage = 0; phase ^= 1; }
        }
        if (!ok) { *abort_flag = 1; break; }
      }
      // no bulk copy left in flight: the last fill of every stage has landed
      // (a pair's copies complete on the leader's barriers; the final cluster
      // barrier keeps the peer's shared memory until then)
      for (int i = 1; leader && i <= n_stages && i <= issued; ++i) {
        int s = stage - i;
        uint32_t ph = phase;
        if (s < 0) { s += n_stages; ph ^= 1; }
        mbar_wait(&full[s], ph, p.status);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (leader && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int seg = 0;  // accumulations so far: they alternate between the two accumulators
      bool ok = true;
      for (int i = 0; ok && deal.at(i, tile, two); ++i) {
        if (*abort_flag) break;
        const Gemm& g = p.g[two];
        const bool a_mn = g.a_mn, b_mn = g.b_mn;
        split = g.splits > 1 ? tile / (g.m_tiles * g.n_tiles) : 0;
        const int ksteps = g.k_begin(split + 1) - g.k_begin(split), k_step = g.k_step;
        const uint32_t idesc = idesc_bf16_f32(128 * kCtas, static_cast<uint32_t>(g.n_step)) |
                               (static_cast<uint32_t>(a_mn) << 15) |
                               (static_cast<uint32_t>(b_mn) << 16);
        // a K=16 step is 32 bytes along a K-major plane, which holds four (the
        // next plane four more), and 16 rows of 128 bytes of MN-major planes,
        // which hold eight; in units of 16 bytes
        const uint32_t as = a_mn ? 128 : 2, bs = b_mn ? 128 : 2;
        const uint32_t a4 = a_mn ? 512 : static_cast<uint32_t>(g.a_rows) * 8;
        const uint32_t b4 = b_mn ? 512 : static_cast<uint32_t>(g.n_step / kCtas) * 8;
        const int per_seg = kMode == CeMode::kLse ? kPromote : ksteps;
        for (int k0 = 0; ok && k0 < ksteps; k0 += per_seg, ++seg) {
          const int buf = seg & 1;
          if (!mbar_wait(&tempty[buf], ((seg >> 1) & 1) ^ 1, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + buf * kTileN;
          const int k1 = min(ksteps, k0 + per_seg);
          for (int kb = k0; kb < k1; ++kb) {
            if (!mbar_wait(&full[stage], phase, p.status)) { ok = false; break; }
            tc_fence_after();
            const uint32_t a = smem_u32(sA + stage * a_stage);
            const uint32_t b = smem_u32(sB + stage * b_stage);
            const uint64_t ad = a_mn ? mn_desc(a, k_step) : sw128_kmajor_desc(a);
            const uint64_t bd = b_mn ? mn_desc(b, k_step) : sw128_kmajor_desc(b);
#pragma unroll
            for (int kk = 0; kk < kTileK / 16; ++kk) {
              if (kk * 16 >= k_step) break;
              C::mma(d_tmem, ad + (kk & 3) * as + (kk >> 2) * a4,
                        bd + (kk & 3) * bs + (kk >> 2) * b4, idesc, kb > k0 || kk != 0);
            }
            C::commit(&empty[stage]);
            if (++stage == n_stages) { stage = 0; phase ^= 1; }
          }
          if (ok) C::commit(&tfull[buf]);
        }
        if (!ok) *abort_flag = 1;
      }
      C::commit_here(drain);  // every MMA done before TMEM is released
      mbar_wait(drain, 0, p.status);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue
    const int quad = warp & 3;  // the TMEM lanes this warp may access
    uint8_t* staging = s_out + (warp - 2) * kStagingBuffers * kStagingBox;
    const int rsw = lane & 7;
    const uint32_t t_quad = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t tempty_leader = kPair ? pair::mapa(smem_u32(tempty), 0) : 0;
    int seg = 0, n_stores = 0;
    bool go = true;
    float inv_unit = 1.f;
    if (kMode == CeMode::kGrad) {
      // s: the largest finite |d_loss| of a token that is not masked (1 if it is
      // 0, or so small that its reciprocal is not a number); every CTA for
      // itself, while the first tile is on its way
      float x = 0.f;
      bool bad = false;
#pragma unroll 4
      for (int t = static_cast<int>(threadIdx.x) - 64; t < p.T; t += 32 * epi_warps<kMode>()) {
        const float d = fabsf(__ldg(p.d_loss + t));
        const int id = __ldg(p.labels + t);
        bad |= id >= p.V;
        if (d <= 3e38f && id >= 0 && id < p.V) x = fmaxf(x, d);
      }
      if (blockIdx.x == 0 && bad) record_status(p.status, kStatusIndex);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
      if (lane == 0) s_unit[warp - 2] = x;
      bar_sync_named(1, 32 * epi_warps<kMode>());
#pragma unroll
      for (int w = 0; w < epi_warps<kMode>(); ++w) x = fmaxf(x, s_unit[w]);
      if (!(x >= 0x1p-100f)) x = 1.f;
      if (blockIdx.x == 0 && threadIdx.x == 64) *p.unit = x;
      inv_unit = 1.f / x;
    }
    // the next accumulation is complete
    auto wait_full = [&]() {
      go = __all_sync(0xffffffffu, mbar_wait(&tfull[seg & 1], (seg >> 1) & 1, p.status));
      if (!go && lane == 0) *abort_flag = 1;
      tc_fence_after();
      return go;
    };
    // it has been read (the leader's barrier of this accumulator)
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair) pair::arrive_remote(tempty_leader + (seg & 1) * 8);
        else mbar_arrive(&tempty[seg & 1]);
      }
      ++seg;
    };
    for (int i = 0; go && deal.at(i, tile, two); ++i) {
      if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
      const Gemm& g = p.g[two];
      tile_of(g, tile, m, n, split);
      const int wrow0 = m * (128 * kCtas) + static_cast<int>(rank) * 128 + quad * 32;
      const int row = wrow0 + lane;
      const bool row_ok = row < g.M, warp_ok = wrow0 < g.M;
      const int col0 = n * g.n_step;
      const int ncols = min(g.n_step, g.N - col0);
      int label = -1;
      float lse2 = 0.f, ga = 0.f, gb = 0.f;
      if (kMode != CeMode::kProducts && row_ok) {
        const int id = __ldg(p.labels + row);
        const bool valid = id >= 0 && id < p.V;
        if (valid) label = id - p.v0 - col0;  // column of this tile, if it is one
        if (kMode == CeMode::kGrad) {
          const float dl = valid ? __ldg(p.d_loss + row) : 0.f;
          ga = inv_unit * (dl + (p.d_lse ? __ldg(p.d_lse + row) : 0.f));
          gb = inv_unit * dl;
          lse2 = __ldg(p.lse + row) * kLog2e;
        }
      }
      const float c2 = p.scale * kLog2e;

      if (kMode == CeMode::kLse) {
        // this warp's half of the columns: up to 128 of a row per thread, of one
        // CTA's tiles up to 64
        constexpr int kChunks = kPair ? 4 : 2;
        const int half = (warp - 2) >> 2, c0 = half * 32 * kChunks;
        uint32_t z[kChunks][32];  // fp32
        for (int k0 = 0; k0 < g.ksteps; k0 += kPromote) {
          if (!wait_full()) break;
          const uint32_t t_lane = t_quad + (seg & 1) * kTileN + c0;
          if (warp_ok) {
            __syncwarp();
            if (k0 == 0) {  // all at once (columns past the tile's are not used)
#pragma unroll
              for (int q = 0; q < kChunks; ++q) tmem_ld_32x32b_x32(t_lane + 32 * q, z[q]);
              tmem_ld_wait();
            } else {
#pragma unroll
              for (int q = 0; q < kChunks; ++q) {
                uint32_t a[32];
                tmem_ld_32x32b_x32(t_lane + 32 * q, a);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  z[q][j] = __float_as_uint(__uint_as_float(z[q][j]) + __uint_as_float(a[j]));
              }
            }
          }
          release();
        }
        if (!go) break;
        float mx = -INFINITY, sum = 0.f;
#pragma unroll
        for (int q = 0; q < kChunks; ++q) {
          const int c = c0 + 32 * q, left = ncols - c;
          if (!warp_ok || left <= 0) continue;
          if (label >= c && label < c + 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j == label) p.label_logit[row] = p.scale * __uint_as_float(z[q][j]);
          }
          // four chains each for the maximum and the sum
          float v[32], cm[4] = {mx, mx, mx, mx}, s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            v[j] = j < left ? c2 * __uint_as_float(z[q][j]) : -INFINITY;
            cm[j & 3] = fmaxf(cm[j & 3], v[j]);
          }
          const float m4 = fmaxf(fmaxf(cm[0], cm[1]), fmaxf(cm[2], cm[3]));
          // one rescaling a chunk
          const float unit = sum_unit(m4);
#pragma unroll
          for (int j = 0; j < 32; ++j) s4[j & 3] += ex2(v[j] - unit);
          sum = fmaf(sum, ex2(mx - unit), (s4[0] + s4[1]) + (s4[2] + s4[3]));
          mx = m4;
        }
        if (row_ok) p.part[static_cast<long>(2 * n + half) * g.M + row] = make_float2(mx, sum);
      } else {
        if (!wait_full()) break;
        const uint32_t t_lane = t_quad + (seg & 1) * kTileN;
        const bool f32_only = kMode == CeMode::kProducts && g.keep;
        float* acc = nullptr;
        if (kMode == CeMode::kProducts && (g.add || g.keep))
          acc = g.acc + (static_cast<long>(split) * g.M + row) * g.N + col0;
        const CUtensorMap* out = two ? &m1.out : &m0.out;
        const float S = kMode == CeMode::kProducts ? p.scale * __ldg(p.unit) : 1.f;
#pragma unroll 1
        for (int c = 0; c < (warp_ok ? ncols : 0); c += 64) {
          uint8_t* box = staging + (n_stores % kStagingBuffers) * kStagingBox;
          if (!f32_only) {
            if (lane == 0) bulk_wait_group_read<kStagingBuffers - 1>();
            __syncwarp();
          }
          __syncwarp();
          uint32_t a[2][32];
          tmem_ld_32x32b_x32(t_lane + c, a[0]);
          tmem_ld_32x32b_x32(t_lane + c + 32, a[1]);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int cc = c + 32 * h;
            float v[32];
#pragma unroll
            for (int i2 = 0; i2 < 32; ++i2) v[i2] = __uint_as_float(a[h][i2]);
            if (kMode == CeMode::kGrad) {
              // columns past the vocabulary, up to the store's 64: zeros, which
              // the products read along K
#pragma unroll
              for (int i2 = 0; i2 < 32; ++i2) {
                const float e = ga * ex2(fmaf(v[i2], c2, -lse2));
                v[i2] = cc + i2 < ncols ? (cc + i2 == label ? e - gb : e) : 0.f;
              }
            } else if (acc && row_ok) {
              // the width is a multiple of 8: whole float4s
#pragma unroll
              for (int i2 = 0; i2 < 32; i2 += 4) {
                if (cc + i2 < ncols) {
                  float4* q = reinterpret_cast<float4*>(acc + cc + i2);
                  if (g.add) {
                    const float4 o = *q;
                    v[i2] += o.x, v[i2 + 1] += o.y, v[i2 + 2] += o.z, v[i2 + 3] += o.w;
                  }
                  if (g.keep) *q = make_float4(v[i2], v[i2 + 1], v[i2 + 2], v[i2 + 3]);
                }
              }
            }
            if (!f32_only) {
              if (kMode == CeMode::kProducts) {
#pragma unroll
                for (int i2 = 0; i2 < 32; ++i2) v[i2] *= S;
              }
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
            if (lane == 0) {  // rows and columns past the matrix are clipped by the map
              tma_store_2d(out, box, col0 + c, wrow0);
              bulk_commit_group();
            }
            ++n_stores;
          }
        }
        release();
      }
    }
    if (kMode != CeMode::kLse && lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA frees TMEM or exits while the other may still signal its
  // barriers or the leader's MMAs may still write its TMEM
  C::sync();
  if (warp == 1) {
    tc_fence_after();
    if (kPair) pair::tmem_dealloc2<512>(tmem_base);
    else tmem_dealloc<512>(tmem_base);
  }
}

// lse and loss of every token from its tiles' (max, sum), in tile order: 32
// tokens x 32 runs of tiles per block.
__global__ void __launch_bounds__(1024)
ce_join_kernel(const float2* __restrict__ part, const float* __restrict__ label_logit,
               const int32_t* __restrict__ labels, int T, int V, int tiles,
               float* __restrict__ loss, float* __restrict__ lse, uint32_t* status) {
  pdl_enter();
  __shared__ float2 s[32][32];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int t = blockIdx.x * 32 + lane;
  float m = -INFINITY, sum = 0.f;
  auto add = [&](float2 x) {
    const float cm = fmaxf(m, x.x), unit = sum_unit(cm);
    sum = sum * ex2(m - unit) + x.y * ex2(x.x - unit);
    m = cm;
  };
  if (t < T) {
    const int per = (tiles + 31) / 32, i1 = min(tiles, (q + 1) * per);
#pragma unroll 8
    for (int i = q * per; i < i1; ++i) add(part[static_cast<long>(i) * T + t]);
  }
  s[q][lane] = make_float2(m, sum);
  __syncthreads();
  if (q || t >= T) return;
  m = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) add(s[i][lane]);
  const float l = (m + log2f(sum)) * kLn2;
  lse[t] = l;
  const int id = labels[t];
  if (id >= V) record_status(status, kStatusIndex);
  loss[t] = id >= 0 && id < V ? l - label_logit[t] : 0.f;
}

// out [n] bf16 = scale * unit * the sum of the splits' fp32 sums, in order; n a
// multiple of 8.
__global__ void __launch_bounds__(256)
ce_split_join_kernel(const float* __restrict__ acc, int splits, long n, float scale,
                     const float* __restrict__ unit, uint4* __restrict__ out) {
  pdl_enter();
  const float f = scale * *unit;
  const long step = static_cast<long>(gridDim.x) * 256;
  for (long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x; i < n / 8; i += step) {
    float v[8] = {};
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float4* q = reinterpret_cast<const float4*>(acc + s * n) + 2 * i;
      const float4 a = __ldg(q), b = __ldg(q + 1);
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
      v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
    out[i] = make_uint4(pack_bf16(f * v[0], f * v[1]), pack_bf16(f * v[2], f * v[3]),
                        pack_bf16(f * v[4], f * v[5]), pack_bf16(f * v[6], f * v[7]));
  }
}

// dst [rows, cols] = src [rows, H], zeros behind it: rows of whole planes.  H
// and cols multiples of 8.
__global__ void __launch_bounds__(256)
ce_pad_kernel(const uint4* __restrict__ src, uint4* __restrict__ dst, long rows, int h_vecs,
              int col_vecs) {
  pdl_enter();
  const long total = rows * col_vecs, step = static_cast<long>(gridDim.x) * 256;
#pragma unroll 4
  for (long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x; i < total; i += step) {
    const long r = i / col_vecs;
    const int c = static_cast<int>(i - r * col_vecs);
    dst[i] = c < h_vecs ? __ldg(src + r * h_vecs + c) : make_uint4(0, 0, 0, 0);
  }
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

// bf16 [rows, cols] with rows ld elements apart, as planes of 64 columns; boxes
// of two planes x box_rows rows with the 128-byte swizzle (cols a multiple
// of 64).
bool make_planes(CUtensorMap* map, const void* base, long rows, long cols, long ld, int box_rows) {
  const EncodeFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(cols / 64)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, 128};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 2};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same matrix in boxes of 64 columns x box_rows rows.
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

// Tiles of one CTA each (at most 128 columns: a stage is then as large as a
// pair's) instead of a pair's.  Forward / logit gradients and products, one CTA
// against pairs, us: T=1 H=64 V=32000 10.8 against 13.8 / 24.2 against 27.4; T=8
// H=128 V=50021 12.9, 17.8 / 37.7, 42.0; T=32 H=256 V=32000 11.3, 15.9 / 30.1,
// 33.4; T=128 H=1024 V=32000 22.6, 25.3 / 75.6, 77.6; T=4 H=4096 V=128000 172,
// 176 / 780, 775 (the only row where one of the two, the backward, is slower, by
// less than 1%).  Rows that are not whole planes copy slowly, and tiles half
// as wide copy those of x twice as often: T=96 H=1000 V=50021 44.7, 39.2 / 115,
// 113; T=128 H=8 V=200000 141, 93 / 251, 209: pairs there.
bool one_cta(const moe_ce_problem* p) { return p->T <= 128 && p->H % 64 == 0; }

// Columns per tile: with the waves that the widest tiles would take over the
// CTA pairs (or the CTAs), the narrowest tile (a multiple of `unit`) that needs
// no more waves, so that the last wave is as full as the others.  The unit is what
// the epilogue takes at a time: 32 columns, or 64 where it stores them.
constexpr int kUnitLse = 32, kUnitGrad = 64;
int tile_columns(const moe_ce_problem* p, int N, int unit) {
  const int m_tiles = ceil_div(p->T, kTileM);
  const int workers = one_cta(p) ? num_sms() : std::max(1, num_sms() / 2);
  const int most = one_cta(p) ? 128 : kTileN;
  const long waves = ceil_div(static_cast<long>(m_tiles) * ceil_div(N, most), workers);
  int n = most;
  while (n > unit && static_cast<long>(m_tiles) * ceil_div(N, n - unit) <= waves * workers)
    n -= unit;
  return n;
}

// A row-major bf16 matrix in global memory.
struct Matrix {
  const void* p;
  long rows, cols, ld;
};

// C[M, N] = A B^T over K from the operands as stored ([M, K] and [N, K], or
// [K, M] and [K, N] read MN-major) and their maps; false if a map could not be
// made.
bool make_gemm(Gemm* g, CeMaps* maps, long M, long N, long K, int n_step, const Matrix& a,
               bool a_mn, const Matrix& b, bool b_mn, bool pair = true) {
  *g = Gemm{};
  g->M = static_cast<int>(M);
  g->N = static_cast<int>(N);
  g->m_tiles = ceil_div(M, kTileM);
  g->n_tiles = ceil_div(N, n_step);
  g->ksteps = ceil_div(K, kTileK);
  // A stage of MN-major operands can have any multiple of 16 along K: stages of
  // equal depth leave no last one whose rows are mostly filled with zeros,
  // which copies slowly.
  g->k_step = a_mn && b_mn ? ceil_div(ceil_div(K, g->ksteps), 16) * 16 : kTileK;
  g->n_step = n_step;
  g->splits = 1;
  g->a_mn = a_mn;
  g->b_mn = b_mn;
  g->a_planes = a.cols % 64 == 0;
  g->b_planes = b.cols % 64 == 0;
  g->a_rows = a_mn || M > 128 ? 128 : ceil_div(M, 8) * 8;
  auto make = [](CUtensorMap* m, const Matrix& x, bool planes, int rows) {
    return planes ? make_planes(m, x.p, x.rows, x.cols, x.ld, rows)
                  : make_map(m, x.p, x.rows, x.cols, x.ld, rows);
  };
  return make(&maps->a, a, g->a_planes, a_mn ? g->k_step : g->a_rows) &&
         make(&maps->b, b, g->b_planes, b_mn ? g->k_step : pair ? n_step / 2 : n_step);
}

template <CeMode kMode, bool kPair>
cudaError_t launch_ce(const CeMaps& m0, const CeMaps& m1, CeParams& p, cudaStream_t s) {
  auto kern = linear_ce_kernel<kMode, kPair>;
  p.a_stage = p.b_stage = 0;
  for (const Gemm& g : p.g) {
    if (g.tiles() == 0) continue;
    p.a_stage = std::max(p.a_stage, static_cast<uint32_t>(g.a_rows) * 256);
    p.b_stage = std::max(p.b_stage, static_cast<uint32_t>(g.n_step) * (kPair ? 128 : 256));
  }
  // the forward has no staging for output tiles: its ring takes that room too
  const uint32_t ring = kRingCe + (kMode == CeMode::kLse ? kStagingCe : 0);
  p.stages = std::min<int>(kMaxStages, ring / (p.a_stage + p.b_stage));
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kSmemCe));
  if (err != cudaSuccess) return err;
  const long tiles = static_cast<long>(p.g[0].tiles()) + p.g[1].tiles();
  constexpr int kCtas = kPair ? 2 : 1;
  const int groups = static_cast<int>(std::max(1L, std::min<long>(num_sms() / kCtas, tiles)));
  return launch_kernel(kern, dim3(kCtas * groups), dim3(threads_ce<kMode>()), kSmemCe, s, kCtas, m0,
                       m1, p);
}
template <CeMode kMode>
cudaError_t launch_ce_logits(const CeMaps& m, bool one, CeParams& p, cudaStream_t s) {
  return one ? launch_ce<kMode, false>(m, m, p, s)
             : launch_ce<kMode, true>(m, m, p, s);
}

constexpr size_t kCeHeader = 256;
constexpr size_t kUnitOffset = 64;  // of s in the header
// A piece's logit gradients: 128 MB, and 4096 vocabulary rows at least.  Larger
// pieces mean fewer passes over dx's fp32 sums and fuller last waves, smaller
// ones less workspace.  The backward with 32, 64, 128, 256 MB and one piece:
// T=4096 H=4096 V=32000 2.16, 1.87, 1.79, 1.73, 1.74 ms; T=2048 H=1024 V=131072
// 1.64, 1.22, 1.11, 1.03, 1.00 ms.  128 MB is not the fastest, it is what 3% and 10%
// more time buy: a workspace that does not double.
constexpr size_t kPieceBytes = 128u << 20;
constexpr int kPieceRows = 4096;

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

// Rows whose length is not a multiple of 16 start off the 32-byte sectors, and
// the copies move a sector more with every 128 bytes of theirs.  From three
// m-tiles on, where W is read from L2 again and again, x and W are copied once
// to rows of whole planes.  Both directions with / without the copy, V=50021:
// H=1000 T=777 354 / 429 us, T=1024 395 / 471, T=600 298 / 321, T=300 257 / 255,
// T=64 208 / 155; H=1008, whose rows start on sectors: T=600 297 / 257,
// T=2048 641 / 620, T=4096 1178 / 1226.
bool padded(const moe_ce_problem* p) { return p->H % 16 != 0 && p->T > 2 * kTileM; }
int padded_width(const moe_ce_problem* p) { return ceil_div(p->H, 64) * 64; }

size_t ce_pad_bytes(const moe_ce_problem* p, long w_rows) {
  return padded(p) ? up(2 * static_cast<size_t>(p->T) * padded_width(p)) +
                         up(2 * static_cast<size_t>(w_rows) * padded_width(p))
                   : 0;
}

size_t ce_forward_bytes(const moe_ce_problem* p) {
  const int n = tile_columns(p, p->V, kUnitLse);
  const size_t T = static_cast<size_t>(p->T);
  return kCeHeader + up(sizeof(float2) * T * 2 * ceil_div(p->V, n)) + up(sizeof(float) * T) +
         ce_pad_bytes(p, p->V);
}

// Vocabulary rows per piece (a multiple of the tile), pieces of equal size.
int piece_rows(const moe_ce_problem* p) {
  const long most = std::max<long>(
      kPieceRows, static_cast<long>(kPieceBytes / 2 / std::max(1, p->T)) / kTileM * kTileM);
  const int pieces = ceil_div(p->V, most);
  return ceil_div(ceil_div(p->V, pieces), kTileM) * kTileM;
}

// Splits of the two products of a piece.  A tile with few others and a long K
// (dx for few tokens, dW for a small vocabulary) would keep one CTA pair busy
// long after the rest have finished: K is cut so that no tile takes more than
// half of a pair's share of the launch, into parts of eight stages at least.
// T=777 H=1000 V=50021: dx is 16 tiles of 391 stages, and both products took
// 270 us unsplit.
struct Splits {
  int dx, dw;
};
Splits splits_of(const moe_ce_problem* p, int rows) {
  const long cols = ceil_div(p->H, kTileN), pairs = std::max(1, num_sms() / 2);
  const long nv = std::min(rows, p->V);
  const long t0 = ceil_div(p->T, kTileM) * cols, k0 = ceil_div(nv, kTileK);
  const long t1 = ceil_div(nv, kTileM) * cols, k1 = ceil_div(p->T, kTileK);
  const long share = std::max(1L, (t0 * k0 + t1 * k1) / pairs);
  auto cut = [&](long k) {
    return static_cast<int>(std::max(1L, std::min((2 * k + share - 1) / share, k / 8)));
  };
  return {cut(k0), cut(k1)};
}

// The backward's workspace past the header.
struct BackwardLayout {
  size_t grad, dx, dw, pad_x, pad_w, total;
};
BackwardLayout backward_layout(const moe_ce_problem* p) {
  const size_t T = static_cast<size_t>(p->T), H = static_cast<size_t>(p->H);
  const int rows = piece_rows(p);
  const size_t nv = static_cast<size_t>(std::min(rows, p->V));
  const Splits sp = splits_of(p, rows);
  BackwardLayout L;
  size_t o = kCeHeader;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up(bytes);
    return at;
  };
  L.grad = take(2 * T * rows);
  L.dx = take(sizeof(float) * T * H * (sp.dx > 1 ? sp.dx : rows < p->V ? 1 : 0));
  L.dw = take(sizeof(float) * nv * H * (sp.dw > 1 ? sp.dw : 0));
  L.pad_x = take(padded(p) ? 2 * T * padded_width(p) : 0);
  L.pad_w = take(padded(p) ? 2 * nv * padded_width(p) : 0);
  L.total = o;
  return L;
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

// A [rows, H] matrix as the GEMMs read it: itself, or its padded copy at `copy`
// (one launch).
cudaError_t operand(Matrix* m, const moe_ce_problem* p, const void* src, long rows, void* copy,
                    cudaStream_t s, int* launches) {
  *m = {src, rows, p->H, p->H};
  if (!padded(p)) return cudaSuccess;
  const int cols = padded_width(p);
  *m = {copy, rows, cols, cols};
  ++*launches;
  const long blocks = std::min<long>(8L * num_sms(), (rows * (cols / 8) + 255) / 256);
  return launch_kernel(ce_pad_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, 1,
                       static_cast<const uint4*>(src), static_cast<uint4*>(copy), rows, p->H / 8,
                       cols / 8);
}

cudaError_t join_splits(const float* acc, int splits, long n, float scale, const float* unit,
                        void* out, cudaStream_t s, int* launches) {
  ++*launches;
  const long blocks = std::min<long>(8L * num_sms(), (n / 8 + 255) / 256);
  return launch_kernel(ce_split_join_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s,
                       1, acc, splits, n, scale, unit, static_cast<uint4*>(out));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_linear_ce_workspace_size(const moe_ce_problem* p) {
  return check_ce(p) == MOE_OK ? ce_forward_bytes(p) : 0;
}

extern "C" size_t moe_linear_ce_backward_workspace_size(const moe_ce_problem* p) {
  return check_ce(p) == MOE_OK ? std::max(ce_forward_bytes(p), backward_layout(p).total) : 0;
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
  const int n_step = tile_columns(p, p->V, kUnitLse);
  uint8_t* base = static_cast<uint8_t*>(ws) + kCeHeader;
  CeParams k{};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int launches = 0;
  const size_t n_part = up(sizeof(float2) * static_cast<size_t>(p->T) * 2 * ceil_div(p->V, n_step));
  uint8_t* pad = base + n_part + up(sizeof(float) * static_cast<size_t>(p->T));
  Matrix xm, wm;
  if (operand(&xm, p, x, p->T, pad, s, &launches) != cudaSuccess ||
      operand(&wm, p, w, p->V, pad + up(2 * static_cast<size_t>(p->T) * padded_width(p)), s,
              &launches) != cudaSuccess)
    return MOE_ERR_CUDA;
  CeMaps m{};
  if (!make_gemm(&k.g[0], &m, p->T, p->V, xm.cols, n_step, xm, false, wm, false, !one_cta(p)))
    return MOE_ERR_CUDA;
  k.labels = labels;
  k.V = p->V;
  k.scale = p->logit_scale;
  k.part = reinterpret_cast<float2*>(base);
  k.label_logit = reinterpret_cast<float*>(base + n_part);
  k.status = static_cast<uint32_t*>(ws);
  if (launch_ce_logits<CeMode::kLse>(m, one_cta(p), k, s) != cudaSuccess) return MOE_ERR_CUDA;
  if (launch_kernel(ce_join_kernel, dim3(ceil_div(p->T, 32)), dim3(1024), 0, s, 1,
                    static_cast<const float2*>(k.part), static_cast<const float*>(k.label_logit),
                    labels, p->T, p->V, 2 * k.g[0].n_tiles, loss, lse, k.status) != cudaSuccess)
    return MOE_ERR_CUDA;
  set_last_launch_count(launches + 2);
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
  const BackwardLayout L = backward_layout(p);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const int rows = piece_rows(p);
  const int pieces = ceil_div(p->V, rows);
  const Splits sp = splits_of(p, rows);
  uint8_t* base = static_cast<uint8_t*>(ws);
  void* grad = base + L.grad;  // [T, rows] bf16
  float* acc_dx = reinterpret_cast<float*>(base + L.dx);
  float* acc_dw = reinterpret_cast<float*>(base + L.dw);
  CeParams k{};
  k.labels = labels;
  k.V = p->V;
  k.scale = p->logit_scale;
  k.lse = lse;
  k.d_loss = d_loss;
  k.d_lse = d_lse;
  k.status = static_cast<uint32_t*>(ws);
  float* unit = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kUnitOffset);
  k.unit = unit;
  k.T = p->T;
  Matrix xm, wm;
  if (operand(&xm, p, x, p->T, base + L.pad_x, s, &launches) != cudaSuccess) return MOE_ERR_CUDA;
  for (int i = 0; i < pieces; ++i) {
    const int v0 = i * rows, nv = std::min(rows, p->V - v0);
    const uint8_t* wp = static_cast<const uint8_t*>(w) + 2 * static_cast<size_t>(v0) * p->H;
    uint8_t* dwp = static_cast<uint8_t*>(dw) + 2 * static_cast<size_t>(v0) * p->H;
    k.v0 = v0;
    const int n_step = tile_columns(p, nv, kUnitGrad);
    if (operand(&wm, p, wp, nv, base + L.pad_w, s, &launches) != cudaSuccess) return MOE_ERR_CUDA;
    // padded to whole planes: the epilogue writes zeros there
    const Matrix gm{grad, p->T, ceil_div(nv, 64) * 64L, rows};
    CeMaps m{}, m1{};
    k.g[1] = Gemm{};
    if (!make_gemm(&k.g[0], &m, p->T, nv, xm.cols, n_step, xm, false, wm, false,
                   !one_cta(p)) ||
        !make_map(&m.out, grad, p->T, gm.cols, rows, 32))
      return MOE_ERR_CUDA;
    if (launch_ce_logits<CeMode::kGrad>(m, one_cta(p), k, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (!make_gemm(&k.g[0], &m, p->T, p->H, nv, kTileN, gm, false, wm, true) ||
        !make_map(&m.out, dx, p->T, p->H, p->H, 32) ||
        !make_gemm(&k.g[1], &m1, nv, p->H, p->T, kTileN, gm, true, xm, true) ||
        !make_map(&m1.out, dwp, nv, p->H, p->H, 32))
      return MOE_ERR_CUDA;
    // a short last piece may have fewer stages than there are splits: it adds
    // to the first ones' sums
    k.g[0].splits = std::min(sp.dx, k.g[0].ksteps);
    k.g[0].acc = acc_dx;
    k.g[0].add = i > 0;
    k.g[0].keep = sp.dx > 1 || i + 1 < pieces;
    k.g[1].splits = sp.dw;
    k.g[1].acc = acc_dw;
    k.g[1].keep = sp.dw > 1;
    if (launch_ce<CeMode::kProducts, true>(m, m1, k, s) != cudaSuccess) return MOE_ERR_CUDA;
    launches += 2;
    if (sp.dw > 1 && join_splits(acc_dw, sp.dw, static_cast<long>(nv) * p->H, p->logit_scale, unit,
                                 dwp, s, &launches) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  if (sp.dx > 1 && join_splits(acc_dx, sp.dx, static_cast<long>(p->T) * p->H, p->logit_scale, unit,
                               dx, s, &launches) != cudaSuccess)
    return MOE_ERR_CUDA;
  set_last_launch_count(launches);
  return MOE_OK;
}
