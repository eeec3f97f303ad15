// Grouped matrix product of E4M3 operands with a scale per 128 of a row of x and
// per 128 x 128 of the weights (moe_fp8_matmul of include/moe_experts.h).
//
//   out[r, n] = sum_b x_scale[r, b] w_scale[e, n / 128, b] <x[r, b], w[e, n, b]>
//
// The tensor core (tcgen05.mma kind::f8f6f4, fp32 accumulators in TMEM) sums one
// block of 128 along K at a time; the epilogue warps multiply the block's sums by
// the two scales and add them up in registers while it fills the other
// accumulator.
//
// Tiles of 256 rows x 256 columns on CTA pairs (128 rows of both operands per
// CTA).  A thread of the epilogue has one row of the tile and the columns of one
// weight block, so that a block's factor is one product of two scalars and the
// sums are 128 registers.  Eight warps do it (registers are moved to them from
// the other four): a block takes the tensor core 512 cycles, and the epilogue 64
// packed FMA and four 32-column reads of TMEM a thread.
//
// Operands move in stages of two blocks.  Where K is a multiple of 128 one
// bulk-tensor copy brings both blocks of an operand as two 128-byte planes, every
// row one 256-byte segment; otherwise two copies of 128-byte rows do, which
// zero-fill past the row's end.
//
// Every wait is bounded (ptx.cuh).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/moe_experts.h"
#include "internal.h"
#include "pair_tiles.cuh"
#include "ptx.cuh"
#include "rowwise.cuh"

namespace moe {
namespace {

constexpr int kBlk = 128;                       // a scale's extent along K and N
constexpr uint32_t kPlane = 128 * kBlk;         // 128 rows x 128 codes, 16 KB
constexpr uint32_t kStageBytes = 4 * kPlane;    // two blocks of both operands
constexpr int kStages = 3;
constexpr int kMaxE = MOE_MAX_EXPERTS;
constexpr int kGroupM = 8;  // row tiles whose sweep over the columns shares weight tiles in L2
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;  // warps 0-3: copies, MMA, two idle
constexpr uint32_t kBarBytes = 256;
constexpr size_t kSmem = 1024 + kStages * kStageBytes + kBarBytes + 2 * (kMaxE + 1) * sizeof(int32_t);
static_assert(kSmem <= 232448, "shared memory budget");
// registers: a launch's 168 x 384, moved as 40 x 128 + 232 x 256
static_assert(40 * 128 + 232 * 256 <= 168 * kThreads, "register split");

struct MmParams {
  const int32_t* offsets;  // NULL: one expert, all rows
  const float* xs;
  const float* ws;
  void* out;
  int M, N, E, kblocks, nblocks, n_tiles;
  int planes;  // operands come as planes
  int f32;     // out
  int vec;     // 32-byte stores
  uint32_t* status;
};

// Instruction descriptor, kind::f8f6f4 with E4M3 A/B, fp32 D, both K-major.
__device__ __forceinline__ uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

template <bool kPair>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  if (kPair) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

template <uint32_t kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <uint32_t kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Copies two blocks of `rows` rows into shared memory: one copy of two planes, or
// two copies (the second one's zeros past the end of K too).
template <bool kPair>
__device__ __forceinline__ void load_x(void* dst, const CUtensorMap* map, bool planes, int kb,
                                       int r, uint32_t plane, uint64_t* bar, uint64_t pol) {
  uint8_t* second = static_cast<uint8_t*>(dst) + plane;
  if (kPair) {
    const uint32_t b = pair::mapa(smem_u32(bar), 0);
    if (planes) {
      pair::tma_load_3d(dst, map, 0, r, kb, b, pol);
    } else {
      pair::tma_load(dst, map, kb * kBlk, r, b, pol);
      pair::tma_load(second, map, (kb + 1) * kBlk, r, b, pol);
    }
  } else if (planes) {
    tma_load_3d(dst, map, 0, r, kb, bar, pol);
  } else {
    tma_load_2d(dst, map, kb * kBlk, r, bar, pol);
    tma_load_2d(second, map, (kb + 1) * kBlk, r, bar, pol);
  }
}
template <bool kPair>
__device__ __forceinline__ void load_w(void* dst, const CUtensorMap* map, bool planes, int kb,
                                       int n, int e, uint32_t plane, uint64_t* bar, uint64_t pol) {
  uint8_t* second = static_cast<uint8_t*>(dst) + plane;
  if (kPair) {
    const uint32_t b = pair::mapa(smem_u32(bar), 0);
    if (planes) {
      pair::tma_load_4d(dst, map, 0, n, kb, e, b, pol);
    } else {
      pair::tma_load_3d(dst, map, kb * kBlk, n, e, b, pol);
      pair::tma_load_3d(second, map, (kb + 1) * kBlk, n, e, b, pol);
    }
  } else if (planes) {
    tma_load_4d(dst, map, 0, n, kb, e, bar, pol);
  } else {
    tma_load_3d(dst, map, kb * kBlk, n, e, bar, pol);
    tma_load_3d(second, map, (kb + 1) * kBlk, n, e, bar, pol);
  }
}

// Expert offsets into s_off[E + 1] and the experts' first tiles into
// s_tile[E + 1], tile heights of `rows`; the number of tiles (0, and the status,
// where the offsets decrease or leave [0, M]).  Every thread of the block.
template <int kBlockThreads>
__device__ __forceinline__ int build_tiles(const int32_t* offsets, int E, int M, int n_tiles,
                                           int rows, int32_t* s_off, int32_t* s_tile,
                                           uint32_t* status) {
  __shared__ int s_part[kBlockThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i <= E; i += kBlockThreads)
    s_off[i] = offsets ? offsets[i] : i == 0 ? 0 : M;
  __syncthreads();
  const int per = (E + kBlockThreads - 1) / kBlockThreads;
  const int e0 = min(E, static_cast<int>(threadIdx.x) * per), e1 = min(E, e0 + per);
  bool bad = false;
  int run = 0;
  for (int e = e0; e < e1; ++e) {
    const int a = s_off[e], b = s_off[e + 1];
    if (a < 0 || b < a || b > M) bad = true;
    else run += (b - a + rows - 1) / rows * n_tiles;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) record_status(status, kStatusIndex);
    return 0;
  }
  int incl = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_part[warp] = incl;
  __syncthreads();
  int acc = incl - run, total = 0;
  for (int w = 0; w < kBlockThreads / 32; ++w) {
    if (w < warp) acc += s_part[w];
    total += s_part[w];
  }
  for (int e = e0; e < e1; ++e) {
    s_tile[e] = acc;
    acc += (s_off[e + 1] - s_off[e] + rows - 1) / rows * n_tiles;
  }
  if (threadIdx.x == 0) s_tile[E] = total;
  __syncthreads();
  return total;
}

// Where tile `i` lies: `e` only ever grows along a CTA's tiles.
struct Cursor {
  int e = 0, m = 0, n = 0;
  __device__ __forceinline__ void at(int i, const int32_t* s_tile, int n_tiles) {
    while (s_tile[e + 1] <= i) ++e;
    const int local = i - s_tile[e], m_tiles = (s_tile[e + 1] - s_tile[e]) / n_tiles;
    if (m_tiles == 1) {
      m = 0;
      n = local;
      return;
    }
    const int per = kGroupM * n_tiles, grp = local / per, within = local - grp * per;
    const int size = min(kGroupM, m_tiles - grp * kGroupM);
    n = within / size;
    m = grp * kGroupM + (within - n * size);
  }
};

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Arrival on a barrier of the pair that hands over no memory.
__device__ __forceinline__ void arrive_remote_relaxed(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster)
               : "memory");
}

// Until the loads from TMEM have come; the values take part, so that their uses
// stay behind it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

struct Maps {
  CUtensorMap x, w;
};

template <bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
fp8_matmul_kernel(const __grid_constant__ Maps maps, const __grid_constant__ MmParams p) {
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int kN = 128 * kCtas;           // columns of a tile
  constexpr int kCols = kN / 2;             // of an epilogue thread
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sX = smem;                        // [stage][2 planes]
  uint8_t* sW = smem + kStages * 2 * kPlane;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* s_off = reinterpret_cast<int32_t*>(smem + kStages * kStageBytes + kBarBytes);
  int32_t* s_tile = s_off + kMaxE + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0;
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kCtas * kEpiWarps);  // one arrival per epilogue warp
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.x);
    prefetch_tensormap(&maps.w);
  }
  if (warp == 1) {
    if (kPair) pair::tmem_alloc2<512>(tmem_slot);
    else tmem_alloc<512>(tmem_slot);
  }
  // nothing above touches global memory
  pdl_enter();
  const int total = build_tiles<kThreads>(p.offsets, p.E, p.M, p.n_tiles, 128 * kCtas, s_off,
                                          s_tile, p.status);
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();  // both CTAs' barriers exist before anything signals them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int first = static_cast<int>(blockIdx.x) / kCtas, step = static_cast<int>(gridDim.x) / kCtas;

  if (warp < 4) {
    regs_down<40>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- producer
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      Cursor c;
      bool ok = true;
      for (int i = first; ok && i < total && !*abort_flag; i += step) {
        c.at(i, s_tile, p.n_tiles);
        const int row = s_off[c.e] + (c.m * kCtas + static_cast<int>(rank)) * 128;
        const int col = (c.n * kCtas + static_cast<int>(rank)) * 128;
        for (int kb = 0; kb < p.kblocks; kb += 2) {
          if (!mbar_wait(&empty[stage], phase ^ 1, p.status)) { ok = false; break; }
          if (leader) mbar_arrive_expect_tx(&full[stage], kCtas * kStageBytes);
          load_x<kPair>(sX + stage * 2 * kPlane, &maps.x, p.planes, kb, row, kPlane, &full[stage], pol);
          load_w<kPair>(sW + stage * 2 * kPlane, &maps.w, p.planes, kb, col, c.e, kPlane, &full[stage],
                        pol);
          ++issued;
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) *abort_flag = 1;
      // no bulk copy left in flight (a pair's complete on the leader's barriers)
      for (int i = 1; leader && i <= kStages && i <= issued; ++i) {
        int s = stage - i;
        uint32_t ph = phase;
        if (s < 0) { s += kStages; ph ^= 1; }
        mbar_wait(&full[s], ph, p.status);
      }
    } else if (warp == 1 && leader && lane == 0) {
      // -------------------------------------------------------------- MMA issuer
      const uint32_t idesc = idesc_e4m3(128 * kCtas, kN);
      int stage = 0;
      uint32_t phase = 0;
      int seg = 0;  // blocks so far: they alternate between the two accumulators
      bool ok = true;
      for (int i = first; ok && i < total && !*abort_flag; i += step) {
        for (int kb = 0; ok && kb < p.kblocks; kb += 2) {
          if (!mbar_wait(&full[stage], phase, p.status)) { ok = false; break; }
          tc_fence_after();
          for (int h = 0; h < 2 && kb + h < p.kblocks; ++h, ++seg) {
            const int buf = seg & 1;
            if (!mbar_wait(&tempty[buf], ((seg >> 1) & 1) ^ 1, p.status)) { ok = false; break; }
            tc_fence_after();
            const uint64_t a = sw128_kmajor_desc(smem_u32(sX + (stage * 2 + h) * kPlane));
            const uint64_t b = sw128_kmajor_desc(smem_u32(sW + (stage * 2 + h) * kPlane));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_e4m3<kPair>(tmem_base + buf * 256, a + 2 * kk, b + 2 * kk, idesc, kk != 0);
            if (kPair) pair::commit_both(&tfull[buf]);
            else mma_commit(&tfull[buf]);
          }
          if (!ok) break;
          if (kPair) pair::commit_both(&empty[stage]);
          else mma_commit(&empty[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) *abort_flag = 1;
      if (kPair) pair::commit_local(drain);  // every MMA done before TMEM is released
      else mma_commit(drain);
      mbar_wait(drain, 0, p.status);
    }
    __syncwarp();
  } else {
    regs_up<232>();
    // ---------------------------------------------------------------- epilogue
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + half * kCols;
    const uint32_t tempty_leader = kPair ? pair::mapa(smem_u32(tempty), 0) : 0;
    int seg = 0;
    bool go = true;
    Cursor c;
    for (int i = first; go && i < total; i += step) {
      if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
      c.at(i, s_tile, p.n_tiles);
      const int row0 = s_off[c.e] + (c.m * kCtas + static_cast<int>(rank)) * 128 + quad * 32;
      const int rows = s_off[c.e + 1];
      const long row = row0 + lane;
      const int col = c.n * kN + half * kCols;
      const bool live = row0 < rows && col < p.N, row_ok = row < rows;
      const float* xs = p.xs + (row_ok ? row : 0) * p.kblocks;
      const float* ws = p.ws + (static_cast<long>(c.e) * p.nblocks + min(col / kBlk, p.nblocks - 1)) *
                                   p.kblocks;
      Pair acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = 0;
      // The next block's sums are complete: the accumulator's columns.
      auto wait_full = [&]() {
        go = __all_sync(0xffffffffu, mbar_wait(&tfull[seg & 1], (seg >> 1) & 1, p.status));
        tc_fence_after();
        return t_lane + (seg & 1) * 256;
      };
      // They have been read (the leader's barrier; nothing else is handed over).
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kPair) arrive_remote_relaxed(tempty_leader + (seg & 1) * 8);
          else mbar_arrive(&tempty[seg & 1]);
        }
        ++seg;
      };
      // A step is 32 columns of a block: the next step's sums are on their way
      // from TMEM while this one's are scaled and added, and the accumulator is
      // free as soon as its last ones have come.
      constexpr int kSteps = kCols / 32;
      constexpr int kAhead = 2;  // factors on their way
      float fx[kAhead], fw[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        fx[j] = j < p.kblocks ? __ldg(xs + j) : 0.f;
        fw[j] = j < p.kblocks ? __ldg(ws + j) : 0.f;
      }
      uint32_t a[2][32], t = wait_full();
      if (go && live) tmem_ld_32x32b_x32(t, a[0]);
      for (int kb0 = 0; go && kb0 < p.kblocks; kb0 += kAhead) {
        float f[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          f[j] = fx[j] * fw[j];
          const int kb = kb0 + kAhead + j;
          fx[j] = kb < p.kblocks ? __ldg(xs + kb) : 0.f;
          fw[j] = kb < p.kblocks ? __ldg(ws + kb) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (!go || kb0 + j >= p.kblocks) break;
          const Pair f2 = pair_of(f[j], f[j]);
#pragma unroll
          for (int q = 0; q < kSteps; ++q) {
            const int here = (j * kSteps + q) & 1;
            if (live) tmem_ld_wait_for(a[here]);
            if (q + 1 < kSteps) {
              if (live) tmem_ld_32x32b_x32(t + 32 * (q + 1), a[here ^ 1]);
            } else {
              release();
              if (kb0 + j + 1 < p.kblocks) {
                t = wait_full();
                if (go && live) tmem_ld_32x32b_x32(t, a[here ^ 1]);
              }
            }
            if (live) {
#pragma unroll
              for (int n = 0; n < 16; ++n)
                acc[q * 16 + n] = pair_fma(
                    pair_of(__uint_as_float(a[here][2 * n]), __uint_as_float(a[here][2 * n + 1])), f2,
                    acc[q * 16 + n]);
            }
          }
        }
      }
      if (!go && lane == 0) *abort_flag = 1;
      if (!go) break;
      if (!live || !row_ok) continue;
      const int ncols = min(kCols, p.N - col);
      const long at = row * p.N + col;
      if (p.vec && ncols % 16 == 0) {
        if (p.f32) {
          float* o = static_cast<float*>(p.out) + at;
#pragma unroll
          for (int j = 0; j < kCols; j += 8) {
            if (j >= ncols) continue;
            uint32_t w[8];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              float lo, hi;
              unpair(acc[j / 2 + n], lo, hi);
              w[2 * n] = __float_as_uint(lo);
              w[2 * n + 1] = __float_as_uint(hi);
            }
            store32(o + j, w);
          }
        } else {
          uint16_t* o = static_cast<uint16_t*>(p.out) + at;
#pragma unroll
          for (int j = 0; j < kCols; j += 16) {
            if (j >= ncols) continue;
            uint32_t w[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              float lo, hi;
              unpair(acc[j / 2 + n], lo, hi);
              w[n] = pack_bf16(lo, hi);
            }
            store32(o + j, w);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
          float v[2];
          unpair(acc[j], v[0], v[1]);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (2 * j + n < ncols) {
              if (p.f32) static_cast<float*>(p.out)[at + 2 * j + n] = v[n];
              else from_float(static_cast<Bf16*>(p.out)[at + 2 * j + n], v[n]);
            }
          }
        }
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA frees TMEM or exits while the other may still signal its
  // barriers or the leader's MMAs may still write its TMEM
  if (kPair) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if (kPair) pair::tmem_dealloc2<512>(tmem_base);
    else tmem_dealloc<512>(tmem_base);
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

// Codes [experts][rows][K] in boxes of 128 columns (two planes of them where
// `planes`) x box_rows rows, with the 128-byte swizzle; experts 0: no such axis.
bool make_codes_map(CUtensorMap* map, const void* base, long K, long rows, long experts,
                    bool planes, int box_rows) {
  const EncodeFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4], strides[3];
  cuuint32_t box[4], estr[4] = {1, 1, 1, 1};
  int n = 0;
  dims[n] = static_cast<cuuint64_t>(planes ? kBlk : K);
  box[n++] = kBlk;
  strides[n - 1] = static_cast<cuuint64_t>(K);
  dims[n] = static_cast<cuuint64_t>(rows);
  box[n++] = static_cast<cuuint32_t>(box_rows);
  if (planes) {
    strides[n - 1] = kBlk;
    dims[n] = static_cast<cuuint64_t>(K / kBlk);
    box[n++] = 2;
  }
  if (experts) {
    strides[n - 1] = static_cast<cuuint64_t>(K) * static_cast<cuuint64_t>(rows);
    dims[n] = static_cast<cuuint64_t>(experts);
    box[n++] = 1;
  }
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(n),
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kHeader = 256;

bool off(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

int check_matmul(const moe_fp8_problem* p) {
  if (!p || p->M < 0 || p->N < 1 || p->K < 1 || p->E < 1) return MOE_ERR_INVALID_ARG;
  if (p->out_dtype != MOE_DTYPE_BF16 && p->out_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (p->E > MOE_MAX_EXPERTS || p->K % 16 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  // tile counts and the coordinates of copies are 32-bit
  if (p->M > (1 << 30) || p->N > (1 << 30) || p->K > (1 << 30) ||
      (static_cast<int64_t>(ceil_div(p->M, 16)) + p->E) * ceil_div(p->N, kBlk) >= (1LL << 30))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  // a tensor map's strides are below 2^40 bytes
  if (static_cast<int64_t>(p->N) * p->K >= (1LL << 40)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

template <bool kPair>
cudaError_t launch_tiles(const moe_fp8_problem* p, const void* x, const void* w, MmParams& k,
                         cudaStream_t s) {
  constexpr int kCtas = kPair ? 2 : 1;
  Maps maps;
  if (!make_codes_map(&maps.x, x, p->K, p->M, 0, k.planes, 128) ||
      !make_codes_map(&maps.w, w, p->K, p->N, p->E, k.planes, 128))
    return cudaErrorInvalidValue;
  k.n_tiles = ceil_div(p->N, 128 * kCtas);
  auto kern = fp8_matmul_kernel<kPair>;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kSmem));
  if (err != cudaSuccess) return err;
  const long most = (ceil_div(p->M, 128 * kCtas) + static_cast<long>(std::min(p->E, p->M))) * k.n_tiles;
  const int groups = static_cast<int>(std::max(1L, std::min<long>(num_sms() / kCtas, most)));
  return launch_kernel(kern, dim3(static_cast<unsigned>(kCtas * groups)), dim3(kThreads), kSmem, s,
                       kCtas, maps, k);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_fp8_matmul_workspace_size(const moe_fp8_problem* p) {
  return check_matmul(p) == MOE_OK ? kHeader : 0;
}

extern "C" int moe_fp8_matmul(const moe_fp8_problem* p, const void* x, const float* x_scale,
                              const void* w, const float* w_scale, const int32_t* expert_offsets,
                              void* out, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_matmul(p);
  if (rc != MOE_OK) return rc;
  if (!expert_offsets && p->E != 1) return MOE_ERR_INVALID_ARG;
  set_last_launch_count(0);
  if (p->M == 0) return MOE_OK;
  if (!x || !x_scale || !w || !w_scale || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (off(x, 16) || off(w, 16) || off(out, 16) || off(x_scale, 4) || off(w_scale, 4) ||
      off(expert_offsets, 4) || off(ws, 256))
    return MOE_ERR_MISALIGNED;
  if (ws_bytes < moe_fp8_matmul_workspace_size(p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  MmParams k{};
  k.offsets = expert_offsets;
  k.xs = x_scale;
  k.ws = w_scale;
  k.out = out;
  k.M = p->M;
  k.N = p->N;
  k.E = p->E;
  k.kblocks = ceil_div(p->K, kBlk);
  k.nblocks = ceil_div(p->N, kBlk);
  k.planes = p->K % kBlk == 0;
  k.f32 = p->out_dtype == MOE_DTYPE_F32;
  k.vec = p->N % 16 == 0 && !off(out, 32);
  k.status = static_cast<uint32_t*>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_tiles<true>(p, x, w, k, s) != cudaSuccess) return MOE_ERR_CUDA;
  set_last_launch_count(1);
  return MOE_OK;
}
