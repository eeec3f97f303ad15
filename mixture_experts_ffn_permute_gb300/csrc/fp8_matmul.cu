// Grouped matrix product of E4M3 operands with a scale per 128 of a row of x and
// per 128 x 128 of the weights (moe_fp8_matmul of include/moe_experts.h).
//
//   out[r, n] = sum_b x_scale[r, b] w_scale[e, n / 128, b] <x[r, b], w[e, n, b]>
//
// The tensor core (tcgen05.mma kind::f8f6f4, fp32 accumulators in TMEM) sums one
// block of 128 along K at a time; the epilogue warps multiply the block's sums by
// the two scales and add them up in registers while it fills the other
// accumulator.  Two kinds of tiles:
//
//   wide    256 rows of x on the M side, 256 columns on the N side, on CTA pairs
//           (128 rows of both operands per CTA).  A thread of the epilogue has one
//           row and the 128 columns of one weight block, so that a block's factor is
//           one number.
//   narrow  128 columns (weights) per CTA on the M side and up to 128 rows of x on
//           the N side, as many as there are: the form for few rows, where the
//           weights' bytes are the time.  Single CTAs, or in a pair an expert's last
//           rows.  A thread has one column; the rows' factors come from shared
//           memory, four at a time.
//
// Where there are few narrow tiles, clusters of two or four CTAs share one along K
// and add their sums up, in the order of K, through distributed shared memory.
//
// Warp roles: 0 copies; 1 and 2 issue MMAs, each into accumulators of its own; 3
// multiplies the scales ahead of the epilogue, 8 warps, to which most registers are
// moved.
//
// Operands move in stages of two blocks.  Where K is a multiple of 128 one
// bulk-tensor copy brings both blocks of an operand as two 128-byte planes, every
// row one 256-byte segment; otherwise two copies of 128-byte rows do, which
// zero-fill past the row's end.
//
// What bounds it.  Wide: the epilogue.  A block takes the tensor core 512 cycles, its
// commits some 100, and the epilogue 770: reading TMEM and FMAs, 250 cycles each and
// behind one another (the two warps of a scheduler go in step), and 270 for the
// hand-over.  A tile's end, whose sums go out while nothing else is done, takes 5000
// of its 31000.  M=8192 E=8 N=28672 K=4096: 0.75 ms in short runs (2580 TFLOP/s), 0.85 in
// long ones or on another GB300 (2260); without the FMAs, before they were packed, 0.72 for
// 0.87, and the copies and hand-overs alone take 0.57.
// Measured and not kept, us at that size: 16 epilogue warps (870 to 1000), loads of the
// next columns under the FMAs (745 to 1100: registers move), four accumulators of 128
// columns (the MMA is slower at N = 128; 985 to 1150), tiles of 192 columns (877 to 1007),
// one commit for epilogue and producer (745 to 755), looking at the next accumulator's
// barrier ahead of the FMAs (745 to 782), one lane's wait for the warp (816 to 876).
// Narrow: HBM where there are many tiles (M=2048 E=256 N=4096 K=7168 886 us, 6.9 TB/s);
// with one tile a CTA its latency, 0.17 us a block and some 6 us of launch, tiles and
// first copies (M=8 of 128 experts, N=1536 K=2048: 11 us).
//
// Every wait is bounded (ptx.cuh).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
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
constexpr uint32_t kRing = 3 * 4 * kPlane;      // stages of two blocks of both operands
constexpr int kMaxStages = kRing / (2 * kPlane + 2 * kBlk * 64);  // (of the lowest tiles: 4)
constexpr int kMaxE = MOE_MAX_EXPERTS;
constexpr int kGroupM = 8;  // row tiles whose sweep over the columns shares weight tiles in L2
constexpr int kNarrow = 128;                    // rows of a narrow tile at most
constexpr int kBoxes = 4;                       // heights of its copies: 16, 32, 64, 128 rows
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;  // warps 0-3: copies, MMA (two), factors
constexpr uint32_t kBarBytes = 256;
constexpr int kChunk = 8;                        // blocks whose factors come together
constexpr uint32_t kFactors = kChunk * 2 * 128;  // [block][weight block][row]
constexpr size_t kSmem = 1024 + kRing + kBarBytes + 2 * kFactors * sizeof(float) +
                         2 * (kMaxE + 1) * sizeof(int32_t);
static_assert(kSmem <= 232448, "shared memory budget");
static_assert((2 * kMaxStages + 10) * 8 + 8 <= kBarBytes, "barrier area");
// registers: a launch's 168 x 384, moved to the epilogue as far as the others can do
// without
template <bool kSplit>
struct Regs {
  static constexpr int kOther = kSplit ? 72 : 56, kEpilogue = kSplit ? 216 : 224;
  static_assert(kOther * 128 + kEpilogue * 32 * kEpiWarps <= 168 * kThreads, "register split");
};

struct MmParams {
  const int32_t* offsets;  // NULL: one expert, all rows
  const float* xs;
  const float* ws;
  void* out;
  int M, N, E, kblocks, nblocks, n_tiles;
  int tile_rows;    // rows of a tile at most: 256 (pairs), or of a narrow one
  int tile_shift;   // its logarithm
  int stages;       // of the ring
  int splits;       // of K: CTAs of a cluster that share a tile (single CTAs, else 1)
  uint32_t x_stage; // bytes of a stage's rows in one CTA
  int planes;  // operands come as planes
  int f32;     // out
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
// s_tile[E + 1]; the number of tiles (0, and the status, where the offsets decrease
// or leave [0, M]).  Every thread of the block.
__device__ __forceinline__ int build_tiles(const MmParams& p, int32_t* s_off, int32_t* s_tile) {
  __shared__ int s_part[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.E + kThreads - 1) / kThreads;
  const int e0 = min(p.E, static_cast<int>(threadIdx.x) * per), e1 = min(p.E, e0 + per);
  bool bad = false;
  int run = 0, a = 0;
  for (int e = e0; e < e1; ++e) {
    if (e == e0) a = p.offsets ? p.offsets[e] : 0;
    const int b = p.offsets ? p.offsets[e + 1] : p.M;
    s_off[e] = a;
    if (e + 1 == p.E) s_off[p.E] = b;
    if (a < 0 || b < a || b > p.M) bad = true;
    else run += (b - a + p.tile_rows - 1) / p.tile_rows * p.n_tiles;
    a = b;
  }
  int incl = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_part[warp] = incl;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) record_status(p.status, kStatusIndex);
    return 0;
  }
  int acc = incl - run, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int part = s_part[w];
    if (w < warp) acc += part;
    total += part;
  }
  for (int e = e0; e < e1; ++e) {
    s_tile[e] = acc;
    acc += (s_off[e + 1] - s_off[e] + p.tile_rows - 1) / p.tile_rows * p.n_tiles;
  }
  if (threadIdx.x == 0) s_tile[p.E] = total;
  return total;  // (the caller's barrier shows the tiles to every thread)
}

// The tiles of a CTA (pair), in order: which expert's, and where.
//
// A wide tile (pairs alone) has 256 rows on the tensor core's M side and 256
// columns on its N side.  A narrow one, an expert's last rows where they are at
// most 128, has the weights on the M side and only as many rows as there are on
// the N side: its tensor core and epilogue time goes with them, and the weights'
// bytes are what is left.
struct Tile {
  int e = 0, m = 0, n = 0;
  int row, left;  // first row, rows (at most the tile's)
  bool narrow;
  int half;       // narrow: rows per CTA, a multiple of 16
  int box;        // rows per copy: 16 << index
  // `e` only ever grows along a CTA's tiles
  template <bool kPair>
  __device__ __forceinline__ void at(int i, const MmParams& p, const int32_t* s_off,
                                     const int32_t* s_tile) {
    while (s_tile[e + 1] <= i) ++e;
    const int local = i - s_tile[e];
    row = s_off[e];
    const int m_tiles = (s_off[e + 1] - row + p.tile_rows - 1) >> p.tile_shift;
    if (m_tiles == 1) {
      m = 0;
      n = local;
    } else {  // (divisions where they are needed: each is some 150 cycles of a tile's start)
      const int per = kGroupM * p.n_tiles;
      const int grp = m_tiles <= kGroupM ? 0 : local / per, within = local - grp * per;
      const int size = min(kGroupM, m_tiles - grp * kGroupM);
      n = size == kGroupM ? within / kGroupM : within / size;
      m = grp * kGroupM + (within - n * size);
    }
    row += m * p.tile_rows;
    left = min(s_off[e + 1] - row, p.tile_rows);
    narrow = !kPair || left <= kNarrow;
    half = kPair ? ((left + 1) / 2 + 15) & ~15 : (left + 15) & ~15;
    box = !narrow ? 3 : half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
  }
  __device__ __forceinline__ uint32_t x_plane() const { return 16u * kBlk << box; }
};

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Four lanes' rows of four times eight words each to a row after the other of which
// every lane has eight: words 8 s .. 8 s + 7 of lane c are then those that lane s of
// the four had at 8 c.
__device__ __forceinline__ void rows_across(uint32_t (&v)[32]) {
#pragma unroll
  for (int b = 1; b <= 2; b *= 2) {
    const bool high = (threadIdx.x & b) != 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & b) continue;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        uint32_t &x = v[8 * k + n], &y = v[8 * (k | b) + n];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? x : y, b);
        x = high ? got : x;
        y = high ? y : got;
      }
    }
  }
}

// The value, of which the compiler knows nothing: what depends on it is not worked
// out ahead of the tiles' loops, to lie in registers that the sums need.
__device__ __forceinline__ long opaque(long v) {
  asm volatile("" : "+l"(v));
  return v;
}

// One thread's arrival by a predicate: a branch that not all lanes take costs the
// epilogue some 50 cycles a block (M=8192 E=8 N=28672 K=4096 762 us with branches for the
// arrivals, 743 without).
__device__ __forceinline__ void arrive_if(bool mine, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(static_cast<uint32_t>(mine))
      : "memory");
}
// On a barrier of the pair's first CTA; hands over no memory.
__device__ __forceinline__ void arrive_leader_if(bool mine, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(
          pair::mapa(smem_u32(bar), 0)),
      "r"(static_cast<uint32_t>(mine))
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

// 64 columns of 32 lanes, when they have come.
__device__ __forceinline__ void tmem_ld_64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
               : "r"(taddr)
               : "memory");
}

// Two sums at once: half the issue slots of two FMAs.
__device__ __forceinline__ void fma2(uint64_t& s, uint32_t a0, uint32_t a1, uint64_t f) {
  uint64_t a;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "r"(a0), "r"(a1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(s) : "l"(a), "l"(f));
}

// v += four values of a CTA's shared memory of the cluster.
__device__ __forceinline__ void add_cluster(float (&v)[4], uint32_t addr_cluster) {
  float a[4];
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3])
               : "r"(addr_cluster)
               : "memory");
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] += a[j];
}

struct Maps {
  CUtensorMap x[kBoxes], w;  // x in boxes of 16, 32, 64 and 128 rows
};

// Shared memory behind the ring, by constant offsets from its aligned base; and (where
// CTAs share a tile) how many blocks along K this CTA has of it.
struct Smem {
  uint8_t* base;
  int part;
  template <bool kSplit>
  __device__ __forceinline__ int blocks(const MmParams& p) const {
    return kSplit ? part : p.kblocks;
  }
  __device__ __forceinline__ uint64_t* bar(int i) const {
    return reinterpret_cast<uint64_t*>(base + kRing) + i;
  }
  __device__ __forceinline__ uint64_t* full(int s) const { return bar(s); }
  __device__ __forceinline__ uint64_t* empty(int s) const { return bar(kMaxStages + s); }
  __device__ __forceinline__ uint64_t* tfull(int b) const { return bar(2 * kMaxStages + b); }
  __device__ __forceinline__ uint64_t* tempty(int b) const { return bar(2 * kMaxStages + 2 + b); }
  __device__ __forceinline__ uint64_t* ffull(int b) const { return bar(2 * kMaxStages + 4 + b); }
  __device__ __forceinline__ uint64_t* fempty(int b) const { return bar(2 * kMaxStages + 6 + b); }
  // of either issuer
  __device__ __forceinline__ uint64_t* drain(int b) const { return bar(2 * kMaxStages + 8 + b); }
  __device__ __forceinline__ uint32_t* tmem_slot() const {
    return reinterpret_cast<uint32_t*>(bar(2 * kMaxStages + 10));
  }
  __device__ __forceinline__ volatile int* abort_flag() const {
    return reinterpret_cast<volatile int*>(tmem_slot() + 1);
  }
  __device__ __forceinline__ float* factors(int b) const {
    return reinterpret_cast<float*>(base + kRing + kBarBytes) + b * kFactors;
  }
  __device__ __forceinline__ int32_t* off() const { return reinterpret_cast<int32_t*>(factors(2)); }
  __device__ __forceinline__ int32_t* tile() const { return off() + kMaxE + 1; }
};

// Rows of 128 bytes, four lanes to each: 32 words of a row of every lane, `out` where the
// lane's words of the first of its four rows belong, whose first `rows` are there.
template <typename T>
__device__ __forceinline__ void store_rows(T* out, int N, uint32_t (&w)[32], int rows, bool in) {
  rows_across(w);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (s < rows && in) {
      uint32_t v[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) v[n] = w[8 * s + n];
      store32(out, v);
    }
    out += N;
  }
}

// What an epilogue warp carries from tile to tile.
struct Turn {
  int chunk = 0;             // chunks of factors so far
  uint32_t buf = 0, par = 0; // the accumulator that comes next, and its phase
  int stage = 0;             // of the ring, of the blocks that come next (single CTAs)
  bool go = true;            // no wait has run out
};

// The epilogue warps' part of a tile.
template <bool kPair, bool kSplit>
struct Epilogue {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kN = 128 * kCtas;
  static constexpr int kHand = kPair ? 1 : 2;  // blocks handed over at once
  // Its way through a tile's blocks.
  struct Walk : Turn {
    const MmParams& p;
    const Smem sm;
    // Of this lane's waits: it skips them once one has run out, and the warp
    // leaves together before the next factors.
    bool ok = true;
    const float* factors = nullptr;
    __device__ __forceinline__ Walk(const MmParams& p_, Smem s, Turn t) : Turn(t), p(p_), sm(s) {}
    __device__ __forceinline__ bool first_lane() const { return (threadIdx.x & 31) == 0; }
    // The next blocks' factors are at `factors`.
    __device__ __forceinline__ bool next_factors() {
      ok = ok && mbar_wait(sm.ffull(chunk & 1), (chunk >> 1) & 1, p.status);
      go = __all_sync(0xffffffffu, ok);
      factors = sm.factors(chunk & 1);
      return go;
    }
    // The next block's sums are in accumulator `buf`.
    __device__ __forceinline__ void next() {
      // (one answer for the warp: no branch that lanes could take apart)
      if (!__all_sync(0xffffffffu, mbar_try_wait(sm.tfull(buf), par)))
        ok = __all_sync(0xffffffffu, ok && mbar_wait(sm.tfull(buf), par, p.status));
      tc_fence_after();
      if (!kPair) {  // the tensor core is through with the stage's operands
        arrive_if(threadIdx.x == 128, sm.empty(stage));
        if (++stage == p.stages) stage = 0;
      }
    }
    // The accumulator has been read (nothing else is handed over).
    __device__ __forceinline__ void release() {
      tc_fence_before();
      if (kPair) arrive_leader_if(first_lane(), sm.tempty(buf));
      else arrive_if(first_lane(), sm.tempty(buf));
      par ^= buf;
      buf ^= 1;
    }
    // So have the factors.
    __device__ __forceinline__ void release_factors() {
      __syncwarp();
      arrive_if(first_lane(), sm.fempty(chunk & 1));
      ++chunk;
    }
    __device__ __forceinline__ Turn done() {
      go = __all_sync(0xffffffffu, ok);
      return *this;
    }
  };

  // A tile that this warp has no part of.
  static __device__ __forceinline__ Turn idle(const MmParams& p, Smem sm, Turn turn) {
    Walk walk(p, sm, turn);
    for (int kb = 0; kb < sm.blocks<kSplit>(p); kb += kChunk) {
      if (!walk.next_factors()) break;
      for (int j = 0; j < min(kChunk, sm.blocks<kSplit>(p) - kb); j += kHand) {
        walk.next();
        walk.release();
      }
      walk.release_factors();
    }
    return walk.done();
  }

  // A wide tile: a thread has a row and the columns of one weight block.
  static __device__ __forceinline__ Turn wide(const MmParams& p, Smem sm, uint32_t tmem_base, int rank,
                                              const Tile& t, Turn turn) {
    const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, group = (threadIdx.x >> 7) - 1;
    const uint32_t tm0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + group * 128;
    uint64_t sum2[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) sum2[j] = 0;
    // where the tile lies, a lane each: a register, where the sums need nearly all of them
    int place = lane == 0 ? t.row : lane == 1 ? t.left : t.n * kN + group * 128;
    asm volatile("" : "+r"(place));
    Walk walk(p, sm, turn);
    for (int kb = 0; kb < sm.blocks<kSplit>(p); kb += kChunk) {
      if (!walk.next_factors()) break;
      const float* factor = walk.factors + group * 128 + quad * 32 + lane;
      const float* const end = factor + 256 * min(kChunk, sm.blocks<kSplit>(p) - kb);
#pragma unroll 1
      for (; factor != end; factor += 256) {
        walk.next();
        const float f = *factor;
        const uint32_t tm = tm0 + walk.buf * 256;
        uint64_t ff;
        asm("mov.b64 %0, {%1, %1};" : "=l"(ff) : "r"(__float_as_uint(f)));
#pragma unroll
        for (int q = 0; q < 128; q += 64) {
          uint32_t a[64];
          tmem_ld_64(tm + q, a);
          if (q == 64) walk.release();
#pragma unroll
          for (int n = 0; n < 64; n += 2) fma2(sum2[(q + n) / 2], a[n], a[n + 1], ff);
        }
      }
      walk.release_factors();
    }
    turn = walk.done();
    float sum[128];
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      sum[2 * j] = __uint_as_float(static_cast<uint32_t>(sum2[j]));
      sum[2 * j + 1] = __uint_as_float(static_cast<uint32_t>(sum2[j] >> 32));
    }
    const int row = __shfl_sync(0xffffffffu, place, 0), rows = __shfl_sync(0xffffffffu, place, 1);
    const int r0 = rank * 128 + quad * 32, col = __shfl_sync(0xffffffffu, place, 2);
    const int ncols = min(128, p.N - col);
    if (turn.go) {
      // Four lanes store 128 bytes of a row (a store to 32 rows takes the load and store
      // unit four times as long as one to eight); columns come in multiples of 16,
      // on 32 bytes.
      const int r = r0 + (lane & ~3), part = lane & 3;
      const long at = static_cast<long>(row + r) * p.N + col;
      if (p.f32) {
#pragma unroll
        for (int j = 0; j < 128; j += 32) {
          if (j >= ncols) continue;
          uint32_t w[32];
#pragma unroll
          for (int n = 0; n < 32; ++n) w[n] = __float_as_uint(sum[j + n]);
          store_rows(static_cast<float*>(p.out) + at + j + 8 * part, p.N, w, rows - r,
                     j + 8 * part < ncols);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 128; j += 64) {
          if (j >= ncols) continue;
          uint32_t w[32];
#pragma unroll
          for (int n = 0; n < 32; ++n) w[n] = pack_bf16(sum[j + 2 * n], sum[j + 2 * n + 1]);
          store_rows(static_cast<uint16_t*>(p.out) + at + j + 16 * part, p.N, w, rows - r,
                     j + 16 * part < ncols);
        }
      }
    }
    return turn;
  }

  // A narrow tile: a thread has a column and kParts of every other 32 rows.
  template <int kParts>
  static __device__ __forceinline__ Turn narrow(const MmParams& p, Smem sm, uint32_t tmem_base,
                                                int rank, const Tile& t, Turn turn) {
    const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, group = (threadIdx.x >> 7) - 1;
    const uint32_t tm0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + group * 32;
    float sum[32 * kParts];
#pragma unroll
    for (int j = 0; j < 32 * kParts; ++j) sum[j] = 0.f;
    Walk walk(p, sm, turn);
    int left = 0;  // blocks whose factors are there
    for (int kb = 0; kb < sm.blocks<kSplit>(p); kb += kHand) {
      if (left == 0) {
        if (!walk.next_factors()) break;
        left = min(kChunk, sm.blocks<kSplit>(p) - kb);
      }
      walk.next();
      const uint32_t tm = tm0 + walk.buf * 256;
      const int blocks = min(kHand, sm.blocks<kSplit>(p) - kb);
      uint32_t a[kHand][kParts][32];
#pragma unroll
      for (int h = 0; h < kHand; ++h) {  // (a second block that is not there is not used)
#pragma unroll
        for (int q = 0; q < kParts; ++q) tmem_ld_32x32b_x32(tm + 128 * h + 64 * q, a[h][q]);
      }
#pragma unroll
      for (int h = 0; h < kHand; ++h) {
#pragma unroll
        for (int q = 0; q < kParts; ++q) tmem_ld_wait_for(a[h][q]);
      }
      walk.release();
#pragma unroll
      for (int h = 0; h < kHand; ++h) {
        if (h < blocks) {
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            const float4* f =
                reinterpret_cast<const float4*>(walk.factors + 256 * h + 64 * q + 32 * group);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const float4 f4 = f[n];
              float* s = sum + 32 * q + 4 * n;
              s[0] = fmaf(__uint_as_float(a[h][q][4 * n]), f4.x, s[0]);
              s[1] = fmaf(__uint_as_float(a[h][q][4 * n + 1]), f4.y, s[1]);
              s[2] = fmaf(__uint_as_float(a[h][q][4 * n + 2]), f4.z, s[2]);
              s[3] = fmaf(__uint_as_float(a[h][q][4 * n + 3]), f4.w, s[3]);
            }
          }
        }
      }
      walk.factors += 256 * blocks;
      left -= blocks;
      if (left == 0) walk.release_factors();
    }
    turn = walk.done();
    if (kSplit) {  // for the join, in the ring (this tile is the CTA's last)
      float* part = reinterpret_cast<float*>(sm.base) + quad * 32 + lane;
#pragma unroll
      for (int j = 0; j < 32 * kParts; ++j)
        part[(group * 32 + (j / 32) * 64 + j % 32) * 128] = sum[j];
      return turn;
    }
    const int col = t.n * kN + rank * 128 + quad * 32 + lane;
    if (turn.go && col < p.N) {
      const long step = opaque(p.N);
      long at = static_cast<long>(t.row + group * 32) * step + col;
#pragma unroll
      for (int j = 0; j < 32 * kParts; ++j) {
        if (group * 32 + (j / 32) * 64 + j % 32 < t.left) {
          if (p.f32) static_cast<float*>(p.out)[at] = sum[j];
          else from_float(static_cast<Bf16*>(p.out)[at], sum[j]);
        }
        at += j == 31 ? 33 * step : step;
      }
    }
    return turn;
  }

  static __device__ __forceinline__ Turn tile(const MmParams& p, Smem sm, uint32_t tmem_base, int rank,
                                              const Tile& t, Turn turn) {
    const int quad = (threadIdx.x >> 5) & 3, group = (threadIdx.x >> 7) - 1;
    if (kPair && !t.narrow) {
      if (rank * 128 + quad * 32 >= t.left || t.n * kN + group * 128 >= p.N)
        return idle(p, sm, turn);
      return wide(p, sm, tmem_base, rank, t, turn);
    }
    const int parts = ((t.left + 31) / 32 - group + 1) / 2;  // 32s of rows
    if (parts <= 0 || t.n * kN + rank * 128 + quad * 32 >= p.N) return idle(p, sm, turn);
    return parts == 1 ? narrow<1>(p, sm, tmem_base, rank, t, turn)
                      : narrow<2>(p, sm, tmem_base, rank, t, turn);
  }
};

// kSplit (single CTAs): the CTAs of a cluster share one tile along K.
template <bool kPair, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
fp8_matmul_kernel(const __grid_constant__ Maps maps, const __grid_constant__ MmParams p) {
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int kN = 128 * kCtas;           // columns of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sW = smem;  // [stage][2 planes]
  uint8_t* sX = smem + p.stages * 2 * kPlane;
  static_assert(!(kPair && kSplit), "pairs have whole tiles");
  // the blocks of K, whole stages of them, that are this CTA's
  const int split = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
  const int all = (p.kblocks + 1) / 2;
  const int kb0 = kSplit ? all * split / p.splits * 2 : 0;
  const Smem sm{smem, kSplit ? min(p.kblocks, all * (split + 1) / p.splits * 2) - kb0 : 0};
  volatile int* abort_flag = sm.abort_flag();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(sm.full(s), 1);
      mbar_init(sm.empty(s), 2);  // either issuer, or one and the epilogue
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sm.tfull(b), 1);
      mbar_init(sm.tempty(b), kCtas * kEpiWarps);  // one arrival per epilogue warp
      mbar_init(sm.ffull(b), 1);
      mbar_init(sm.fempty(b), kEpiWarps);
      mbar_init(sm.drain(b), 1);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane < kBoxes + 1)
    prefetch_tensormap(lane < kBoxes ? &maps.x[lane] : &maps.w);
  if (warp == 1) {
    if (kPair) pair::tmem_alloc2<512>(sm.tmem_slot());
    else tmem_alloc<512>(sm.tmem_slot());
  }
  // nothing above touches global memory
  pdl_enter();
  const int total = build_tiles(p, sm.off(), sm.tile());
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();  // both CTAs' barriers exist before anything signals them
  tc_fence_after();
  const uint32_t tmem_base = *sm.tmem_slot();
  const int group_ctas = kPair ? 2 : kSplit ? p.splits : 1;
  const int first = static_cast<int>(blockIdx.x) / group_ctas;
  const int step = static_cast<int>(gridDim.x) / group_ctas;

  if (warp < 4) {
    regs_down<Regs<kSplit>::kOther>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- producer
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      Tile t;
      bool ok = true;
      for (int i = first; ok && i < total && !*abort_flag; i += step) {
        t.at<kPair>(i, p, sm.off(), sm.tile());
        const int row = t.row + rank * (t.narrow ? t.half : 128);
        const int col = (t.n * kCtas + rank) * 128;
        const uint32_t plane = t.x_plane(), bytes = kCtas * 2 * (kPlane + plane);
        const CUtensorMap* map = &maps.x[t.box];
        for (int kb = 0; kb < sm.blocks<kSplit>(p); kb += 2) {
          if (!mbar_wait(sm.empty(stage), phase ^ 1, p.status)) { ok = false; break; }
          if (leader) mbar_arrive_expect_tx(sm.full(stage), bytes);
          load_w<kPair>(sW + stage * 2 * kPlane, &maps.w, p.planes, kb0 + kb, col, t.e, kPlane, sm.full(stage),
                        pol);
          load_x<kPair>(sX + stage * p.x_stage, map, p.planes, kb0 + kb, row, plane, sm.full(stage), pol);
          ++issued;
          if (++stage == p.stages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) *abort_flag = 1;
      // no bulk copy left in flight (a pair's complete on the leader's barriers)
      for (int i = 1; leader && i <= p.stages && i <= issued; ++i) {
        int s = stage - i;
        uint32_t ph = phase;
        if (s < 0) { s += p.stages; ph ^= 1; }
        mbar_wait(sm.full(s), ph, p.status);
      }
    } else if ((warp == 1 || warp == 2) && leader && lane == 0) {
      // -------------------------------------------------------------- MMA issuers
      // What is handed to the epilogue at once, a block, or of single CTAs the two of
      // a stage (each in columns of its own: a commit, some 100 cycles in which the
      // tensor core stands still, is then one for both), alternates between the
      // accumulators, and either issuer has one of them: what one thread needs to
      // wait, issue and commit for a block (some 800 cycles) is more than the block
      // takes the tensor core.
      const int mine = warp - 1;
      const uint32_t d = tmem_base + mine * 256;
      int stage = 0;
      uint32_t phase = 0;
      int seg = 0;  // hand-overs so far
      Tile t;
      bool ok = true;
      for (int i = first; ok && i < total && !*abort_flag; i += step) {
        t.at<kPair>(i, p, sm.off(), sm.tile());
        const uint32_t plane = t.x_plane();
        const uint32_t idesc = idesc_e4m3(128 * kCtas, t.narrow ? kCtas * t.half : kN);
        for (int kb = 0; kb < sm.blocks<kSplit>(p); kb += 2) {
          const int blocks = min(2, sm.blocks<kSplit>(p) - kb), units = kPair ? blocks : 1;
          const int u = (seg ^ mine) & 1;  // this issuer's of the stage's units, if it has one
          if (!mbar_wait(sm.full(stage), phase, p.status)) { ok = false; break; }
          // A stage is empty when the tensor core is through with it and both issuers
          // have seen it full (one that came to it when it was full again would take
          // it for not filled yet).  Pairs: both commit to it.  Single CTAs: the
          // epilogue tells, and so does the issuer that has not the stage.
          if (!kPair && u != 0) mbar_arrive(sm.empty(stage));
          if (u < units) {
            if (!mbar_wait(sm.tempty(mine), (((seg + u) >> 1) & 1) ^ 1, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            for (int h = kPair ? u : 0; h < (kPair ? u + 1 : blocks); ++h) {
              const uint64_t w = sw128_kmajor_desc(smem_u32(sW + (stage * 2 + h) * kPlane));
              const uint64_t x = sw128_kmajor_desc(smem_u32(sX + stage * p.x_stage + h * plane));
              const uint64_t a = t.narrow ? w : x, b = t.narrow ? x : w;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_e4m3<kPair>(d + (kPair ? 0 : h * 128), a + 2 * kk, b + 2 * kk, idesc, kk != 0);
            }
            if (kPair) pair::commit_both(sm.tfull(mine));
            else mma_commit(sm.tfull(mine));
          }
          if (kPair) pair::commit_both(sm.empty(stage));
          seg += units;
          if (++stage == p.stages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) *abort_flag = 1;
      if (kPair) pair::commit_local(sm.drain(mine));  // every MMA done before TMEM is released
      else mma_commit(sm.drain(mine));
      mbar_wait(sm.drain(mine), 0, p.status);
    } else if (warp == 3) {
      // -------------------------------------------------------------- factors
      // x_scale * w_scale of every block and row, ahead of the epilogue (whose own
      // loads, a row to a lane, would each touch 32 sectors): of a wide tile for both
      // of its weight blocks, of a narrow one for this CTA's.
      int chunk = 0;
      Tile t;
      bool ok = true;
      for (int i = first; ok && i < total; i += step) {
        if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
        t.at<kPair>(i, p, sm.off(), sm.tile());
        const int row0 = t.row + (t.narrow ? 0 : rank * 128);
        const int rows = t.narrow ? t.left : t.left - rank * 128;
        const int nb = min(t.n * kCtas + (t.narrow ? rank : 0), p.nblocks - 1);
        const float* ws = p.ws + (static_cast<long>(t.e) * p.nblocks + nb) * p.kblocks + kb0;
        const long second = nb + 1 < p.nblocks ? p.kblocks : 0;  // the next weight block's
        for (int kb = 0; ok && kb < sm.blocks<kSplit>(p); kb += kChunk, ++chunk) {
          const int buf = chunk & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(sm.fempty(buf), ((chunk >> 1) & 1) ^ 1, p.status));
          if (!ok) break;
          float* out = sm.factors(buf);
          const int n = min(kChunk, sm.blocks<kSplit>(p) - kb);
          // lane j of eight has block j's weight scales
          const int j8 = lane & 7;
          const float w0 = j8 < n ? __ldg(ws + kb + j8) : 0.f;
          const float w1 = !t.narrow && j8 < n ? __ldg(ws + second + kb + j8) : 0.f;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            if (32 * q >= rows && q > 0) break;  // rows that nothing uses
            const int r = 32 * q + lane;
            const float* xs = p.xs + (static_cast<long>(row0) + r) * p.kblocks + kb0 + kb;
            float x[kChunk];
#pragma unroll
            for (int j = 0; j < kChunk; ++j) x[j] = r < rows && j < n ? __ldg(xs + j) : 0.f;
#pragma unroll
            for (int j = 0; j < kChunk; ++j) {
              out[(2 * j) * 128 + r] = x[j] * __shfl_sync(0xffffffffu, w0, j);
              if (kPair) out[(2 * j + 1) * 128 + r] = x[j] * __shfl_sync(0xffffffffu, w1, j);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(sm.ffull(buf));
        }
      }
      if (!ok && lane == 0) *abort_flag = 1;
    }
    __syncwarp();
    if (kSplit) {  // with the epilogue's below
      cluster_sync();
      cluster_sync();
    }
  } else {
    regs_up<Regs<kSplit>::kEpilogue>();
    // ---------------------------------------------------------------- epilogue
    Turn turn;
    int e = 0;
    for (int i = first; turn.go && i < total; i += step) {
      if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
      Tile t;
      t.e = e;
      t.at<kPair>(i, p, sm.off(), sm.tile());
      e = t.e;
      turn = Epilogue<kPair, kSplit>::tile(p, sm, tmem_base, rank, t, turn);
      if (!turn.go && lane == 0) *abort_flag = 1;
    }
    __syncwarp();
    if (kSplit) {
      // Every CTA of the cluster has its part of the tile's sums in its ring; each adds
      // every so manieth row of them up, in the order of K.
      cluster_sync();
      if (first < total) {
        Tile t;
        t.at<kPair>(first, p, sm.off(), sm.tile());
        // a warp has a row at a time, a lane four columns; four rows are on their way
        constexpr int kRows = 4;
        const int col = t.n * 128 + 4 * lane;
        const uint32_t part = smem_u32(sm.base) + 16 * lane;
        for (int r0 = split + p.splits * (warp - 4); r0 < t.left; r0 += kRows * kEpiWarps * p.splits) {
          float v[kRows][4] = {};
#pragma unroll 2
          for (int s = 0; s < p.splits; ++s) {
            const uint32_t from = pair::mapa(part, s);
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
              const int r = r0 + u * kEpiWarps * p.splits;
              if (r < t.left) add_cluster(v[u], from + r * 512);
            }
          }
#pragma unroll
          for (int u = 0; u < kRows; ++u) {
            const int r = r0 + u * kEpiWarps * p.splits;
            const long at = static_cast<long>(t.row + r) * p.N + col;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (r < t.left && col + j < p.N) {
                if (p.f32) static_cast<float*>(p.out)[at + j] = v[u][j];
                else from_float(static_cast<Bf16*>(p.out)[at + j], v[u][j]);
              }
            }
          }
        }
      }
      cluster_sync();  // no CTA's shared memory goes before it has been read
    }
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

// Rows of a tile: 64 or 128, narrow ones of single CTAs, or 256, wide ones of
// pairs (whose rows of out have to lie on 32 bytes).
//
// A block takes a CTA about 0.2 us (its weights' 16 KB at the rate of HBM, and less
// from L2) and 1.9 ns a row of the tile, a pair 0.5 us for a wide tile; the fewest
// waves of those are the shortest, and of 64 and 128 rows in as many tiles 64 leave
// room for a stage more.  With 64, 128 and 256 rows, us: N=4096 K=7168 of 256 experts by
// popularity, M=2048 886, 925, 918; M=16384 1468, 1413, 1299 (all experts alike 1268, 1213,
// 1248: the rows of each are not known here); M=32768 2026, 1817, 1533.  M=4096 E=8 N=4096
// K=4096 128, 107, 75; M=300 E=1 N=2048 K=2048 9.3, 11.8, 13.7; M=600 13.8, 12.4, 13.9; M=256
// E=1 N=8192 K=8192 36.1, 30.9, 31.8; M=384 51, 55, 35.
int rows_of_tile(const moe_fp8_problem* p, bool wide) {
  const long groups = std::min(p->E, p->M), mean = ceil_div(p->M, groups);
  int best = 0;
  double least = 0;
  for (int rows = 64; rows <= (wide ? 256 : 128); rows *= 2) {
    const int ctas = rows == 256 ? 2 : 1;
    // experts of very different sizes end half a tile behind a whole one
    const double tall = p->E == 1        ? ceil_div(p->M, rows)
                        : 2 * mean <= rows ? static_cast<double>(groups)
                                           : static_cast<double>(p->M) / rows + 0.5 * groups;
    const double tiles = tall * ceil_div(p->N, 128 * ctas);
    const double waves = std::max(1.0, std::ceil(tiles / std::max(1, num_sms() / ctas)));
    const double t = waves * (rows == 256 ? 0.5 : 0.2 + 0.0019 * std::min<long>(rows, mean));
    if (best == 0 || t < least) best = rows, least = t;
  }
  return best;
}

// Tiles at most, whatever the offsets.
long most_tiles(const moe_fp8_problem* p, int rows, int n_tiles) {
  return (ceil_div(p->M, rows) + (p->E == 1 ? 0L : std::min(p->E, p->M))) * n_tiles;
}

// CTAs that share a tile along K: two where the tiles leave at least as many SMs idle
// as they take, four where they leave three times as many (clusters of four do not
// fill every GPC: of five sixths of the SMs), each with eight blocks or more.  With
// 1, 2, 4 and 8, us: M=1 N=4096 K=4096 11.6, 9.9, 9.8, 16.0; M=8 N=8192 K=8192 18.2,
// 13.9, 19.2, 25.1; M=1 N=1024 K=8192 17.6, 12.7, 9.7, 9.6; M=60 N=2048 K=4096 12.8,
// 10.8, 9.4, 16.6; M=100 N=1024 K=8192 20.1, 14.9, 11.7, 18.0; M=1 N=2048 K=1024 8.7, 8.5,
// 8.6, 13.3.
int splits_of(long tiles, int kblocks) {
  return 4 * tiles <= num_sms() * 5 / 6 && kblocks >= 32 ? 4 : 2 * tiles <= num_sms() && kblocks >= 16 ? 2 : 1;
}

template <bool kPair>
cudaError_t launch_tiles(const moe_fp8_problem* p, const void* x, const void* w, MmParams& k,
                         cudaStream_t s) {
  constexpr int kCtas = kPair ? 2 : 1;
  Maps maps;
  // boxes up to the rows of a tile, or all rows (the others' maps are not used: copies)
  const int most_rows = std::min(kPair ? 128 : k.tile_rows, p->M);
  for (int i = 0; i < kBoxes; ++i) {
    if (i > 0 && (8 << i) >= most_rows) maps.x[i] = maps.x[i - 1];
    else if (!make_codes_map(&maps.x[i], x, p->K, p->M, 0, k.planes, 16 << i)) return cudaErrorInvalidValue;
  }
  if (!make_codes_map(&maps.w, w, p->K, p->N, p->E, k.planes, 128)) return cudaErrorInvalidValue;
  k.n_tiles = ceil_div(p->N, 128 * kCtas);
  k.x_stage = 2 * kBlk * (kPair ? 128 : k.tile_rows);
  k.stages = static_cast<int>(kRing / (2 * kPlane + k.x_stage));
  const long most = most_tiles(p, k.tile_rows, k.n_tiles);
  k.splits = kPair ? 1 : splits_of(most, k.kblocks);
  const int ctas = kPair ? 2 : k.splits;  // of a tile
  auto kern = k.splits > 1 ? fp8_matmul_kernel<false, true> : fp8_matmul_kernel<kPair, false>;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kSmem));
  if (err != cudaSuccess) return err;
  const int groups = static_cast<int>(std::max(1L, std::min<long>(num_sms() / ctas, most)));
  return launch_kernel(kern, dim3(static_cast<unsigned>(ctas * groups)), dim3(kThreads), kSmem, s, ctas,
                       maps, k);
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
  k.status = static_cast<uint32_t*>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  k.tile_rows = rows_of_tile(p, p->N % 16 == 0 && !off(out, 32));
  k.tile_shift = k.tile_rows == 64 ? 6 : k.tile_rows == 128 ? 7 : 8;
  if ((k.tile_rows == 256 ? launch_tiles<true>(p, x, w, k, s) : launch_tiles<false>(p, x, w, k, s)) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  set_last_launch_count(1);
  return MOE_OK;
}
