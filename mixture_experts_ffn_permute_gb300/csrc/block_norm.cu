// RMS norms after and before a block, fused with the block's gate and the
// residual update, and their backward (moe_block_norm_* of
// include/moe_block.h has the formulas).
//
// Forward, per row: one read of the branch and the residual, kept in
// registers through both row sums (mean y^2, then mean residual_out^2), one
// write of residual_out and normed.  HBM bound: 2 (branch + residual type)
// bytes per element.
//
// Backward, per row, with u = r' / rms(r'), v = y / rms(y), a = dn w_pre':
//   g  = d_residual_out + (a - u mean(a u)) / rms(r')
//   B  = branch_scale g,  c = B gate w_post',  S = sum(c v)
//   d_residual = residual_scale g,  d_branch = (c - v S / H) / rms(y)
//   d_w_pre += dn u,  d_w_post += B gate v,  d_gate += B v w_post'
// The statistics are recomputed (the rows are read anyway): one round of row
// sums gives sum r'^2, sum a r' and sum y^2, a second gives S.  Every thread
// keeps the same columns on all rows of its block, so the column sums over
// tokens are two fp32 accumulators per column in registers; each block
// writes its sums to the workspace and a second kernel adds the blocks' in
// order.  A channel gate shares the accumulator of w_post: with
// A = sum_t B v, d_w_post = gate A and d_gate = w_post' A.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/moe_block.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowwise.cuh"

namespace moe {
namespace {

struct NormParams {
  const void* branch;
  const void* residual;  // forward: residual; backward: residual_out
  WeightPtr w_post, w_pre, gate;
  void* residual_out;
  void* normed;
  const void* d_residual_out;
  const void* d_normed;
  void* d_residual;
  void* d_branch;
  void* d_gate;  // token and element gates
  float* part;   // backward: [blocks][2][part_ld] column sums (w_pre, w_post)
  int part_ld;   // H, or (flat rows, whose column c lies at c + shift) with room for that
  long ld_branch, ld_residual, ld_residual_out, ld_normed;
  int T, H, gate_kind;
  float eps, offset, residual_scale, branch_scale, inv_h;
};

// gate * x for the eight columns of one step
template <bool kWide>
__device__ __forceinline__ void apply_gate(float (&x)[8], const NormParams& p, long row, int v,
                                           int tid, int n, float token_gate) {
  if (p.gate_kind == MOE_GATE_TOKEN) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= token_gate;
  } else if (p.gate_kind != MOE_GATE_NONE) {
    float g[8];
    load_weight8<kWide>(g, p.gate, p.gate_kind == MOE_GATE_ELEMENT ? row * p.H : 0, v, tid, n, p.H);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= g[j];
  }
}

// One row per warp (kWarp) or per block of at most kThreads threads.
template <typename TB, typename TR, int kSteps, int kThreads, bool kWarp, bool kWide>
__global__ void __launch_bounds__(kThreads)
block_norm_fwd_kernel(const NormParams p) {
  pdl_enter();
  __shared__ float s_sum[2][32];
  const int n = kWarp ? 32 : blockDim.x;
  const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const long row = kWarp ? static_cast<long>(blockIdx.x) * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= p.T) return;  // whole warps (kWarp) only
  const bool has_branch = p.branch != nullptr;
  Oct<TB> y[kSteps];
  Oct<TR> r[kSteps];
  const TR* rrow = static_cast<const TR*>(p.residual) + row * p.ld_residual;
  if (has_branch) {
    const TB* yrow = static_cast<const TB*>(p.branch) + row * p.ld_branch;
#pragma unroll
    for (int v = 0; v < kSteps; ++v) load_oct<kWide>(y[v], yrow, v, tid, n, p.H);
  }
#pragma unroll
  for (int v = 0; v < kSteps; ++v) load_oct<kWide>(r[v], rrow, v, tid, n, p.H);

  float x[kSteps][8];  // residual_out, unrounded
  if (has_branch) {
    float scale = p.branch_scale;
    const bool post = p.w_post.p != nullptr;
    if (post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int v = 0; v < kSteps; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] = fmaf(y[v].get(j), y[v].get(j), ss[0]);
      row_sum<kWarp>(ss, s_sum[0]);
      scale *= rsqrtf(fmaf(ss[0], p.inv_h, p.eps));
    }
    const float tg = p.gate_kind == MOE_GATE_TOKEN ? p.gate.at(row) : 1.f;
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      float w[8];
      if (post) {
        load_weight8<kWide>(w, p.w_post, 0, v, tid, n, p.H);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = scale * (w[j] + p.offset);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = scale;
      }
      apply_gate<kWide>(w, p, row, v, tid, n, tg);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[v][j] = fmaf(p.residual_scale, r[v].get(j), w[j] * y[v].get(j));
    }
    TR* orow = static_cast<TR*>(p.residual_out) + row * p.ld_residual_out;
#pragma unroll
    for (int v = 0; v < kSteps; ++v) store_oct<kWide>(x[v], orow, v, tid, n, p.H);
  } else {
#pragma unroll
    for (int v = 0; v < kSteps; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] = r[v].get(j);
  }
  if (!p.normed) return;
  float ss[1] = {0.f};
#pragma unroll
  for (int v = 0; v < kSteps; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      // columns past the row hold zeros of r and y, but 0 * inf of a gate is not 0
      if (oct_col<kWide>(v, j, tid, n) < p.H) ss[0] = fmaf(x[v][j], x[v][j], ss[0]);
  row_sum<kWarp>(ss, s_sum[1]);
  const float rstd = rsqrtf(fmaf(ss[0], p.inv_h, p.eps));
  TB* nrow = static_cast<TB*>(p.normed) + row * p.ld_normed;
#pragma unroll
  for (int v = 0; v < kSteps; ++v) {
    float w[8];
    load_weight8<kWide>(w, p.w_pre, 0, v, tid, n, p.H);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = x[v][j] * rstd * (w[j] + p.offset);
    store_oct<kWide>(w, nrow, v, tid, n, p.H);
  }
}

// Rows blockIdx.x * rows_per_pass + ..., grid-strided; kWarp: eight warps of a
// block each take a row and their column sums are joined at the end.
template <typename TB, typename TR, int kSteps, int kThreads, bool kWarp, bool kWide>
__global__ void __launch_bounds__(kThreads)
block_norm_bwd_kernel(const NormParams p) {
  pdl_enter();
  __shared__ float s_sum[2][3 * 32];
  extern __shared__ float s_cols[];  // kWarp: [8 warps][2][H]
  const int n = kWarp ? 32 : blockDim.x;
  const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int warp = threadIdx.x >> 5;
  const bool has_branch = p.branch != nullptr, post = p.w_post.p != nullptr,
             pre = p.d_normed != nullptr;
  float acc_pre[kSteps][8] = {}, acc_post[kSteps][8] = {};
  int sums = 0;  // the row sums' two buffers alternate
  const long stride = static_cast<long>(gridDim.x) * (kWarp ? 8 : 1);
  for (long row = kWarp ? static_cast<long>(blockIdx.x) * 8 + warp : blockIdx.x; row < p.T;
       row += stride) {
    Oct<TB> y[kSteps], dn[kSteps];
    Oct<TR> r[kSteps], dr[kSteps];
    const TR* rrow = static_cast<const TR*>(p.residual) + row * p.ld_residual_out;
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      if (pre) {
        load_oct<kWide>(r[v], rrow, v, tid, n, p.H);
        load_oct<kWide>(dn[v], static_cast<const TB*>(p.d_normed) + row * p.ld_normed, v, tid, n,
                        p.H);
      }
      if (has_branch)
        load_oct<kWide>(y[v], static_cast<const TB*>(p.branch) + row * p.ld_branch, v, tid, n, p.H);
      if (p.d_residual_out)
        load_oct<kWide>(dr[v], static_cast<const TR*>(p.d_residual_out) + row * p.ld_residual_out,
                        v, tid, n, p.H);
    }
    float s3[3] = {0.f, 0.f, 0.f};  // sum r'^2, sum a r', sum y^2
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      float w[8];
      if (pre) load_weight8<kWide>(w, p.w_pre, 0, v, tid, n, p.H);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (oct_col<kWide>(v, j, tid, n) >= p.H) continue;
        if (pre) {
          const float x = r[v].get(j);
          s3[0] = fmaf(x, x, s3[0]);
          s3[1] = fmaf(dn[v].get(j) * (w[j] + p.offset), x, s3[1]);
        }
        if (post) s3[2] = fmaf(y[v].get(j), y[v].get(j), s3[2]);
      }
    }
    row_sum<kWarp>(s3, s_sum[sums++ & 1]);
    const float rstd = pre ? rsqrtf(fmaf(s3[0], p.inv_h, p.eps)) : 0.f;
    const float mean_au = rstd * s3[1] * p.inv_h;
    const float ystd = post ? rsqrtf(fmaf(s3[2], p.inv_h, p.eps)) : 1.f;
    // g, the gradient of residual_out
    float g[kSteps][8];
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      float w[8];
      if (pre) load_weight8<kWide>(w, p.w_pre, 0, v, tid, n, p.H);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x = p.d_residual_out ? dr[v].get(j) : 0.f;
        if (pre) {
          const float u = r[v].get(j) * rstd, d = dn[v].get(j);
          acc_pre[v][j] = fmaf(d, u, acc_pre[v][j]);
          x = fmaf(rstd, fmaf(-u, mean_au, d * (w[j] + p.offset)), x);
        }
        g[v][j] = x;
      }
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = has_branch ? p.residual_scale * g[v][j] : g[v][j];
      store_oct<kWide>(o, static_cast<TR*>(p.d_residual) + row * p.ld_residual, v, tid, n, p.H);
    }
    if (!has_branch) continue;
    // with k = B * (channel or element gate): c = k w_post' (token gate apart)
    const float tg = p.gate_kind == MOE_GATE_TOKEN ? p.gate.at(row) : 1.f;
    float s1[1] = {0.f};
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      float w[8], k[8];
      if (post) load_weight8<kWide>(w, p.w_post, 0, v, tid, n, p.H);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = post ? w[j] + p.offset : 1.f;
        k[j] = p.branch_scale * g[v][j];
      }
      if (p.gate_kind == MOE_GATE_ELEMENT) {
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = k[j] * (y[v].get(j) * ystd) * w[j];
        const long at = row * p.H;
        if (p.w_post.f32)
          store_oct<kWide>(d, static_cast<float*>(p.d_gate) + at, v, tid, n, p.H);
        else
          store_oct<kWide>(d, static_cast<Bf16*>(p.d_gate) + at, v, tid, n, p.H);
      }
      // the sum over tokens of w_post (token gate: of tg k v; channel: before the gate)
      if (p.gate_kind != MOE_GATE_ELEMENT) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc_post[v][j] = fmaf(tg * k[j], y[v].get(j) * ystd, acc_post[v][j]);
      }
      if (p.gate_kind == MOE_GATE_ELEMENT || p.gate_kind == MOE_GATE_CHANNEL)
        apply_gate<kWide>(k, p, row, v, tid, n, 1.f);
      if (p.gate_kind == MOE_GATE_ELEMENT) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc_post[v][j] = fmaf(k[j], y[v].get(j) * ystd, acc_post[v][j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[v][j] = k[j] * w[j];  // c
        if (oct_col<kWide>(v, j, tid, n) < p.H)
          s1[0] = fmaf(g[v][j], y[v].get(j) * ystd, s1[0]);
      }
    }
    float mean_cv = 0.f;
    if (post || p.gate_kind == MOE_GATE_TOKEN) {
      row_sum<kWarp>(s1, s_sum[sums++ & 1]);
      if (post) mean_cv = s1[0] * p.inv_h;
      if (p.gate_kind == MOE_GATE_TOKEN && tid == 0) {
        if (p.w_post.f32) static_cast<float*>(p.d_gate)[row] = s1[0];
        else from_float(static_cast<Bf16*>(p.d_gate)[row], s1[0]);
      }
    }
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        o[j] = tg * ystd * fmaf(-(y[v].get(j) * ystd), mean_cv, g[v][j]);
      store_oct<kWide>(o, static_cast<TB*>(p.d_branch) + row * p.ld_branch, v, tid, n, p.H);
    }
  }
  if (!p.part) return;
  float* part = p.part + static_cast<long>(blockIdx.x) * 2 * p.part_ld;  // ld = H here
  if (kWarp) {
#pragma unroll
    for (int v = 0; v < kSteps; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = oct_col<kWide>(v, j, tid, n);
        if (c < p.H) {
          s_cols[(warp * 2 + 0) * p.H + c] = acc_pre[v][j];
          s_cols[(warp * 2 + 1) * p.H + c] = acc_post[v][j];
        }
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.H; c += 256) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) t += s_cols[w * 2 * p.H + c];
      part[c] = t;
    }
  } else {
#pragma unroll
    for (int v = 0; v < kSteps; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = oct_col<kWide>(v, j, tid, n);
        if (c < p.H) {
          part[c] = acc_pre[v][j];
          part[p.H + c] = acc_post[v][j];
        }
      }
  }
}

// ------------------------------------------------------------------ streamed rows
// The same rows and sums by blocks that stay on their SM: a block keeps its
// columns' weights in registers and copies the rows to come into shared memory
// (cp.async; rows of wide accesses: every warp its own octets) while it works
// on the present one, so that the two row sums' barriers do not leave HBM
// idle.  The
// phases read their octets from shared memory again rather than hold them,
// and compute in packed pairs of fp32: the backward is otherwise bound by the
// issue of instructions (63 us of a first version with 70 an element at T=4096
// H=4096 bf16; 41 with 40: 201 MB, 30 us at HBM rate).  The forward: T=8192
// H=7168 with an fp32 residual 122 us (705 MB; 104 at HBM rate).
constexpr int kMaxDepth = 4;  // rows in shared memory, the present one among them

// One tensor's part of a row in shared memory.
template <typename T, int kSteps>
__host__ __device__ constexpr uint32_t slot_bytes(int n) {
  return static_cast<uint32_t>(kSteps * n * oct_align<T>());
}

// The two forms of the rows.  kWide: every row starts on an octet (any row
// stride).  Otherwise the rows are dense, of any width, and taken as octets of
// the whole tensor (rowwise.cuh); the blocks' row stride is a multiple of 8, so
// that a block's shift, and with it the columns of a thread, stays the same.
template <bool kWide>
__device__ __forceinline__ int first_col(int v, int tid, int n, int shift) {
  return (v * n + tid) * 8 - (kWide ? 0 : shift);
}
template <bool kWide>
__device__ __forceinline__ int row_shift(int H) {
  return kWide ? 0 : static_cast<int>(static_cast<long>(blockIdx.x) * H & 7);
}

template <typename T, int kSteps, bool kWide>
struct Rows {
  const T* base;
  long ld;
  __device__ __forceinline__ void copy(uint32_t slot, long r, const NormParams& p, int tid, int n,
                                       int shift) const {
    const T* row = base + r * ld;
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      const uint32_t step = slot + v * n * oct_align<T>();
      const int c = first_col<kWide>(v, tid, n, shift);
      if (kWide) oct_copy(step, row, c, tid, p.H);
      else flat_copy(step, row, c, tid, p.H, base + static_cast<long>(p.T) * p.H);
    }
  }
  // for a step inside the row
  __device__ __forceinline__ void read(Oct<T>& o, uint32_t slot, int v, int tid, int n, int H,
                                       int shift) const {
    oct_read(o, slot + v * n * oct_align<T>(), tid);
    if (!kWide) {
      const int c = first_col<kWide>(v, tid, n, shift);
      if (!oct_whole(c, H)) oct_mask(o, c, H);
    }
  }
};
template <bool kWide, typename T>
__device__ __forceinline__ void store_pairs(const Pair (&x)[4], T* row, int c, int H) {
  if (kWide || oct_whole(c, H)) {
    Oct<T> o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.set_pair(i, x[i]);
    o.store(row + c);
  } else {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpair(x[i], f[2 * i], f[2 * i + 1]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j >= 0 && c + j < H) from_float(row[c + j], f[j]);
  }
}
// Makes the present row readable and starts the copy of the row that takes the
// place of the one before it.
template <typename F>
__device__ __forceinline__ void next_row(int depth, F&& fetch_next) {
  __syncwarp();  // the slot that is filled now has been read by the whole warp
  fetch_next();
  copy_async_wait(depth - 1);
  __syncwarp();
}

// scale * (weight + offset), times the gate's channel where that is its kind,
// of this thread's columns
template <bool kWide>
__device__ __forceinline__ void load_weights(Pair (&w)[4], const NormParams& p,
                                             const WeightPtr& ptr, bool gated, float scale, int c) {
  float x[8];
  if (ptr.p) {
    load_weight_cols(x, ptr, 0, c, p.H, kWide);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = scale * (x[j] + p.offset);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = scale;
  }
  if (gated && p.gate_kind == MOE_GATE_CHANNEL) {
    float g[8];
    load_weight_cols(g, p.gate, 0, c, p.H, kWide);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= g[j];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pair_of(x[2 * i], x[2 * i + 1]);
}

__device__ __forceinline__ void load_gate(Pair (&w)[4], const NormParams& p, long row, int c) {
  float x[8];
  load_weight_cols(x, p.gate, row * p.H, c, p.H, true);  // octets of the tensor in both forms
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pair_of(x[2 * i], x[2 * i + 1]);
}

// kPlain: branch, w_post and w_pre given, no gate or a channel gate; the
// general form decides by the row.
template <typename TB, typename TR, int kSteps, bool kPlain, bool kWide>
__global__ void __launch_bounds__(1024 / kSteps, 1)
block_norm_fwd_stream_kernel(const NormParams p, int depth) {
  pdl_enter();
  __shared__ float s_sum[2][32];
  extern __shared__ __align__(16) uint8_t s_rows[];
  const int tid = threadIdx.x, n = blockDim.x;
  const uint32_t at_r = slot_bytes<TB, kSteps>(n);
  const uint32_t row_bytes = at_r + slot_bytes<TR, kSteps>(n), ring = smem_u32(s_rows);
  const Rows<TB, kSteps, kWide> rows_y{static_cast<const TB*>(p.branch), p.ld_branch};
  const Rows<TR, kSteps, kWide> rows_r{static_cast<const TR*>(p.residual), p.ld_residual};
  const bool has_branch = kPlain || p.branch != nullptr;
  const bool post = kPlain || p.w_post.p != nullptr, pre = kPlain || p.normed != nullptr;
  const bool token = !kPlain && p.gate_kind == MOE_GATE_TOKEN;
  const bool element = !kPlain && p.gate_kind == MOE_GATE_ELEMENT;
  const int shift = row_shift<kWide>(p.H);
  bool in[kSteps];  // steps inside the row
#pragma unroll
  for (int v = 0; v < kSteps; ++v) in[v] = oct_inside(first_col<kWide>(v, tid, n, shift), p.H);
  auto fetch = [&](long row, int slot) {
    if (row < p.T) {
      const uint32_t at = ring + slot * row_bytes;
      if (has_branch) rows_y.copy(at, row, p, tid, n, shift);
      rows_r.copy(at + at_r, row, p, tid, n, shift);
    }
    copy_async_commit();
  };
  const long stride = gridDim.x;
  for (int i = 0; i < depth - 1; ++i) fetch(blockIdx.x + i * stride, i);
  Pair w_post[kSteps][4], w_pre[kSteps][4];
#pragma unroll
  for (int v = 0; v < kSteps; ++v) {
    load_weights<kWide>(w_post[v], p, p.w_post, true, p.branch_scale,
                        first_col<kWide>(v, tid, n, shift));
    load_weights<kWide>(w_pre[v], p, p.w_pre, false, 1.f, first_col<kWide>(v, tid, n, shift));
  }
  const Pair rscale = pair_of(p.residual_scale, p.residual_scale);
  int slot = 0, sums = 0;  // the row sums' two buffers alternate
  for (long row = blockIdx.x; row < p.T; row += stride) {
    next_row(depth, [&]() {
      fetch(row + (depth - 1) * stride, slot == 0 ? depth - 1 : slot - 1);
    });
    const uint32_t at = ring + slot * row_bytes;
    slot = slot + 1 == depth ? 0 : slot + 1;
    Pair x[kSteps][4];  // residual_out, unrounded
    if (has_branch) {
      float scale = token ? p.gate.at(row) : 1.f;
      if (post) {
        Pair acc = 0;
#pragma unroll
        for (int v = 0; v < kSteps; ++v) {
          if (!in[v]) continue;
          Oct<TB> y;
          rows_y.read(y, at, v, tid, n, p.H, shift);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc = pair_fma(y.pair(i), y.pair(i), acc);
        }
        float ss[1] = {pair_sum(acc)};
        row_sum<false>(ss, s_sum[sums++ & 1]);
        scale *= rsqrtf(fmaf(ss[0], p.inv_h, p.eps));
      }
      const Pair sc = pair_of(scale, scale);
      TR* orow = static_cast<TR*>(p.residual_out) + row * p.ld_residual_out;
#pragma unroll
      for (int v = 0; v < kSteps; ++v) {
        if (!in[v]) continue;
        Oct<TB> y;
        Oct<TR> r;
        rows_y.read(y, at, v, tid, n, p.H, shift);
        rows_r.read(r, at + at_r, v, tid, n, p.H, shift);
        Pair w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pair_mul(sc, w_post[v][i]);
        if (element) {
          Pair g[4];
          load_gate(g, p, row, first_col<kWide>(v, tid, n, shift));
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pair_mul(w[i], g[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[v][i] = pair_fma(rscale, r.pair(i), pair_mul(w[i], y.pair(i)));
        }
        store_pairs<kWide>(x[v], orow, first_col<kWide>(v, tid, n, shift), p.H);
      }
    } else {
#pragma unroll
      for (int v = 0; v < kSteps; ++v) {
        if (!in[v]) continue;
        Oct<TR> r;
        rows_r.read(r, at + at_r, v, tid, n, p.H, shift);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[v][i] = r.pair(i);
      }
    }
    if (!pre) continue;
    Pair acc = 0;
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      if (!in[v]) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = pair_fma(x[v][i], x[v][i], acc);
    }
    float ss[1] = {pair_sum(acc)};
    row_sum<false>(ss, s_sum[sums++ & 1]);
    const float rstd = rsqrtf(fmaf(ss[0], p.inv_h, p.eps));
    const Pair rs = pair_of(rstd, rstd);
    TB* nrow = static_cast<TB*>(p.normed) + row * p.ld_normed;
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      if (!in[v]) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[v][i] = pair_mul(x[v][i], pair_mul(rs, w_pre[v][i]));
      store_pairs<kWide>(x[v], nrow, first_col<kWide>(v, tid, n, shift), p.H);
    }
  }
  copy_async_wait(0);
}

// kPlain: every input given, no gate or a channel gate.
template <typename TB, typename TR, int kSteps, bool kPlain, bool kWide>
__global__ void __launch_bounds__(1024 / kSteps, 1)
block_norm_bwd_stream_kernel(const NormParams p, int depth) {
  pdl_enter();
  __shared__ float s_sum[2][3 * 32];
  extern __shared__ __align__(16) uint8_t s_rows[];
  const int tid = threadIdx.x, n = blockDim.x;
  const uint32_t bb = slot_bytes<TB, kSteps>(n);
  const uint32_t rb = slot_bytes<TR, kSteps>(n);
  const uint32_t row_bytes = 2 * (bb + rb), ring = smem_u32(s_rows);
  // a row's parts in shared memory
  const uint32_t at_y = 0, at_dn = bb, at_r = 2 * bb, at_dr = at_r + rb;
  const Rows<TB, kSteps, kWide> rows_y{static_cast<const TB*>(p.branch), p.ld_branch};
  const Rows<TB, kSteps, kWide> rows_dn{static_cast<const TB*>(p.d_normed), p.ld_normed};
  const Rows<TR, kSteps, kWide> rows_r{static_cast<const TR*>(p.residual), p.ld_residual_out};
  const Rows<TR, kSteps, kWide> rows_dr{static_cast<const TR*>(p.d_residual_out),
                                        p.ld_residual_out};
  const bool has_branch = kPlain || p.branch != nullptr, post = kPlain || p.w_post.p != nullptr;
  const bool pre = kPlain || p.d_normed != nullptr, later = kPlain || p.d_residual_out != nullptr;
  const bool token = !kPlain && p.gate_kind == MOE_GATE_TOKEN;
  const bool element = !kPlain && p.gate_kind == MOE_GATE_ELEMENT;
  const int shift = row_shift<kWide>(p.H);
  bool in[kSteps];  // steps inside the row
#pragma unroll
  for (int v = 0; v < kSteps; ++v) in[v] = oct_inside(first_col<kWide>(v, tid, n, shift), p.H);
  auto fetch = [&](long row, int slot) {
    if (row < p.T) {
      const uint32_t at = ring + slot * row_bytes;
      if (pre) {
        rows_r.copy(at + at_r, row, p, tid, n, shift);
        rows_dn.copy(at + at_dn, row, p, tid, n, shift);
      }
      if (has_branch) rows_y.copy(at + at_y, row, p, tid, n, shift);
      if (later) rows_dr.copy(at + at_dr, row, p, tid, n, shift);
    }
    copy_async_commit();
  };
  const long stride = gridDim.x;
  for (int i = 0; i < depth - 1; ++i) fetch(blockIdx.x + i * stride, i);
  // w_pre', and branch_scale * gate (channel) * w_post'
  Pair w_pre[kSteps][4], w_post[kSteps][4];
  Pair acc_pre[kSteps][4], acc_post[kSteps][4];
#pragma unroll
  for (int v = 0; v < kSteps; ++v) {
    load_weights<kWide>(w_pre[v], p, p.w_pre, false, 1.f, first_col<kWide>(v, tid, n, shift));
    load_weights<kWide>(w_post[v], p, p.w_post, true, p.branch_scale,
                        first_col<kWide>(v, tid, n, shift));
#pragma unroll
    for (int i = 0; i < 4; ++i) acc_pre[v][i] = acc_post[v][i] = 0;
  }
  const float res_scale = has_branch ? p.residual_scale : 1.f;
  const Pair rscale = pair_of(res_scale, res_scale);
  int slot = 0, sums = 0;  // the row sums' two buffers alternate
  for (long row = blockIdx.x; row < p.T; row += stride) {
    next_row(depth, [&]() {
      fetch(row + (depth - 1) * stride, slot == 0 ? depth - 1 : slot - 1);
    });
    const uint32_t at = ring + slot * row_bytes;
    slot = slot + 1 == depth ? 0 : slot + 1;
    Pair a0 = 0, a1 = 0, a2 = 0;  // sum r'^2, sum a r', sum y^2
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      if (!in[v]) continue;
      if (pre) {
        Oct<TR> r;
        Oct<TB> dn;
        rows_r.read(r, at + at_r, v, tid, n, p.H, shift);
        rows_dn.read(dn, at + at_dn, v, tid, n, p.H, shift);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a0 = pair_fma(r.pair(i), r.pair(i), a0);
          a1 = pair_fma(pair_mul(dn.pair(i), w_pre[v][i]), r.pair(i), a1);
        }
      }
      if (post) {
        Oct<TB> y;
        rows_y.read(y, at + at_y, v, tid, n, p.H, shift);
#pragma unroll
        for (int i = 0; i < 4; ++i) a2 = pair_fma(y.pair(i), y.pair(i), a2);
      }
    }
    float s3[3] = {pair_sum(a0), pair_sum(a1), pair_sum(a2)};
    row_sum<false>(s3, s_sum[sums++ & 1]);
    const float rstd = pre ? rsqrtf(fmaf(s3[0], p.inv_h, p.eps)) : 0.f;
    const float ystd = post ? rsqrtf(fmaf(s3[2], p.inv_h, p.eps)) : 1.f;
    // g = dr + rstd a - rstd u mean(a u), u = rstd r': the last factor of r'
    const float kr = -rstd * rstd * (rstd * s3[1] * p.inv_h);
    const Pair rs = pair_of(rstd, rstd), k2 = pair_of(kr, kr), ys = pair_of(ystd, ystd);
    const float tg = token ? p.gate.at(row) : 1.f;
    Pair g[kSteps][4];  // c = gradient of v, without the token gate
    Pair sc = 0;
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      if (!in[v]) continue;
      const int c = first_col<kWide>(v, tid, n, shift);
      if (later) {
        Oct<TR> dr;
        rows_dr.read(dr, at + at_dr, v, tid, n, p.H, shift);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[v][i] = dr.pair(i);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) g[v][i] = 0;
      }
      if (pre) {
        Oct<TR> r;
        Oct<TB> dn;
        rows_r.read(r, at + at_r, v, tid, n, p.H, shift);
        rows_dn.read(dn, at + at_dn, v, tid, n, p.H, shift);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Pair d = pair_mul(dn.pair(i), rs);
          acc_pre[v][i] = pair_fma(d, r.pair(i), acc_pre[v][i]);
          g[v][i] = pair_fma(r.pair(i), k2, pair_fma(d, w_pre[v][i], g[v][i]));
        }
      }
      Pair o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pair_mul(rscale, g[v][i]);
      store_pairs<kWide>(o, static_cast<TR*>(p.d_residual) + row * p.ld_residual, c, p.H);
      if (!has_branch) continue;
      Oct<TB> y;
      rows_y.read(y, at + at_y, v, tid, n, p.H, shift);
      if (element) {
        Pair gate[4];
        load_gate(gate, p, row, c);
        Pair dg[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Pair gv = pair_mul(g[v][i], pair_mul(y.pair(i), ys));
          dg[i] = pair_mul(gv, w_post[v][i]);
          acc_post[v][i] = pair_fma(gv, gate[i], acc_post[v][i]);
          g[v][i] = pair_mul(g[v][i], pair_mul(gate[i], w_post[v][i]));
          sc = pair_fma(g[v][i], pair_mul(y.pair(i), ys), sc);
        }
        if (p.w_post.f32)
          store_pairs<kWide>(dg, static_cast<float*>(p.d_gate) + row * p.H, c, p.H);
        else
          store_pairs<kWide>(dg, static_cast<Bf16*>(p.d_gate) + row * p.H, c, p.H);
      } else {
        const Pair t = pair_of(tg, tg);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Pair vv = pair_mul(y.pair(i), ys);
          acc_post[v][i] = pair_fma(kPlain ? g[v][i] : pair_mul(t, g[v][i]), vv, acc_post[v][i]);
          g[v][i] = pair_mul(g[v][i], w_post[v][i]);
          sc = pair_fma(g[v][i], vv, sc);
        }
      }
    }
    if (!has_branch) continue;
    float mean_cv = 0.f;
    if (post || token) {
      float s1[1] = {pair_sum(sc)};
      row_sum<false>(s1, s_sum[sums++ & 1]);
      if (post) mean_cv = s1[0] * p.inv_h;
      if (token && tid == 0) {
        if (p.w_post.f32) static_cast<float*>(p.d_gate)[row] = s1[0];
        else from_float(static_cast<Bf16*>(p.d_gate)[row], s1[0]);
      }
    }
    // d_branch = gate ystd (c - v mean(c v)), v = ystd y
    const float f = tg * ystd, ky = -f * ystd * mean_cv;
    const Pair fc = pair_of(f, f), fy = pair_of(ky, ky);
#pragma unroll
    for (int v = 0; v < kSteps; ++v) {
      if (!in[v]) continue;
      Oct<TB> y;
      Pair o[4];
      rows_y.read(y, at + at_y, v, tid, n, p.H, shift);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = pair_fma(y.pair(i), fy, pair_mul(g[v][i], fc));
      store_pairs<kWide>(o, static_cast<TB*>(p.d_branch) + row * p.ld_branch,
                         first_col<kWide>(v, tid, n, shift), p.H);
    }
  }
  copy_async_wait(0);
  if (!p.part) return;
  // octets again: what a flat row's first and last ones hold outside it is not read
  float* part = p.part + static_cast<long>(blockIdx.x) * 2 * p.part_ld;
#pragma unroll
  for (int v = 0; v < kSteps; ++v) {
    if (!in[v]) continue;
    float* at = part + (v * n + tid) * 8;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      float a[4], b[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        unpair(acc_pre[v][i + j], a[2 * j], a[2 * j + 1]);
        unpair(acc_post[v][i + j], b[2 * j], b[2 * j + 1]);
      }
      reinterpret_cast<float4*>(at)[i / 2] = make_float4(a[0], a[1], a[2], a[3]);
      reinterpret_cast<float4*>(at + p.part_ld)[i / 2] =
          make_float4(p.branch_scale * b[0], p.branch_scale * b[1], p.branch_scale * b[2],
                      p.branch_scale * b[3]);
    }
  }
}

// Sum of the blocks' column sums: 32 columns of w_pre's (blockIdx.y 0) or w_post's
// x 32 runs of blocks per CTA.
__global__ void __launch_bounds__(1024)
block_norm_cols_kernel(const float* __restrict__ part, int blocks, int H, int ld, int flat,
                       WeightPtr w_post, WeightPtr gate, int channel_gate, float offset,
                       void* d_w_pre, void* d_w_post, void* d_gate) {
  pdl_enter();
  __shared__ float s[32][32];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < H) {
    const float* at = part + static_cast<long>(blockIdx.y) * ld + c;
#pragma unroll 8
    for (int i = q; i < blocks; i += 32) {
      const int shift = flat ? static_cast<int>(static_cast<long>(i) * H & 7) : 0;
      a += at[static_cast<long>(i) * 2 * ld + shift];
    }
  }
  s[q][lane] = a;
  __syncthreads();
  if (q || c >= H) return;
  a = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) a += s[i][lane];
  auto put = [&](void* d, float x) {
    if (!d) return;
    if (w_post.f32) static_cast<float*>(d)[c] = x;
    else from_float(static_cast<Bf16*>(d)[c], x);
  };
  if (blockIdx.y == 0) {
    put(d_w_pre, a);
  } else {
    put(d_w_post, channel_gate ? gate.at(c) * a : a);
    if (channel_gate) put(d_gate, (w_post.p ? w_post.at(c) + offset : 1.f) * a);
  }
}

// How a tensor's rows lie: every row on an octet; dense, the first one on an
// octet; or anyhow.
enum class Lay { kWide, kFlat, kAny };

// Threads and row mapping.
//   - A warp takes a row up to 1024 columns in the forward (32 per lane: the row
//     sums then need no barrier), up to 256 in the backward (its column sums
//     would not fit the registers of more).
//   - Wider rows take a block.  Streamed (wide or flat rows up to 8192 columns):
//     8 columns a thread in the forward, 16 in the backward, whose registers
//     allow 512 threads an SM; all rows of the backward, and of the forward
//     where every SM has several rows to work on.
//   - Otherwise, 8 columns a thread up to 512 threads, else 16.
struct Shape {
  bool warp, stream;
  int steps, threads, per_sm, depth;
};
constexpr int kStreamRows = 4;            // rows per SM from which the forward streams
constexpr int kStreamBytes = 200 * 1024;  // shared memory of an SM for the rings
constexpr int kFwdSteps = 1, kBwdSteps = 2;

// Blocks that T rows are worth: every block of the backward leaves column sums
// to be added, so one for two rows but where that leaves SMs without one.
int stay_rows(int T) { return std::max(std::min(T, num_sms()), ceil_div(T, 2)); }

Shape norm_shape(const moe_norm_problem* p, bool bwd, Lay lay) {
  const int H = p->H;
  if (H <= 256) return {true, false, 1, 256, 2, 0};
  if (!bwd && H <= 1024) return {true, false, H <= 512 ? 2 : 4, 256, 0, 0};
  const int span = H + (lay == Lay::kFlat ? 7 : 0);  // columns with the shift
  if (lay != Lay::kAny && span <= 512 * 16 && (bwd || p->T >= kStreamRows * num_sms())) {
    Shape s{false, true, bwd ? kBwdSteps : kFwdSteps, 0, 0, 0};
    s.threads = ceil_div(ceil_div(span, 8 * s.steps), 32) * 32;
    s.per_sm = std::max(1, 1024 / s.steps / s.threads);
    auto slot = [&](int dtype) {
      return static_cast<int>(dtype == MOE_DTYPE_F32 ? slot_bytes<float, 1>(s.threads)
                                                     : slot_bytes<Bf16, 1>(s.threads)) *
             s.steps;
    };
    const int row = (slot(p->branch_dtype) + slot(p->residual_dtype)) * (bwd ? 2 : 1);
    // two rows in the ring at least, with fewer blocks an SM if need be, but two
    // (fp32 backward: T=4096 H=2048 42.5 us with four blocks of one row, 39.7
    // with three of two; T=8192 H=4096 129 us with two of one, 139 with one of
    // three)
    s.per_sm = std::max(std::min(s.per_sm, 2), std::min(s.per_sm, kStreamBytes / (2 * row)));
    const int used = std::max(1, std::min(s.per_sm, ceil_div(stay_rows(p->T), num_sms())));
    s.depth = std::max(1, std::min(kMaxDepth, kStreamBytes / used / row));
    return s;
  }
  const int steps = H <= 512 * 8 ? 1 : 2;
  const int threads = ceil_div(ceil_div(H, 8 * steps), 32) * 32;
  return {false, false, steps, threads, std::max(1, 512 / threads), 0};
}

// Blocks that stay: what the SMs hold at once, and no more than the rows are
// worth (eight rows a block for the warp form); a multiple of 8 for flat rows.
int norm_blocks(int T, const Shape& s, Lay lay) {
  const int rows = s.warp ? ceil_div(T, 8) : stay_rows(T);
  const int most = std::max(1, std::min(num_sms() * s.per_sm, rows));
  return s.stream && lay == Lay::kFlat ? std::max(8, most / 8 * 8) : most;
}

int elt(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
bool dtype_ok(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }
bool aligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

int check_norm(const moe_norm_problem* p) {
  if (!p || p->T < 0 || p->H < 1) return MOE_ERR_INVALID_ARG;
  if (!dtype_ok(p->branch_dtype) || !dtype_ok(p->residual_dtype) || !dtype_ok(p->weight_dtype))
    return MOE_ERR_INVALID_ARG;
  if (p->gate_kind < MOE_GATE_NONE || p->gate_kind > MOE_GATE_ELEMENT) return MOE_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (p->H > MOE_MAX_NORM_WIDTH) return MOE_ERR_UNSUPPORTED_SHAPE;
  for (const int64_t ld : {p->ld_branch, p->ld_residual, p->ld_residual_out, p->ld_normed})
    if (ld != 0 && (ld < p->H || ld > (1LL << 40))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int part_ld(int H, Lay lay) { return lay == Lay::kFlat ? ceil_div(H + 7, 8) * 8 : H; }

size_t norm_part_bytes(const moe_norm_problem* p) {
  int blocks = 0;  // whichever form the tensors' alignment calls for
  for (const Lay lay : {Lay::kWide, Lay::kFlat, Lay::kAny})
    blocks = std::max(blocks, norm_blocks(p->T, norm_shape(p, true, lay), lay));
  return sizeof(float) * 2 * static_cast<size_t>(part_ld(p->H, Lay::kFlat)) * blocks;
}

constexpr size_t kNormHeader = 256;  // status word

// Collects the pointer checks and how the rows lie.
struct RowCheck {
  bool ok = true, octets = true, dense = true, wide;
  int H;
  explicit RowCheck(int h) : wide(h % 8 == 0), H(h) {}
  void add(const void* p, int dtype, long ld) {
    if (!p) return;
    if (!aligned(p, elt(dtype))) ok = false;
    if (!aligned(p, 8 * elt(dtype))) octets = false;  // eight elements in one access
    if (ld % 8 != 0) wide = false;
    if (ld != H) dense = false;
  }
  Lay lay() const {
    return octets && wide ? Lay::kWide : octets && dense ? Lay::kFlat : Lay::kAny;
  }
};

NormParams norm_params(const moe_norm_problem* p) {
  NormParams k{};
  k.T = p->T;
  k.H = p->H;
  k.gate_kind = p->gate_kind;
  k.eps = p->eps;
  k.offset = p->weight_offset;
  k.residual_scale = p->residual_scale;
  k.branch_scale = p->branch_scale;
  k.inv_h = 1.f / static_cast<float>(p->H);
  k.ld_branch = p->ld_branch ? p->ld_branch : p->H;
  k.ld_residual = p->ld_residual ? p->ld_residual : p->H;
  k.ld_residual_out = p->ld_residual_out ? p->ld_residual_out : p->H;
  k.ld_normed = p->ld_normed ? p->ld_normed : p->H;
  return k;
}

template <bool kBwd, typename TB, typename TR, int kSteps, int kThreads, bool kWarp, bool kWide>
cudaError_t launch_norm_impl(const NormParams& k, int threads, int blocks, cudaStream_t s) {
  if constexpr (kBwd)
    return launch_kernel(block_norm_bwd_kernel<TB, TR, kSteps, kThreads, kWarp, kWide>,
                         dim3(blocks), dim3(threads),
                         kWarp && k.part ? sizeof(float) * 16 * k.H : 0, s, 1, k);
  else
    return launch_kernel(block_norm_fwd_kernel<TB, TR, kSteps, kThreads, kWarp, kWide>,
                         dim3(blocks), dim3(threads), 0, s, 1, k);
}

template <bool kBwd, typename TB, typename TR, bool kWide>
cudaError_t launch_norm_stream(const NormParams& k, const Shape& sh, int blocks, cudaStream_t s) {
  const bool plain = k.branch && k.w_post.p && k.w_pre.p && (!kBwd || k.d_residual_out) &&
                     (k.gate_kind == MOE_GATE_NONE || k.gate_kind == MOE_GATE_CHANNEL);
  constexpr int kSteps = kBwd ? kBwdSteps : kFwdSteps;
  void (*kern)(NormParams, int);
  if constexpr (kBwd)
    kern = plain ? block_norm_bwd_stream_kernel<TB, TR, kSteps, true, kWide>
                 : block_norm_bwd_stream_kernel<TB, TR, kSteps, false, kWide>;
  else
    kern = plain ? block_norm_fwd_stream_kernel<TB, TR, kSteps, true, kWide>
                 : block_norm_fwd_stream_kernel<TB, TR, kSteps, false, kWide>;
  const size_t smem = static_cast<size_t>(sh.depth) * (kBwd ? 2 : 1) *
                      (slot_bytes<TB, kSteps>(sh.threads) + slot_bytes<TR, kSteps>(sh.threads));
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kStreamBytes);
  if (err != cudaSuccess) return err;
  return launch_kernel(kern, dim3(blocks), dim3(sh.threads), smem, s, 1, k, sh.depth);
}

template <bool kBwd, typename TB, typename TR>
cudaError_t launch_norm_shape(const NormParams& k, Lay lay, const Shape& sh, int blocks,
                              cudaStream_t s) {
  const int n = sh.threads;
  if (sh.stream)
    return lay == Lay::kWide ? launch_norm_stream<kBwd, TB, TR, true>(k, sh, blocks, s)
                             : launch_norm_stream<kBwd, TB, TR, false>(k, sh, blocks, s);
  auto go = [&](auto w) {
    constexpr bool kWide = decltype(w)::value;
    if (sh.warp && sh.steps == 1)
      return launch_norm_impl<kBwd, TB, TR, 1, 256, true, kWide>(k, n, blocks, s);
    if constexpr (!kBwd)
      if (sh.warp)
        return sh.steps == 2 ? launch_norm_impl<kBwd, TB, TR, 2, 256, true, kWide>(k, n, blocks, s)
                             : launch_norm_impl<kBwd, TB, TR, 4, 256, true, kWide>(k, n, blocks, s);
    if constexpr (!kBwd || !kWide) {  // the backward streams these where the rows are wide
      if (sh.steps == 1) return launch_norm_impl<kBwd, TB, TR, 1, 512, false, kWide>(k, n, blocks, s);
      if (n <= 512) return launch_norm_impl<kBwd, TB, TR, 2, 512, false, kWide>(k, n, blocks, s);
    }
    return launch_norm_impl<kBwd, TB, TR, 2, 1024, false, kWide>(k, n, blocks, s);
  };
  return lay == Lay::kWide ? go(std::true_type{}) : go(std::false_type{});
}

template <bool kBwd>
cudaError_t launch_norm(const moe_norm_problem* p, const NormParams& k, Lay lay, const Shape& sh,
                        int blocks, cudaStream_t s) {
  const bool bf = p->branch_dtype == MOE_DTYPE_BF16, rf = p->residual_dtype == MOE_DTYPE_BF16;
  if (bf)
    return rf ? launch_norm_shape<kBwd, Bf16, Bf16>(k, lay, sh, blocks, s)
              : launch_norm_shape<kBwd, Bf16, float>(k, lay, sh, blocks, s);
  return rf ? launch_norm_shape<kBwd, float, Bf16>(k, lay, sh, blocks, s)
            : launch_norm_shape<kBwd, float, float>(k, lay, sh, blocks, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_block_norm_forward(const moe_norm_problem* p, const void* branch,
                                      const void* w_post, const void* gate, const void* residual,
                                      const void* w_pre, void* residual_out, void* normed,
                                      void* stream) {
  const int rc = check_norm(p);
  if (rc != MOE_OK) return rc;
  set_last_launch_count(0);
  if (p->T == 0) return MOE_OK;  // tensors without elements may have null pointers
  const bool has_branch = branch != nullptr;
  if (!residual || has_branch != (residual_out != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!has_branch && (w_post || gate || p->gate_kind != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
  if ((gate != nullptr) != (p->gate_kind != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
  if ((w_pre != nullptr) != (normed != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!has_branch && !normed) return MOE_ERR_INVALID_ARG;
  NormParams k = norm_params(p);
  if (residual_out == residual && k.ld_residual != k.ld_residual_out) return MOE_ERR_INVALID_ARG;
  RowCheck c(p->H);
  c.add(branch, p->branch_dtype, k.ld_branch);
  c.add(normed, p->branch_dtype, k.ld_normed);
  c.add(residual, p->residual_dtype, k.ld_residual);
  c.add(residual_out, p->residual_dtype, k.ld_residual_out);
  c.add(w_post, p->weight_dtype, p->H);
  c.add(w_pre, p->weight_dtype, p->H);
  c.add(gate, p->weight_dtype, p->H);
  if (!c.ok) return MOE_ERR_MISALIGNED;
  const bool wf = p->weight_dtype == MOE_DTYPE_F32;
  k.branch = branch;
  k.residual = residual;
  k.w_post = {w_post, wf};
  k.w_pre = {w_pre, wf};
  k.gate = {gate, wf};
  k.residual_out = residual_out;
  k.normed = normed;
  const Shape sh = norm_shape(p, false, c.lay());
  const int blocks = sh.stream ? norm_blocks(p->T, sh, c.lay())
                     : sh.warp ? ceil_div(p->T, 8)
                               : p->T;
  if (launch_norm<false>(p, k, c.lay(), sh, blocks, static_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  set_last_launch_count(1);
  return MOE_OK;
}

extern "C" size_t moe_block_norm_workspace_size(const moe_norm_problem* p) {
  if (check_norm(p) != MOE_OK) return 0;
  return kNormHeader + (norm_part_bytes(p) + 255) / 256 * 256;
}

extern "C" int moe_block_norm_backward(const moe_norm_problem* p, const void* branch,
                                       const void* w_post, const void* gate,
                                       const void* residual_out, const void* w_pre,
                                       const void* d_residual_out, const void* d_normed,
                                       void* d_residual, void* d_branch, void* d_w_post,
                                       void* d_gate, void* d_w_pre, void* ws, size_t ws_bytes,
                                       void* stream) {
  const int rc = check_norm(p);
  if (rc != MOE_OK) return rc;
  if (!ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
  if (ws_bytes < moe_block_norm_workspace_size(p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const bool channel = p->gate_kind == MOE_GATE_CHANNEL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int launches = 0;
  set_last_launch_count(0);
  if (!aligned(d_w_post, elt(p->weight_dtype)) || !aligned(d_w_pre, elt(p->weight_dtype)))
    return MOE_ERR_MISALIGNED;
  if (p->T == 0) {  // no tokens: the weights' gradients are zero
    const size_t n = static_cast<size_t>(p->H) * elt(p->weight_dtype);
    for (void* d : {d_w_post, d_w_pre, channel ? d_gate : nullptr})
      if (d) {
        if (cudaMemsetAsync(d, 0, n, s) != cudaSuccess) return MOE_ERR_CUDA;
        ++launches;
      }
    set_last_launch_count(launches);
    return MOE_OK;
  }
  const bool has_branch = branch != nullptr, pre = w_pre != nullptr;
  if (!d_residual || has_branch != (d_branch != nullptr) || pre != (d_normed != nullptr) ||
      (pre && !residual_out))
    return MOE_ERR_INVALID_ARG;
  if (!has_branch && (w_post || gate || p->gate_kind != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
  if ((gate != nullptr) != (p->gate_kind != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
  if ((d_w_post != nullptr) != (w_post != nullptr) || (d_gate != nullptr) != (gate != nullptr) ||
      (d_w_pre != nullptr) != pre)
    return MOE_ERR_INVALID_ARG;
  if (!has_branch && !pre) return MOE_ERR_INVALID_ARG;
  NormParams k = norm_params(p);
  if (d_residual == d_residual_out && k.ld_residual != k.ld_residual_out)
    return MOE_ERR_INVALID_ARG;
  RowCheck c(p->H);
  c.add(branch, p->branch_dtype, k.ld_branch);
  c.add(d_branch, p->branch_dtype, k.ld_branch);
  c.add(d_normed, p->branch_dtype, k.ld_normed);
  c.add(residual_out, p->residual_dtype, k.ld_residual_out);
  c.add(d_residual_out, p->residual_dtype, k.ld_residual_out);
  c.add(d_residual, p->residual_dtype, k.ld_residual);
  for (const void* w : {w_post, w_pre, gate, static_cast<const void*>(d_gate)})
    c.add(w, p->weight_dtype, p->H);
  if (!c.ok) return MOE_ERR_MISALIGNED;
  const bool wf = p->weight_dtype == MOE_DTYPE_F32;
  k.branch = branch;
  k.residual = residual_out;
  k.w_post = {w_post, wf};
  k.w_pre = {w_pre, wf};
  k.gate = {gate, wf};
  k.d_residual_out = d_residual_out;
  k.d_normed = d_normed;
  k.d_residual = d_residual;
  k.d_branch = d_branch;
  k.d_gate = d_gate;
  const bool cols = pre || w_post || channel;
  k.part = cols ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kNormHeader) : nullptr;
  const Shape sh = norm_shape(p, true, c.lay());
  const int blocks = norm_blocks(p->T, sh, c.lay());
  k.part_ld = part_ld(p->H, sh.stream ? c.lay() : Lay::kAny);
  if (launch_norm<true>(p, k, c.lay(), sh, blocks, s) != cudaSuccess) return MOE_ERR_CUDA;
  ++launches;
  if (cols) {
    const int flat = sh.stream && c.lay() == Lay::kFlat;
    if (launch_kernel(block_norm_cols_kernel, dim3(ceil_div(p->H, 32), 2), dim3(1024), 0, s, 1,
                      static_cast<const float*>(k.part), blocks, p->H, k.part_ld, flat, k.w_post,
                      k.gate, channel ? 1 : 0, p->weight_offset, d_w_pre, d_w_post, d_gate) != cudaSuccess)
      return MOE_ERR_CUDA;
    ++launches;
  }
  set_last_launch_count(launches);
  return MOE_OK;
}
