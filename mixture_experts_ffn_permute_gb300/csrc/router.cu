// Expert router: scores, balance bias, groups, top-k and weights, and its
// backward (moe_router_* of include/moe_experts.h).
//
// One warp per token, the row in registers: lane i holds the experts i N ..
// i N + N - 1 (N the power of two that fits E), so that among equal keys the lowest
// lane, and in it the first, is the lowest id.  A key is the value's bits in an
// order of unsigned integers; a pick is one warp maximum and one ballot.
//
// The order is that of c in 64 bits.  Without a bias c grows with the logit, and
// logits compare exactly.  With one, c is computed in fp32 with an error of at
// most `tol` / 2 (below); only where two neighbours in the order of the picks (or
// the last group taken and the first one left) are nearer than that, and are not
// the same logit and bias, the token is chosen again with the experts in question
// in fp64.  With 256 sigmoid scores and a random bias that is one token in a few
// hundred; fp64 for all of them would cost 2 M x 60 instructions of a pipe of two
// lanes an SM.
//
// Bound by instruction issue: T=8192 E=256 reads 8.4 MB (1.2 us at HBM rate), a
// pick is about 50 instructions of a warp.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_experts.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowwise.cuh"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kInf = INFINITY;

struct RouterParams {
  const void* logits;
  const float* bias;
  int32_t* idx;
  float* w;
  const int32_t* idx_in;  // backward
  const float* dw;
  void* d_logits;
  int T, E, k;
  int groups, topk_groups, group_top, per_group;  // experts per group
  int sigmoid, renormalize;
  int wide;  // rows can be read and written in whole vectors
  float scale;
  long ld;
};

// Unsigned keys in the order of the values: 0 none, 1 NaN, then -inf .. +inf
// (-0 as +0).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return v != v ? 1u : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return key <= 1u ? NAN : __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.));
  return v != v ? 1ull : (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double value_of(uint64_t key) {
  return key <= 1ull ? static_cast<double>(NAN)
                     : __longlong_as_double(static_cast<long long>(
                           (key >> 63) ? key ^ 0x8000000000000000ull : ~key));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32));
  const uint32_t lo =
      __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ float warp_fmax(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
template <int kN>
__device__ __forceinline__ float tree_sum(const float (&v)[kN]) {
  float t[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) t[i] = v[i];
#pragma unroll
  for (int o = 1; o < kN; o *= 2) {
#pragma unroll
    for (int i = 0; i < kN; i += 2 * o) t[i] += t[i + o];
  }
  return t[0];
}

// A lane's N consecutive values of a row from `e0` on; `fill` past E.
template <typename T, int kN>
__device__ __forceinline__ void load_row(const T* row, int e0, int E, bool wide, float fill,
                                         float (&v)[kN]) {
  constexpr int kPer = 16 / sizeof(T);
  if (kN >= kPer && wide) {  // E is a multiple of N: a lane is whole or past the end
#pragma unroll
    for (int i = 0; i < kN; i += kPer) {
      uint4 q = make_uint4(0, 0, 0, 0);
      const bool in = e0 < E;
      if (in) q = __ldg(reinterpret_cast<const uint4*>(row + e0 + i));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < kPer && i + j < kN; ++j) {
        const float x = sizeof(T) == 4 ? __uint_as_float(w[j & 3])
                                       : ((j & 1) ? bf16_hi(w[(j >> 1) & 3]) : bf16_lo(w[(j >> 1) & 3]));
        v[i + j] = in ? x : fill;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = e0 + i < E ? to_float(row[e0 + i]) : fill;
  }
}

template <typename T, int kN>
__device__ __forceinline__ void store_row(T* row, int e0, int E, bool wide, const float (&v)[kN]) {
  constexpr int kPer = 16 / sizeof(T);
  if (kN >= kPer && wide) {
    if (e0 >= E) return;
#pragma unroll
    for (int i = 0; i < kN; i += kPer) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = sizeof(T) == 4 ? __float_as_uint(v[(i + j) % kN])
                              : pack_bf16(v[(i + 2 * j) % kN], v[(i + 2 * j + 1) % kN]);
      *reinterpret_cast<uint4*>(row + e0 + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (e0 + i < E) from_float(row[e0 + i], v[i]);
  }
}

// (below -20 exp(l), where 1 + exp(l) is 1 and exp(-l) may not be a number)
__device__ __forceinline__ float sigmoid_f32(float l) {
  const bool low = l < -20.f;
  const float e = expf(low ? l : -l);
  return low ? e : 1.f / (1.f + e);
}

// The k picks of a warp, highest key first.  `left` is the lane's highest key;
// lane j keeps pick j (key 0 and id -1 where nothing is left).  One pick more is
// made for the runner-up, whose key lane k keeps where k < 32.
template <int kN, typename Key>
__device__ __forceinline__ void pick(Key (&key)[kN], int k, int lane, int& id, Key& own) {
  Key left = key[0];
#pragma unroll
  for (int i = 1; i < kN; ++i) left = left > key[i] ? left : key[i];
  id = -1;
  own = 0;
  for (int j = 0; j <= k && j < 32; ++j) {
    const Key best = warp_max(left);
    if (best == 0) break;
    const int from = __ffs(__ballot_sync(kAll, left == best)) - 1;
    int at = 0;
    if (lane == from) {
#pragma unroll
      for (int i = kN - 1; i >= 0; --i)
        if (key[i] == best) at = i;
      left = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        if (i == at) key[i] = 0;
        left = left > key[i] ? left : key[i];
      }
    }
    at = __shfl_sync(kAll, at, from);
    if (lane == j) {
      id = from * kN + at;
      own = best;
    }
  }
}

template <int kN, typename Key>
__device__ __forceinline__ void top2(const Key (&key)[kN], uint32_t in, Key& a, Key& b) {
  a = b = 0;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const Key v = (in >> i & 1u) ? key[i] : 0;
    b = v > a ? a : v > b ? v : b;
    a = v > a ? v : a;
  }
}
template <typename Key>
__device__ __forceinline__ void merge2(Key& a, Key& b, int o) {
  const Key x = __shfl_xor_sync(kAll, a, o), y = __shfl_xor_sync(kAll, b, o);
  const Key low = a > x ? x : a;
  a = a > x ? a : x;
  b = b > y ? b : y;
  b = b > low ? b : low;
}

// The two highest keys of group g in lane g (0 in the other lanes and where a
// group has none).
template <int kN, typename Key>
__device__ __forceinline__ void group_top2(const RouterParams& p, const Key (&key)[kN], int lane,
                                           Key& a, Key& b) {
  const int lanes = p.per_group / kN;
  if (lanes * kN == p.per_group && (lanes & (lanes - 1)) == 0) {
    // a group is `lanes` whole lanes: all groups at once
    Key x, y;
    top2(key, kAll, x, y);
    for (int o = 1; o < lanes; o *= 2) merge2(x, y, o);
    const int from = min(31, lane * lanes);
    a = __shfl_sync(kAll, x, from);
    b = __shfl_sync(kAll, y, from);
    if (lane >= p.groups) a = b = 0;
    return;
  }
  a = b = 0;
  for (int g = 0; g < p.groups; ++g) {
    uint32_t in = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = lane * kN + i - g * p.per_group;
      if (e >= 0 && e < p.per_group) in |= 1u << i;
    }
    Key x, y;
    top2(key, in, x, y);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) merge2(x, y, o);
    if (lane == g) a = x, b = y;
  }
}

// Which groups stay, as a mask, from lane g's key of group g; `margin` out: the
// lowest key taken and the highest one left (0: none).
template <typename Key>
__device__ __forceinline__ uint32_t take_groups(const RouterParams& p, Key score, int lane,
                                                Key& last, Key& first) {
  int before = 0;  // groups that come before this lane's
  for (int g = 0; g < p.groups; ++g) {
    const Key o = __shfl_sync(kAll, score, g);
    before += o > score || (o == score && g < lane) ? 1 : 0;
  }
  const bool real = lane < p.groups, taken = real && before < p.topk_groups;
  first = warp_max(real && !taken ? score : static_cast<Key>(0));
  last = ~warp_max(taken ? static_cast<Key>(~score) : static_cast<Key>(0));
  return __ballot_sync(kAll, taken);
}

// Bit i: expert e0 + i is in one of the groups of the mask.
template <int kN>
__device__ __forceinline__ uint32_t in_groups(const RouterParams& p, uint32_t groups, int e0) {
  uint32_t in = 0;
  int g = e0 / p.per_group, r = e0 - g * p.per_group;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    if (g < 32 && (groups >> g & 1u)) in |= 1u << i;
    if (++r == p.per_group) r = 0, ++g;
  }
  return in;
}

// The score of a group from its two highest keys, as a key: a group of one is
// its own sum, a group of none is 0.
template <typename Key>
__device__ __forceinline__ Key group_key(const RouterParams& p, Key a, Key b) {
  if (a == 0) return 0;
  if (p.group_top == 1 || b == 0) return a;
  return key_of(value_of(a) + value_of(b));
}

// The row's softmax in fp64: its maximum and 1 / its sum are the token's.
struct Score64 {
  double max, inv;
  int sigmoid;
  __device__ __forceinline__ double at(float l) const {
    return sigmoid ? 1. / (1. + exp(-static_cast<double>(l)))
                   : exp(static_cast<double>(l) - max) * inv;
  }
};

// The choice again, in fp64 for the experts that can be in question: those
// within tol of the group_top-th of their group, then those of the groups taken
// within tol of the k-th.
template <int kN>
__device__ __noinline__ void choose_64(const RouterParams& p, const float (&l)[kN],
                                       const uint32_t (&key)[kN], float tol, float row_max,
                                       int lane, int& id) {
  const int e0 = lane * kN;
  Score64 s{static_cast<double>(row_max), 0., p.sigmoid};
  if (!p.sigmoid) {
    double sum = 0.;
#pragma unroll 1
    for (int i = 0; i < kN; ++i)
      if (l[i] != -kInf) sum += exp(static_cast<double>(l[i]) - s.max);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    s.inv = 1. / sum;
  }
  uint64_t fine[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) fine[i] = 0;
  uint32_t done = 0;
  auto evaluate = [&](uint32_t want) {  // bit i: expert e0 + i
    want &= ~done;
    done |= want;
#pragma unroll 1
    for (int i = 0; i < kN; ++i) {
      if (want >> i & 1u) {
        const double c = s.at(l[i]) + (p.bias ? static_cast<double>(__ldg(p.bias + e0 + i)) : 0.);
        fine[i] = key_of(c);
      }
    }
  };
  // NaN keys (1) are known as they are
#pragma unroll
  for (int i = 0; i < kN; ++i)
    if (key[i] == 1u) fine[i] = 1, done |= 1u << i;
  uint32_t in = kAll;
  if (p.topk_groups < p.groups) {
    uint32_t a, b;
    group_top2(p, key, lane, a, b);
    const uint32_t edge = p.group_top == 2 && b != 0 ? b : a;
    const float low = edge > 1u ? value_of(edge) : -kInf;
    uint32_t want = 0;
#pragma unroll 1
    for (int g = 0; g < p.groups; ++g) {
      const float from = __shfl_sync(kAll, low, g);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int e = e0 + i - g * p.per_group;
        if (e >= 0 && e < p.per_group && key[i] > 1u &&
            !(value_of(key[i]) < from - (tol + fabsf(from) * 0x1p-21f)))
          want |= 1u << i;
      }
    }
    evaluate(want);
    uint64_t x, y, last, first;
    group_top2(p, fine, lane, x, y);
    const uint32_t groups = take_groups(p, group_key(p, x, y), lane, last, first);
    in = in_groups<kN>(p, groups, e0);
  }
  uint32_t rest[kN], own;
#pragma unroll
  for (int i = 0; i < kN; ++i)
    rest[i] = !(in >> i & 1u) ? 0u : p.bias || key[i] <= 1u ? key[i] : key_of(l[i]);
  if (!p.bias) {  // only the groups were in question
    pick(rest, p.k, lane, id, own);
    return;
  }
  pick(rest, p.k - 1, lane, id, own);  // (its last pick is the k-th)
  const uint32_t kth = __shfl_sync(kAll, own, p.k - 1);
  const float from = kth > 1u ? value_of(kth) : -kInf;
  const float edge = from - (tol + fabsf(from) * 0x1p-21f);
  uint32_t want = 0;
#pragma unroll
  for (int i = 0; i < kN; ++i)
    if ((in >> i & 1u) && key[i] > 1u && !(value_of(key[i]) < edge)) want |= 1u << i;
  evaluate(want);
#pragma unroll
  for (int i = 0; i < kN; ++i)
    if (!(in >> i & 1u)) fine[i] = 0;
  uint64_t none;
  pick(fine, p.k, lane, id, none);
}

template <typename T, int kN>
__global__ void __launch_bounds__(256) router_forward_kernel(const RouterParams p) {
  pdl_enter();
  const int lane = threadIdx.x & 31, e0 = lane * kN;
  const long t = static_cast<long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.T) return;  // whole warps leave together
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  float l[kN];
  load_row<T, kN>(row, e0, p.E, p.wide, -kInf, l);
  const bool by_score = p.bias != nullptr;  // else by the logits themselves
  const bool groups = p.topk_groups < p.groups;

  // the row's maximum and sum; `broken`: its softmax is NaN
  float m = l[0], inv = 1.f, unit = 1.f;
  bool broken = false;
  if (!p.sigmoid) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kN; ++i) m = fmaxf(m, l[i]), nan |= l[i] != l[i];
    m = warp_fmax(m);
    broken = __any_sync(kAll, nan) || m == kInf;
    if (by_score || groups || !p.renormalize) {
      float ex[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) ex[i] = l[i] == -kInf ? 0.f : expf(l[i] - m);
      inv = 1.f / warp_add(tree_sum(ex));
      unit = inv;
    }
  }
  auto score = [&](float x) { return p.sigmoid ? sigmoid_f32(x) : expf(x - m) * inv; };

  // What fp32 leaves of c: a score is off by 2 units of exp, 1 of the division
  // and of 1 + exp (sigmoid), or by the exponent's rounding (|l - m| 2^-24, of
  // a score that falls faster than that) and the sum's (10 of its tree), each of
  // 2^-24 of at most the largest score: 4 and 16 of them; the sum with the bias
  // adds 2^-24 of itself, counted where it is compared.
  const float tol = (p.sigmoid ? 0x1p-20f : 0x1p-18f) * unit;
  uint32_t key[kN];
  if (by_score) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float b = e0 + i < p.E ? __ldg(p.bias + e0 + i) : 0.f;
      key[i] = l[i] == -kInf ? 0u : broken ? 1u : key_of(score(l[i]) + b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) key[i] = l[i] == -kInf ? 0u : broken ? 1u : key_of(l[i]);
  }

  auto near = [&](uint32_t hi, uint32_t lo) {
    const float x = value_of(hi), y = value_of(lo);
    return lo > 1u && !(x - y > tol + (fabsf(x) + fabsf(y)) * 0x1p-22f);
  };
  bool redo = false;
  uint32_t work[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) work[i] = key[i];
  if (groups) {
    uint32_t a, b, last, first;
    group_top2(p, key, lane, a, b);
    // keys are logits without a bias: their sums are the scores'
    const bool sums = p.group_top == 2;
    if (!by_score && sums) {
      if (a > 1u) a = key_of(score(value_of(a)));
      if (b > 1u) b = key_of(score(value_of(b)));
    }
    const uint32_t mask = take_groups(p, group_key(p, a, b), lane, last, first);
    // (a group's sum has twice a score's error)
    if (by_score || sums)
      redo = first > 1u && !(value_of(last) - value_of(first) >
                             2.f * tol + (fabsf(value_of(last)) + fabsf(value_of(first))) * 0x1p-21f);
    const uint32_t in = in_groups<kN>(p, mask, e0);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (!(in >> i & 1u)) work[i] = 0;
  }
  int id;
  uint32_t own;
  pick(work, p.k, lane, id, own);
  if (by_score) {
    // lane j against pick j + 1 (k of 32 has no lane for the runner-up: always
    // looked at again)
    const uint32_t next = __shfl_down_sync(kAll, own, 1);
    const int next_id = __shfl_down_sync(kAll, id, 1);
    bool close = lane < p.k && lane < 31 && near(own, next);
    if (close)  // the same logit and bias are the same score, and in order
      close = !(to_float(row[id]) == to_float(row[next_id]) &&
                __ldg(p.bias + id) == __ldg(p.bias + next_id));
    redo |= __any_sync(kAll, close) || p.k == 32;
  }
  if (redo && !broken) {
    // (copies: what a call takes by reference does not stay in registers)
    float l2[kN];
    uint32_t key2[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      l2[i] = l[i];
      key2[i] = by_score || key[i] <= 1u ? key[i] : key_of(score(l[i]));
    }
    choose_64<kN>(p, l2, key2, tol, m, lane, id);
  }
  if (lane >= p.k) id = -1;

  // weights, lane j's of slot j
  const bool have = id >= 0;
  const float x = have ? to_float(row[id]) : -kInf;
  float w;
  if (!p.renormalize) {
    w = have ? score(x) : 0.f;
  } else {
    const float top = warp_fmax(x);
    float u;
    // relative to the largest, so that small sigmoids do not vanish (below -20
    // 1 + exp(l) is 1)
    if (p.sigmoid && top > -20.f) u = sigmoid_f32(x);
    else u = x == top ? 1.f : expf(x - top);
    if (!have) u = 0.f;
    if (have && x != x) u = x;
    w = u / warp_add(u);
    if (!have) w = 0.f;
  }
  if (broken && have) w = NAN;
  if (lane < p.k) {
    p.idx[t * p.k + lane] = id;
    p.w[t * p.k + lane] = have ? p.scale * w : 0.f;
  }
}

// dl from dw, with g_j = scale dw_j, q the renormalised weights:
//   sigmoid, plain         dl_j = g_j s_j (1 - s_j)
//   sigmoid, renormalised  dl_j = q_j (1 - s_j) (g_j - sum_i g_i q_i)
//   softmax, plain         dl_e = s_e ([e = j] g_j - sum_i g_i s_i)
//   softmax, renormalised  dl_j = q_j (g_j - sum_i g_i q_i)
template <typename T, int kN>
__global__ void __launch_bounds__(256) router_backward_kernel(const RouterParams p) {
  pdl_enter();
  const int lane = threadIdx.x & 31, e0 = lane * kN;
  const long t = static_cast<long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  const int id = lane < p.k ? __ldg(p.idx_in + t * p.k + lane) : -1;
  const float x = id >= 0 && id < p.E ? to_float(row[id]) : -kInf;
  const bool have = x != -kInf;
  const float g = have ? p.scale * __ldg(p.dw + t * p.k + lane) : 0.f;
  float out[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) out[i] = 0.f;
  float mine;  // of slot `lane`
  if (!p.sigmoid && !p.renormalize) {
    float l[kN], ex[kN];
    load_row<T, kN>(row, e0, p.E, p.wide, -kInf, l);
    float m = l[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) m = fmaxf(m, l[i]);
    m = warp_fmax(m);
    // (an expert out of the choice has the score 0, in a row of such ones too)
#pragma unroll
    for (int i = 0; i < kN; ++i) ex[i] = l[i] == -kInf ? 0.f : expf(l[i] - m);
    const float sum = warp_add(tree_sum(ex));
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    mine = have ? g * (expf(x - m) * inv) : 0.f;
    const float dot = warp_add(mine);
#pragma unroll
    for (int i = 0; i < kN; ++i) out[i] = l[i] == -kInf ? 0.f : -(ex[i] * inv) * dot;
  } else {
    const float s = p.sigmoid ? sigmoid_f32(x) : 0.f;
    const float rest = p.sigmoid ? 1.f / (1.f + expf(x)) : 1.f;  // 1 - s
    if (p.renormalize) {
      const float top = warp_fmax(x);
      float u = p.sigmoid && top > -20.f ? s : x == top ? 1.f : expf(x - top);
      if (!have) u = 0.f;
      if (have && x != x) u = x;
      const float total = warp_add(u), q = have ? u / total : 0.f;
      const float dot = warp_add(g * q);
      mine = q * rest * (g - dot);
    } else {
      mine = g * s * rest;
    }
    if (!have) mine = 0.f;
  }
  for (int j = 0; j < p.k; ++j) {
    const int at = __shfl_sync(kAll, have ? id : -1, j) - e0;
    const float v = __shfl_sync(kAll, mine, j);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (at == i) out[i] += v;
  }
  store_row<T, kN>(static_cast<T*>(p.d_logits) + t * p.ld, e0, p.E, p.wide, out);
}

template <typename T, int kN>
cudaError_t launch(const RouterParams& p, bool backward, cudaStream_t s) {
  // few tokens: a warp to a block, so that they lie on as many SMs as there are
  const int warps = p.T <= 8 * num_sms() ? 1 : 8;
  const dim3 grid(static_cast<unsigned>(ceil_div(p.T, warps))), block(32 * warps);
  return backward ? launch_kernel(router_backward_kernel<T, kN>, grid, block, 0, s, 1, p)
                  : launch_kernel(router_forward_kernel<T, kN>, grid, block, 0, s, 1, p);
}

template <typename T>
cudaError_t launch_width(RouterParams p, bool backward, cudaStream_t s) {
  const int n = p.E <= 32 ? 1 : p.E <= 64 ? 2 : p.E <= 128 ? 4 : p.E <= 256 ? 8 : p.E <= 512 ? 16 : 32;
  const uintptr_t all = reinterpret_cast<uintptr_t>(p.logits) |
                        (backward ? reinterpret_cast<uintptr_t>(p.d_logits) : 0);
  p.wide = p.E % n == 0 && all % 16 == 0 && (p.ld * static_cast<long>(sizeof(T))) % 16 == 0;
  return n == 1    ? launch<T, 1>(p, backward, s)
         : n == 2  ? launch<T, 2>(p, backward, s)
         : n == 4  ? launch<T, 4>(p, backward, s)
         : n == 8  ? launch<T, 8>(p, backward, s)
         : n == 16 ? launch<T, 16>(p, backward, s)
                   : launch<T, 32>(p, backward, s);
}

int check_router(const moe_router_problem* p) {
  if (!p || p->T < 0 || p->E < 1 || p->k < 1 || p->k > p->E) return MOE_ERR_INVALID_ARG;
  if (p->logits_dtype != MOE_DTYPE_BF16 && p->logits_dtype != MOE_DTYPE_F32)
    return MOE_ERR_INVALID_ARG;
  if (p->score != MOE_SCORE_SOFTMAX && p->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (p->E > MOE_MAX_EXPERTS || p->k > MOE_MAX_TOPK || p->groups > MOE_MAX_EXPERT_GROUPS)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (p->groups < 1 || p->E % p->groups != 0 || p->topk_groups < 1 || p->topk_groups > p->groups)
    return MOE_ERR_INVALID_ARG;
  const int per = p->E / p->groups;
  if (p->group_top < 1 || p->group_top > 2 || p->group_top > per || p->k > p->topk_groups * per)
    return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale)) return MOE_ERR_INVALID_ARG;
  if (p->ld_logits != 0 && p->ld_logits < p->E) return MOE_ERR_INVALID_ARG;
  if (p->ld_logits > (1LL << 40)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

RouterParams params_of(const moe_router_problem* p) {
  RouterParams r{};
  r.T = p->T;
  r.E = p->E;
  r.k = p->k;
  r.groups = p->groups;
  r.topk_groups = p->topk_groups;
  r.group_top = p->group_top;
  r.per_group = p->E / p->groups;
  r.sigmoid = p->score == MOE_SCORE_SIGMOID;
  r.renormalize = p->renormalize != 0;
  r.scale = p->scale;
  r.ld = p->ld_logits ? p->ld_logits : p->E;
  return r;
}

bool off(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

int run(const moe_router_problem* p, const RouterParams& r, bool backward, cudaStream_t s) {
  const cudaError_t err = p->logits_dtype == MOE_DTYPE_F32 ? launch_width<float>(r, backward, s)
                                                           : launch_width<Bf16>(r, backward, s);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  set_last_launch_count(1);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_router_forward(const moe_router_problem* p, const void* logits,
                                  const float* bias, int32_t* topk_idx, float* topk_w,
                                  void* stream) {
  const int rc = check_router(p);
  if (rc != MOE_OK) return rc;
  set_last_launch_count(0);
  if (p->T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_ERR_INVALID_ARG;
  if (off(logits, p->logits_dtype == MOE_DTYPE_F32 ? 4 : 2) || off(bias, 4) || off(topk_idx, 4) ||
      off(topk_w, 4))
    return MOE_ERR_MISALIGNED;
  RouterParams r = params_of(p);
  r.logits = logits;
  r.bias = bias;
  r.idx = topk_idx;
  r.w = topk_w;
  return run(p, r, false, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_router_backward(const moe_router_problem* p, const void* logits,
                                   const int32_t* topk_idx, const float* d_topk_w, void* d_logits,
                                   void* stream) {
  const int rc = check_router(p);
  if (rc != MOE_OK) return rc;
  set_last_launch_count(0);
  if (p->T == 0) return MOE_OK;
  if (!logits || !topk_idx || !d_topk_w || !d_logits) return MOE_ERR_INVALID_ARG;
  const int size = p->logits_dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (off(logits, size) || off(d_logits, size) || off(topk_idx, 4) || off(d_topk_w, 4))
    return MOE_ERR_MISALIGNED;
  RouterParams r = params_of(p);
  r.logits = logits;
  r.idx_in = topk_idx;
  r.dw = d_topk_w;
  r.d_logits = d_logits;
  return run(p, r, true, static_cast<cudaStream_t>(stream));
}
