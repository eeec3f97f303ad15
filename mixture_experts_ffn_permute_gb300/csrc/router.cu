// Expert router: scores, balance bias, groups, top-k and weights, and its
// backward (moe_router_* of include/moe_experts.h).
//
// One warp per token, the row in registers: lane i holds the experts i N ..
// i N + N - 1 (N the power of two that fits E), so that among equal keys the lowest
// lane, and in it the first, is the lowest id.  A key is the value's bits in an
// order of unsigned integers.  Up to N = 8, and with a bias N = 16, a lane sorts its keys
// once; a pick is then one warp maximum, one ballot and a shift of the winner's list.
//
// The order is that of c in 64 bits.  Without a bias c grows with the logit, and
// logits compare exactly.  With one, c is computed in fp32 with an error of at
// most `tol` / 2 (below); only where two neighbours in the order of the picks (or
// the last group taken and the first one left) are nearer than that, and are not
// the same logit and bias, it is looked at again.  Picks: their scores to 41 bits in
// pairs of fp32, a lane each, put them in order.  Groups: the whole token in such pairs.
// What those do not tell: the token in fp64.  With 256 sigmoid scores and a random bias
// nine tokens of 8192 are looked at.
//
// Bound by latency (half of the issue slots are empty): T=8192 E=256 reads 8.4 MB (1.2 us at
// HBM rate); k = 8 with a bias and 8 groups takes 14.4 to 15 us (a token 8000 cycles, in 1.7 waves; near
// picks 4500 cycles more, near groups 20000, fp64 30000), without a bias and groups 10.0, k = 32
// with a bias 28; T=131072 160 us.  The backward takes 5 us, most of it the call (T=65536 25 us).
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
constexpr int kForwardThreads = 128;  // (256: 0.7 us more at T=8192 E=256, the last blocks' wait)
constexpr float kInf = INFINITY;
constexpr uint32_t kMinusInf = 0x007fffffu;  // its key (below)

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
  int group_lanes;  // lanes per group, where a group is a power of two of whole ones (else 0)
  int sigmoid, renormalize;
  int wide;       // rows can be read and written in whole vectors
  int bias_wide;  // the bias, too
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
__device__ __forceinline__ float warp_fmax(float v) {  // (a NaN counts as nothing)
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
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

// The highest key that is left after picks.
template <bool kSorted, int kN, typename Key>
__device__ __forceinline__ Key highest_left(const Key (&key)[kN]) {
  Key left = key[0];
#pragma unroll
  for (int i = 1; i < (kSorted ? 1 : kN); ++i) left = left > key[i] ? left : key[i];
  return warp_max(left);
}

// The same from lists that every lane has sorted, highest first and the first among
// equal ones.  Packed keys have their places in the lane in their last three or four
// bits (all ones: the first), which do not count; else `at` holds the places, four bits
// each.  Pick `j` alone; false where nothing is left.
template <int kN>
constexpr uint32_t kPlace = kN <= 8 ? 7u : 15u;
template <bool kPacked, int kN>
__device__ __forceinline__ bool pick_one(uint32_t (&key)[kN], uint32_t& at, int j, int lane, int& id,
                                         uint32_t& own) {
  uint32_t best = warp_max(key[0]);
  if (best == 0) return false;
  if (kPacked) best &= ~kPlace<kN>;
  const int from = __ffs(__ballot_sync(kAll, key[0] >= best)) - 1;
  const uint32_t theirs =
      __shfl_sync(kAll, kPacked ? key[0] : at, from) & (kPacked ? kPlace<kN> : 15u);
  const int place = static_cast<int>(kPacked ? kPlace<kN> - theirs : theirs);
  if (lane == from) {
#pragma unroll
    for (int i = 0; i + 1 < kN; ++i) key[i] = key[i + 1];
    key[kN - 1] = 0;
    if (!kPacked) at >>= 4;
  }
  if (lane == j) {
    id = from * kN + place;
    own = best;
  }
  return true;
}
template <bool kPacked, int kN>
__device__ __forceinline__ void pick_sorted(uint32_t (&key)[kN], uint32_t& at, int k, int lane,
                                            int& id, uint32_t& own) {
  id = -1;
  own = 0;
  for (int j = 0; j <= k && j < 32; ++j)
    if (!pick_one<kPacked>(key, at, j, lane, id, own)) break;
}

// Sorts by an odd-even merge network (Batcher): kN = 1, 2, 4, 8 or 16 (packed).
template <int kN, typename Key>
__device__ __forceinline__ void sort_network(Key (&v)[kN]) {
  if constexpr (kN > 1) {
#pragma unroll
    for (int p = 1; p < kN; p *= 2) {
#pragma unroll
      for (int q = p; q > 0; q /= 2) {
#pragma unroll
        for (int j = q % p; j + q < kN; j += 2 * q) {
#pragma unroll
          for (int i = 0; i < q; ++i) {
            const int a = i + j, b = i + j + q;
            if (b < kN && a / (2 * p) == b / (2 * p)) {
              const Key x = v[a], y = v[b];
              v[a] = x > y ? x : y;
              v[b] = x > y ? y : x;
            }
          }
        }
      }
    }
  }
}

// Packed: two instructions an exchange, where 64 bits take six.  (Below kPlace + 1 is
// none, then a NaN, from kPackedInf -inf.)
constexpr uint32_t kPackedInf = 0x00800000u;
template <bool kPacked, int kN>
__device__ __forceinline__ uint32_t sort_lane(uint32_t (&key)[kN]) {
  constexpr uint32_t kOnes = kPlace<kN>;
  uint32_t at = 0;
  if constexpr (kPacked) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      key[i] = key[i] == 0 ? 0u
                           : (max(key[i], key[i] == kMinusInf ? kPackedInf : kOnes + 1) & ~kOnes) | (kOnes - i);
    sort_network(key);
  } else {
    uint64_t v[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = static_cast<uint64_t>(key[i]) << 32 | (kN - 1 - i);
    sort_network(v);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      key[i] = static_cast<uint32_t>(v[i] >> 32);
      at |= (kN - 1 - static_cast<uint32_t>(v[i])) << (4 * i);
    }
  }
  return at;
}
// The key without its place: the value is at most kPlace steps above the key's.
template <int kN>
__device__ __forceinline__ uint32_t unpacked(uint32_t key) {
  constexpr uint32_t kOnes = kPlace<kN>;
  return key <= kOnes ? 0u : key <= 2 * kOnes + 1 ? 1u : key <= kPackedInf + kOnes ? kMinusInf : key & ~kOnes;
}
// The key of a logit in bf16, whose lower half is all zeros (positive) or ones.
__device__ __forceinline__ uint32_t whole_bf16(uint32_t key) {
  return key <= 1u ? key : (key >> 31) ? key & ~0xffffu : key | 0xffffu;
}
template <int kN>
__device__ __forceinline__ uint32_t place_of(bool packed, uint32_t key, uint32_t at, int j) {
  return packed ? kPlace<kN> - (key & kPlace<kN>) : at >> (4 * j) & 15u;
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
                                           bool sorted, Key& a, Key& b) {
  const int lanes = p.group_lanes;
  if (lanes) {  // a group is whole lanes: all groups at once
    Key x, y;
    if (sorted) {
      x = key[0];
      y = kN > 1 ? key[kN > 1 ? 1 : 0] : 0;
    } else {
      top2(key, kAll, x, y);
    }
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

// Which groups stay, as a mask, from lane g's key of group g (0 in the other lanes).
template <typename Key>
__device__ __forceinline__ uint32_t take_groups(const RouterParams& p, Key score, int lane) {
  int before = 0;  // groups that come before this lane's
#pragma unroll 1
  for (int g0 = 0; g0 < p.groups; g0 += 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // (lanes past the groups have 0 and come after)
      const Key o = __shfl_sync(kAll, score, (g0 + i) & 31);
      before += o >= score + (g0 + i < lane ? 0 : 1) ? 1 : 0;
    }
  }
  return __ballot_sync(kAll, lane < p.groups && before < p.topk_groups);
}

// Bit i: expert e0 + i is in one of the groups of the mask.
template <int kN>
__device__ __forceinline__ uint32_t in_groups(const RouterParams& p, uint32_t groups, int e0) {
  if (p.group_lanes) {
    const int g = (e0 / kN) / p.group_lanes;
    return g < p.groups && (groups >> g & 1u) ? kAll : 0u;
  }
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

// Two fp32 values whose sum is the number (Dekker, Knuth): 44 bits and more.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two fast_two_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  const float p = __fmul_rn(a.hi, b.hi);
  const float e = __fmaf_rn(a.hi, b.hi, -p);
  return fast_two_sum(p, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, e)));
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  return fast_two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}

// exp(x) for -80 <= x <= 0 (below: that of -80, 2^-115) to about 2^-43 of it: x = n ln 2
// + r by three parts of ln 2, the first of 16 bits, the Taylor series to r^13, its
// terms from r^7 on in fp32 (below 2^-22 of the sum).
__device__ __forceinline__ Two exp_two(Two x) {
  if (x.hi < -80.f) x = {-80.f, 0.f};
  const float n = rintf(x.hi * 1.4426950408889634f);
  Two r = two_sum(x.hi, -n * 0.693145751953125f);
  const float p2 = __fmul_rn(n, 1.428606765330187e-06f);
  r = add(r, {-p2, x.lo - __fmaf_rn(n, 1.428606765330187e-06f, -p2) - n * 5.497923148104107e-14f});
  float t = 0x1.612462p-33f;
  t = fmaf(t, r.hi, 0x1.1eed8ep-29f);
  t = fmaf(t, r.hi, 0x1.ae6456p-26f);
  t = fmaf(t, r.hi, 0x1.27e4fcp-22f);
  t = fmaf(t, r.hi, 0x1.71de3ap-19f);
  t = fmaf(t, r.hi, 0x1.a01a02p-16f);
  t = fmaf(t, r.hi, 0x1.a01a02p-13f);
  Two e = add({0x1.6c16c2p-10f, -0x1.27d27ep-35f}, mul(r, {t, 0.f}));
  e = add({0x1.111112p-7f, -0x1.dddddep-32f}, mul(r, e));
  e = add({0x1.555556p-5f, -0x1.555556p-30f}, mul(r, e));
  e = add({0x1.555556p-3f, -0x1.555556p-28f}, mul(r, e));
  e = add({0.5f, 0.f}, mul(r, e));
  e = add({1.f, 0.f}, mul(r, e));
  e = add({1.f, 0.f}, mul(r, e));
  const float scale = __int_as_float((static_cast<int>(n) + 127) << 23);  // n >= -116
  return {e.hi * scale, e.lo * scale};
}
__device__ __forceinline__ Two inverse(Two d) {
  const float y = __frcp_rn(d.hi);
  return fast_two_sum(y, y * __fmaf_rn(-y, d.lo, __fmaf_rn(-y, d.hi, 1.f)));
}

// The same logit and bias: the same score, whatever its rounding.
template <typename T>
__device__ __forceinline__ bool same_expert(const RouterParams& p, const T* row, int a, int b) {
  return to_float(row[a]) == to_float(row[b]) && __ldg(p.bias + a) == __ldg(p.bias + b);
}

// The first n picks, lane j's in lane j, in the order of their scores' 41 bits: all
// of them are there that can be among the first n - 1.  False where they do not tell
// two apart that are not the same logit and bias.
template <typename T>
__device__ __noinline__ bool order_picks(const RouterParams& p, const T* row, float m, int n, int lane,
                                         int& id) {
  const bool mine = lane < n && id >= 0;
  const float l = mine ? to_float(row[id]) : 0.f, b = mine ? __ldg(p.bias + id) : 0.f;
  Two c;
  if (p.sigmoid) {
    const Two e = exp_two({-fabsf(l), 0.f});
    c = inverse(add({1.f, 0.f}, e));
    if (l < 0.f) c = mul(e, c);
  } else {
    Two sum{0.f, 0.f};
#pragma unroll 1
    for (int i = lane; i < p.E; i += 32) {
      const float x = to_float(row[i]);
      if (x != -kInf) sum = add(sum, exp_two(two_sum(x, -m)));
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1)
      sum = add(sum, {__shfl_xor_sync(kAll, sum.hi, o), __shfl_xor_sync(kAll, sum.lo, o)});
    c = mul(exp_two(two_sum(l, -m)), inverse(sum));
  }
  c = add(c, {b, 0.f});
  const float eps = 0x1p-40f * (1.f + fabsf(b));  // (twice the error of two)
  int rank = 0;
  bool unsure = false;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const float hi = __shfl_sync(kAll, c.hi, j), lo = __shfl_sync(kAll, c.lo, j);
    const float lj = __shfl_sync(kAll, l, j), bj = __shfl_sync(kAll, b, j);
    const int ij = __shfl_sync(kAll, id, j);
    const float d = (hi - c.hi) + (lo - c.lo);
    const bool same = lj == l && bj == b;
    if (ij >= 0 && j != lane) {
      rank += same ? (ij < id ? 1 : 0) : (d > 0.f ? 1 : 0);
      unsure |= mine && !same && !(fabsf(d) > eps);
    }
  }
  // lane `rank` takes this lane's id
  int at = -1;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const int rj = __shfl_sync(kAll, mine ? rank : -1, j), ij = __shfl_sync(kAll, id, j);
    if (rj == lane) at = ij;
  }
  id = at;
  return !__any_sync(kAll, unsure);
}

// Numbers of two parts as keys: hi is their sum rounded, so that hi and then lo give
// their order.
__device__ __forceinline__ uint64_t key_of(Two v) {
  return static_cast<uint64_t>(key_of(v.hi)) << 32 | key_of(v.lo);
}
__device__ __forceinline__ Two two_of(uint64_t key) {
  return {value_of(static_cast<uint32_t>(key >> 32)), value_of(static_cast<uint32_t>(key))};
}
__device__ __forceinline__ float minus(uint64_t x, uint64_t y) {
  const Two a = two_of(x), b = two_of(y);
  return (a.hi - b.hi) + (a.lo - b.lo);
}

// The whole choice again in pairs of fp32; false where they do not tell two groups, or
// two picks that are not the same logit and bias, apart.
template <typename T, int kN>
__device__ __noinline__ bool choose_two(const RouterParams& p, const T* row, float m, int lane, int& id) {
  const int e0 = lane * kN;
  Two inv{1.f, 0.f};
  if (!p.sigmoid) {
    Two sum{0.f, 0.f};
#pragma unroll 1
    for (int i = lane; i < p.E; i += 32) {
      const float x = to_float(row[i]);
      if (x != -kInf) sum = add(sum, exp_two(two_sum(x, -m)));
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1)
      sum = add(sum, {__shfl_xor_sync(kAll, sum.hi, o), __shfl_xor_sync(kAll, sum.lo, o)});
    inv = inverse(sum);
  }
  uint64_t each[kN], key[kN];
#pragma unroll(kN < 2 ? 1 : 2)
  for (int i = 0; i < kN; ++i) {
    const float x = e0 + i < p.E ? to_float(row[e0 + i]) : -kInf;
    const float b = p.bias && e0 + i < p.E ? __ldg(p.bias + e0 + i) : 0.f;
    const Two e = exp_two(p.sigmoid ? Two{-fabsf(x), 0.f} : two_sum(x, -m));
    Two c = mul(p.sigmoid && x >= 0.f ? Two{1.f, 0.f} : e,
                p.sigmoid ? inverse(add({1.f, 0.f}, e)) : inv);
    c = add(c, {b, 0.f});
    each[i] = x == -kInf ? 0 : key_of(c);
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) key[i] = each[i];
  bool finite = true;
#pragma unroll
  for (int i = 0; i < kN; ++i) finite &= key[i] == 0 || fabsf(two_of(key[i]).hi) < kInf;
  if (!__all_sync(kAll, finite)) return false;
  uint32_t in = kAll;
  if (p.topk_groups < p.groups) {
    uint64_t x, y;
    group_top2(p, key, lane, false, x, y);
    float size = x != 0 ? fabsf(two_of(x).hi) : 0.f;
    if (p.group_top == 2 && y != 0) {
      size += fabsf(two_of(y).hi);
      x = key_of(add(two_of(x), two_of(y)));
    }
    const uint32_t mask = take_groups(p, x, lane);
    const bool taken = mask >> lane & 1u;
    const uint64_t first = warp_max(taken ? uint64_t{0} : x);
    const uint64_t last = ~warp_max(taken ? ~x : uint64_t{0});
    size = warp_fmax(size);
    if (first != 0 && !(minus(last, first) > 0x1p-39f * (1.f + size))) return false;
    in = in_groups<kN>(p, mask, e0);
  }
  if (p.bias) {
    uint64_t own;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (!(in >> i & 1u)) key[i] = 0;
    pick(key, p.k, lane, id, own);
    uint64_t next = __shfl_down_sync(kAll, own, 1);
    const int next_id = __shfl_down_sync(kAll, id, 1);
    const uint64_t left = highest_left<false>(key);
    if (lane == 31) next = left;  // (the last of 32 picks)
    bool close = false;
    if (lane < p.k && next != 0) {
      const float eps = 0x1p-40f * (1.f + fabsf(__ldg(p.bias + id)));
      close = !(minus(own, next) > eps);
      // the same score, and in order; but behind a runner-up that is the last pick's like
      // there may be a near one that is not
      if (close && lane < 31 && same_expert(p, row, id, next_id))
        close = lane == p.k - 1 && left != 0 && !(minus(own, left) > eps);
    }
    return !__any_sync(kAll, close);
  }
  uint32_t logit[kN], own;
#pragma unroll
  for (int i = 0; i < kN; ++i)
    logit[i] = (in >> i & 1u) && e0 + i < p.E && to_float(row[e0 + i]) != -kInf
                   ? key_of(to_float(row[e0 + i])) : 0u;
  pick(logit, p.k - 1, lane, id, own);
  return true;
}

// exp(x) for x <= 0 in fp64, to about 2^-51 of it: x = n ln 2 + r, the Taylor series
// of exp(r) to r^13 (|r| < 0.35: the next term is below 2^-57), the exponent by its bits.
__device__ __forceinline__ double exp64(double x) {
  if (!(x > -700.)) return x != x ? x : 0.;
  const float n = rintf(static_cast<float>(x) * 1.4426950408889634f);
  double r = fma(static_cast<double>(n), -0.69314718055994530942, x);
  r = fma(static_cast<double>(n), -2.3190468138462996e-17, r);  // ln 2 beyond its 53 bits
  double y = 1. / 6227020800.;
  y = fma(y, r, 1. / 479001600.);
  y = fma(y, r, 1. / 39916800.);
  y = fma(y, r, 1. / 3628800.);
  y = fma(y, r, 1. / 362880.);
  y = fma(y, r, 1. / 40320.);
  y = fma(y, r, 1. / 5040.);
  y = fma(y, r, 1. / 720.);
  y = fma(y, r, 1. / 120.);
  y = fma(y, r, 1. / 24.);
  y = fma(y, r, 1. / 6.);
  y = fma(y, r, 0.5);
  y = fma(y, r, 1.);
  y = fma(y, r, 1.);
  return __longlong_as_double(__double_as_longlong(y) + static_cast<long long>(n) * (1LL << 52));
}

// The choice again, in fp64.  Without a bias only the groups were in question, and
// the experts go by their logits.
template <int kN>
__device__ __noinline__ void choose_64(const RouterParams& p, const float (&l)[kN], float row_max,
                                       int lane, int& id) {
  const int e0 = lane * kN;
  uint64_t key[kN];
  double c[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const double x = l[i];
    if (p.sigmoid) {
      const double e = exp64(-fabs(x));
      c[i] = (x < 0. ? e : 1.) / (1. + e);
    } else {
      c[i] = l[i] == -kInf ? 0. : exp64(x - row_max);
    }
  }
  if (!p.sigmoid) {
    double sum = 0.;
#pragma unroll
    for (int i = 0; i < kN; ++i) sum += c[i];
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    const double inv = 1. / sum;
#pragma unroll
    for (int i = 0; i < kN; ++i) c[i] *= inv;
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    if (p.bias && e0 + i < p.E) c[i] += __ldg(p.bias + e0 + i);
    key[i] = l[i] == -kInf ? 0 : key_of(c[i]);
  }
  uint32_t in = kAll;
  if (p.topk_groups < p.groups) {
    uint64_t x, y;
    group_top2(p, key, lane, false, x, y);
    in = in_groups<kN>(p, take_groups(p, group_key(p, x, y), lane), e0);
  }
  if (p.bias) {
    uint64_t own;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (!(in >> i & 1u)) key[i] = 0;
    pick(key, p.k - 1, lane, id, own);
  } else {
    uint32_t logit[kN], own;
#pragma unroll
    for (int i = 0; i < kN; ++i) logit[i] = (in >> i & 1u) && l[i] != -kInf ? key_of(l[i]) : 0u;
    pick(logit, p.k - 1, lane, id, own);
  }
}

// kSort: sorted lists (of 16: with a bias, and groups of whole lanes or none).
template <typename T, int kN, bool kSort>
__global__ void __launch_bounds__(kForwardThreads) router_forward_kernel(const RouterParams p) {
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
  // for the order alone: the fast exponential and quotient
  auto rough = [&](float x) {
    return p.sigmoid ? __fdividef(1.f, 1.f + __expf(-x)) : __expf(x - m) * inv;
  };

  // By how much fp32 may be wrong about the difference of two c, in units of 2^-24 of the
  // largest score.  Sigmoid: the exponential's 2 + 1.2 |l| steps count s (1 - s) times,
  // a unit at most; 1 + exp one, the quotient's 2: below 4 each.  Softmax: the
  // exponent's |l - m| and the fast exponential's 2 + 1.2 |l - m| of a score that
  // falls faster than that, 3; the sum's 10 of its tree and 2 of its terms, the
  // quotient's and the product's: below 24.
  // The sum with the bias adds 2^-24 of itself, counted where it is compared.
  const float tol = (p.sigmoid ? 0x1p-21f : 0x1p-18f) * unit;
  uint32_t key[kN];
  if (by_score) {
    float b[kN];
    load_row<float, kN>(p.bias, e0, p.E, p.bias_wide, 0.f, b);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      key[i] = l[i] == -kInf ? 0u : broken ? 1u : key_of(rough(l[i]) + b[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) key[i] = l[i] == -kInf ? 0u : broken ? 1u : key_of(l[i]);
  }
  // Keys are packed where their last bits do not matter: scores are looked at again where
  // they are near, logits in bf16 have none.
  const bool packed = kSort && (kN > 8 || sizeof(T) == 2 || by_score);
  uint32_t at = 0;
  if constexpr (kSort) {
    if (packed) at = sort_lane<true>(key);
    else if constexpr (kN <= 8) at = sort_lane<false>(key);
  }

  // (a packed value is up to 8 or 16 steps below, 2^-20 or 2^-19 of it: three quarters of
  // that of two which are near each other)
  constexpr float kBelow = kN <= 8 ? 0x1.2p-20f : 0x1.2p-19f;
  const float slack = packed ? (kN <= 8 ? 0x1.cp-21f : 0x1.cp-20f) : 0x1p-22f;
  auto near = [&](uint32_t hi, uint32_t lo) {
    if (packed) hi = unpacked<kN>(hi), lo = unpacked<kN>(lo);
    const float x = value_of(hi), y = value_of(lo);
    return lo > 1u && !(x - y > tol + (fabsf(x) + fabsf(y)) * slack);
  };
  bool redo = false;
  if (groups) {
    uint32_t a, b;
    if (kSort && kN <= 8 && !p.group_lanes) {
      // (by the experts' own places, which sorted keys have lost; a packed key of nothing has
      // no place either, and adds nothing to any)
      uint32_t own[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) own[i] = 0;
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const uint32_t place = place_of<kN>(packed, key[j], at, j);
#pragma unroll
        for (int i = 0; i < kN; ++i) own[i] |= place == static_cast<uint32_t>(i) ? key[j] : 0u;
      }
      group_top2(p, own, lane, false, a, b);
    } else {
      group_top2(p, key, lane, kSort, a, b);
    }
    if (packed) a = unpacked<kN>(a), b = unpacked<kN>(b);
    // keys are logits without a bias: their sums are the scores'
    const bool sums = p.group_top == 2;
    if (!by_score && sums) {
      if (packed) a = whole_bf16(a), b = whole_bf16(b);
      if (a > 1u) a = key_of(score(value_of(a)));
      if (b > 1u) b = key_of(score(value_of(b)));
    }
    const uint32_t total = group_key(p, a, b), mask = take_groups(p, total, lane);
    if (by_score || sums) {
      // The lowest that a group taken may be against the highest that one left may be: a
      // sum has twice a score's error, and what its two parts were rounded by.
      const float v = value_of(total), size = fabsf(value_of(a)) + (sums && b > 1u ? fabsf(value_of(b)) : 0.f);
      const float margin = tol + size * 0x1p-22f;
      const bool taken = mask >> lane & 1u;
      const float least = taken && total != 0 ? (size < kInf ? margin - v : kInf) : -kInf;
      // (a packed -inf may have been the lowest finite value: beside +inf that is +inf, not NaN)
      const bool opposite = total == 1u && a > 1u && b > 1u;
      const float most = taken || (total <= 1u && !opposite) || v == -kInf ? -kInf
                         : size < kInf ? v + margin + (packed ? size * kBelow : 0.f) : kInf;
      const float highest = warp_fmax(most);
      redo = __any_sync(kAll, !taken && total != 0) && !(-warp_fmax(least) > highest);
    }
    const uint32_t in = in_groups<kN>(p, mask, e0);
    if (kSort && kN <= 8 && !p.group_lanes) {
      // (a lane may lie in several groups: its sorted list without those left out)
      uint32_t kept[kN], places = 0;
      int n = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) kept[i] = 0;
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const uint32_t place = place_of<kN>(packed, key[j], at, j);
        if (in >> place & 1u) {
#pragma unroll
          for (int i = 0; i < kN; ++i)
            if (i == n) kept[i] = key[j];
          places |= place << (4 * n);
          ++n;
        }
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) key[i] = kept[i];
      at = places;
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (!(in >> i & 1u)) key[i] = 0;  // (of a sorted list all or none)
    }
  }
  int id;
  uint32_t own;
  if constexpr (kSort) {
    if (packed) pick_sorted<true>(key, at, p.k, lane, id, own);
    else if constexpr (kN <= 8) pick_sorted<false>(key, at, p.k, lane, id, own);
  } else {
    pick(key, p.k, lane, id, own);
  }
  bool fine = true;  // pairs of fp32 may tell
  if (by_score) {
    // lane j against pick j + 1
    uint32_t next = __shfl_down_sync(kAll, own, 1);
    const int next_id = __shfl_down_sync(kAll, id, 1);
    if (p.k == 32) {  // no lane has the runner-up
      const uint32_t left = highest_left<kSort>(key);
      if (lane == 31) next = left;
    }
    const bool close = lane < p.k && near(own, next);
    bool tie = false;
    if (__any_sync(kAll, close)) {
      // the same logit and bias are the same score, and in order
      const bool same = close && lane < 31 && same_expert(p, row, id, next_id);
      tie = __any_sync(kAll, close && !same);
      // (behind a runner-up that is the last pick's like there may be a near one that is not)
      if (!tie && __any_sync(kAll, same && lane == p.k - 1))
        tie = near(__shfl_sync(kAll, own, p.k - 1), highest_left<kSort>(key));
    }
    if constexpr (kSort) {
      if (tie && !redo && !broken && p.k < 31) {
        // More picks, until one lies clear of the one before it; then they are put in
        // order.
        int n = p.k + 1;
        bool clear = !near(__shfl_sync(kAll, own, n - 2), __shfl_sync(kAll, own, n - 1));
        while (!clear && n < 32) {
          clear = !pick_one<true>(key, at, n, lane, id, own);
          if (clear) break;  // no others
          ++n;
          clear = !near(__shfl_sync(kAll, own, n - 2), __shfl_sync(kAll, own, n - 1));
        }
        if (clear) {
          int ordered = id;
          fine = order_picks<T>(p, row, m, n, lane, ordered);
          if (fine) id = ordered, tie = false;
        }
      }
    }
    redo |= tie;
  }
  if (redo && !broken && !(fine && choose_two<T, kN>(p, row, m, lane, id))) {
    float l2[kN];  // (a copy: what a call takes by reference does not stay in registers)
#pragma unroll
    for (int i = 0; i < kN; ++i) l2[i] = l[i];
    choose_64<kN>(p, l2, m, lane, id);
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
  float mine;        // of slot `lane`
  float rest = 0.f;  // what its expert gets besides
  if (!p.sigmoid && !p.renormalize) {
    float l[kN];
    load_row<T, kN>(row, e0, p.E, p.wide, -kInf, l);
    float m = l[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) m = fmaxf(m, l[i]);
    m = warp_fmax(m);
    if (m == -kInf) m = 0.f;  // every expert is out of the choice: scores of 0
    // the fast exponential: off by (2 + 1.2 |l - m|) 2^-24 of a score that falls faster
#pragma unroll
    for (int i = 0; i < kN; ++i) l[i] = __expf(l[i] - m);
    const float sum = warp_add(tree_sum(l));
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float s = have ? __expf(x - m) * inv : 0.f;
    mine = g * s;
    const float dot = warp_add(mine), f = -inv * dot;
#pragma unroll
    for (int i = 0; i < kN; ++i) out[i] = l[i] * f;
    rest = -(s * dot);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) out[i] = 0.f;
    const float s = p.sigmoid ? sigmoid_f32(x) : 0.f;
    const float off = p.sigmoid ? 1.f / (1.f + expf(x)) : 1.f;  // 1 - s
    if (p.renormalize) {
      const float top = warp_fmax(x);
      float u = p.sigmoid && top > -20.f ? s : x == top ? 1.f : expf(x - top);
      if (!have) u = 0.f;
      if (have && x != x) u = x;
      const float total = warp_add(u), q = have ? u / total : 0.f;
      const float dot = warp_add(g * q);
      mine = q * off * (g - dot);
    } else {
      mine = g * s * off;
    }
  }
  T* d_row = static_cast<T*>(p.d_logits) + t * p.ld;
  // an expert in several slots gets their sum
  const uint32_t same = __match_any_sync(kAll, have ? id : -1 - lane);
  if (__any_sync(kAll, (same & (same - 1)) != 0)) {
    for (int j = 0; j < p.k; ++j) {
      const int at = __shfl_sync(kAll, have ? id : -1, j) - e0;
      const float v = __shfl_sync(kAll, mine, j);
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (at == i) out[i] += v;
    }
    store_row<T, kN>(d_row, e0, p.E, p.wide, out);
  } else {  // the row, then the slots' experts over it
    store_row<T, kN>(d_row, e0, p.E, p.wide, out);
    __syncwarp();
    if (have) from_float(d_row[id], mine + rest);
  }
}

template <typename T, int kN>
cudaError_t launch(const RouterParams& p, bool backward, cudaStream_t s) {
  // few tokens: a warp to a block, so that they lie on as many SMs as there are
  const int warps = p.T <= 8 * num_sms() ? 1 : backward ? 8 : kForwardThreads / 32;
  const dim3 grid(static_cast<unsigned>(ceil_div(p.T, warps))), block(32 * warps);
  if (backward) return launch_kernel(router_backward_kernel<T, kN>, grid, block, 0, s, 1, p);
  if constexpr (kN == 16) {
    // Lists of 16 are sorted where packed keys and whole lanes to a group make that enough
    // (us, sorted and not, T=8192 with a bias: E=512 in 8 groups 28.2, 35.2; E=320 without groups
    // 24.8, 32.1; in 64 bits, E=320 without a bias, 33 and 17).
    if (p.bias && (p.topk_groups >= p.groups || p.group_lanes))
      return launch_kernel(router_forward_kernel<T, kN, true>, grid, block, 0, s, 1, p);
  }
  return launch_kernel(router_forward_kernel<T, kN, kN <= 8>, grid, block, 0, s, 1, p);
}

template <typename T>
cudaError_t launch_width(RouterParams p, bool backward, cudaStream_t s) {
  const int n = p.E <= 32 ? 1 : p.E <= 64 ? 2 : p.E <= 128 ? 4 : p.E <= 256 ? 8 : p.E <= 512 ? 16 : 32;
  const uintptr_t all = reinterpret_cast<uintptr_t>(p.logits) |
                        (backward ? reinterpret_cast<uintptr_t>(p.d_logits) : 0);
  p.bias_wide = p.E % n == 0 && reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
  const int lanes = p.per_group / n;
  p.group_lanes = lanes * n == p.per_group && (lanes & (lanes - 1)) == 0 ? lanes : 0;
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
