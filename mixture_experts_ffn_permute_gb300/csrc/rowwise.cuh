// Row access shared by the operators around the expert layer: eight elements
// of a row per thread and step, held as loaded (bf16 pairs stay packed), as
// 16-byte vectors where the rows allow it and as single elements otherwise;
// and sums over a row's threads.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace moe {

struct Bf16 {
  uint16_t bits;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(Bf16 x) {
  return __uint_as_float(static_cast<uint32_t>(x.bits) << 16);
}
__device__ __forceinline__ void from_float(float& d, float x) { d = x; }
__device__ __forceinline__ void from_float(Bf16& d, float x) {
  d.bits = __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// 16 bytes that are read (written) once: past L1, so that the weights stay.
__device__ __forceinline__ uint4 load_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void store_stream16(void* p, uint4 v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// 32 bytes (32-byte aligned): a thread's eight fp32 values in one access, so
// that a warp's access covers whole sectors.
__device__ __forceinline__ void load_stream32(float (&f)[8], const float* p) {
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]),
                 "=f"(f[6]), "=f"(f[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store_stream32(float* p, const float (&f)[8]) {
  asm volatile("st.global.L1::no_allocate.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
               "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]),
               "f"(f[7])
               : "memory");
}
// What eight elements of T in one access need of their address.
template <typename T>
__host__ __device__ constexpr int oct_align() { return 8 * static_cast<int>(sizeof(T)); }

// Two fp32 values in one register pair, for the packed fp32 instructions.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(Pair p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ Pair pair_mul(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair pair_fma(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float pair_sum(Pair p) {
  float lo, hi;
  unpair(p, lo, hi);
  return lo + hi;
}

// Eight elements as loaded.
template <typename T>
struct Oct;

template <>
struct Oct<Bf16> {
  uint32_t w[4];
  __device__ __forceinline__ float get(int j) const {
    return (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
  }
  __device__ __forceinline__ Pair pair(int i) const { return pair_of(bf16_lo(w[i]), bf16_hi(w[i])); }
  __device__ __forceinline__ void set_pair(int i, Pair p) {
    float lo, hi;
    unpair(p, lo, hi);
    w[i] = pack_bf16(lo, hi);
  }
  __device__ __forceinline__ void load(const Bf16* p) {
    const uint4 v = load_stream16(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  __device__ __forceinline__ void store(Bf16* p) const {
    store_stream16(p, make_uint4(w[0], w[1], w[2], w[3]));
  }
  __device__ __forceinline__ void set_bits(int j, Bf16 x) {
    if (j & 1) w[j >> 1] |= static_cast<uint32_t>(x.bits) << 16;
    else w[j >> 1] = x.bits;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
  }
};

template <>
struct Oct<float> {
  float f[8];
  __device__ __forceinline__ float get(int j) const { return f[j]; }
  __device__ __forceinline__ Pair pair(int i) const { return pair_of(f[2 * i], f[2 * i + 1]); }
  __device__ __forceinline__ void set_pair(int i, Pair p) { unpair(p, f[2 * i], f[2 * i + 1]); }
  __device__ __forceinline__ void load(const float* p) { load_stream32(f, p); }
  __device__ __forceinline__ void store(float* p) const { store_stream32(p, f); }
  __device__ __forceinline__ void set_bits(int j, float x) { f[j] = x; }
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = x[i];
  }
};

// The columns of step v of thread `tid` of `n` threads on a row: kWide, eight
// neighbours (one access of 16 bytes of bf16, 32 of fp32; the width is a
// multiple of 8); otherwise eight single columns n apart, so that the threads' single
// loads stay coalesced.
template <bool kWide>
__device__ __forceinline__ int oct_col(int v, int j, int tid, int n) {
  return kWide ? (v * n + tid) * 8 + j : (v * 8 + j) * n + tid;
}

template <bool kWide, typename T>
__device__ __forceinline__ void load_oct(Oct<T>& o, const T* row, int v, int tid, int n, int H) {
  if (kWide) {
    const int c = oct_col<true>(v, 0, tid, n);
    if (c < H) {
      o.load(row + c);
    } else {
      const float z[8] = {};
      o.set(z);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = oct_col<false>(v, j, tid, n);
      T x{};
      if (c < H) x = row[c];
      o.set_bits(j, x);
    }
  }
}

template <bool kWide, typename T>
__device__ __forceinline__ void store_oct(const float (&x)[8], T* row, int v, int tid, int n,
                                          int H) {
  if (kWide) {
    const int c = oct_col<true>(v, 0, tid, n);
    if (c < H) {
      Oct<T> o;
      o.set(x);
      o.store(row + c);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = oct_col<false>(v, j, tid, n);
      if (c < H) from_float(row[c], x[j]);
    }
  }
}

// Copies of a warp's octets to shared memory and back, for rows read some rows
// ahead.  Only the warp's own lanes touch them: after copy_async_wait (and
// before the next copy to the same place) __syncwarp is barrier enough.  A
// step of n threads takes n * 16 bytes (bf16) or n * 32 (fp32, where lane l
// copies the 16-byte pieces l and 32 + l of the warp's 1 KB, so that every
// copy of a warp is contiguous; bit 3 of a piece's number flips its lowest
// bit, which keeps the lanes' reads of two neighbouring pieces free of bank
// conflicts).
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most `pending` (0 .. 3) of this thread's groups are under way.
__device__ __forceinline__ void copy_async_wait(int pending) {
  if (pending >= 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (pending == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (pending == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ uint4 load_shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src)
               : "memory");
  return v;
}
// row: the row's first element; c: this thread's first column in the step.
__device__ __forceinline__ void oct_copy(uint32_t step, const Bf16* row, int c, int tid, int H) {
  if (c < H) copy_async16(step + tid * 16, row + c);
}
__device__ __forceinline__ void oct_copy(uint32_t step, const float* row, int c, int tid, int H) {
  const int lane = tid & 31;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int piece = h * 32 + lane, col = c - lane * 8 + piece * 4;
    if (col < H)
      copy_async16(step + (tid - lane) * 32 + (piece ^ ((piece >> 3) & 1)) * 16, row + col);
  }
}
__device__ __forceinline__ void oct_read(Oct<Bf16>& o, uint32_t step, int tid) {
  const uint4 v = load_shared16(step + tid * 16);
  o.w[0] = v.x, o.w[1] = v.y, o.w[2] = v.z, o.w[3] = v.w;
}
__device__ __forceinline__ void oct_read(Oct<float>& o, uint32_t step, int tid) {
  const int lane = tid & 31;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int piece = 2 * lane + h;
    const uint4 v = load_shared16(step + (tid - lane) * 32 + (piece ^ ((piece >> 3) & 1)) * 16);
    o.f[4 * h] = __uint_as_float(v.x), o.f[4 * h + 1] = __uint_as_float(v.y);
    o.f[4 * h + 2] = __uint_as_float(v.z), o.f[4 * h + 3] = __uint_as_float(v.w);
  }
}

// Dense rows of any width: row r of [T, H] is the elements [r H, (r + 1) H) of one
// sequence, and the octets are the sequence's, so that every access is wide and
// aligned.  Octet k of the row starts at column 8 k - shift, shift = r H mod 8;
// a row's first and last octets hold elements of the rows beside it, which are
// masked after a read and left alone by a write.
__device__ __forceinline__ bool oct_whole(int c, int H) { return c >= 0 && c + 8 <= H; }
__device__ __forceinline__ bool oct_inside(int c, int H) { return c + 8 > 0 && c < H; }
__device__ __forceinline__ void oct_mask(Oct<Bf16>& o, int c, int H) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < 0 || c + j >= H) o.w[j >> 1] &= (j & 1) ? 0x0000ffffu : 0xffff0000u;
}
__device__ __forceinline__ void oct_mask(Oct<float>& o, int c, int H) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < 0 || c + j >= H) o.f[j] = 0.f;
}
// m elements of the row from column c on (the first of them may lie before it,
// and the last behind the tensor's end: those are not copied) to shared memory.
template <typename T>
__device__ __forceinline__ void flat_piece(uint32_t dst, const T* row, int c, int m, int H,
                                           const T* end) {
  if (c + m <= 0 || c >= H) return;
  if (row + c + m <= end) {
    copy_async16(dst, row + c);
    return;
  }
  for (int j = 0; j < m && c + j < H; ++j) {
    if (c + j < 0) continue;
    const uint32_t at = dst + j * static_cast<int>(sizeof(T));
    if constexpr (sizeof(T) == 2)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(row[c + j].bits) : "memory");
    else
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(row[c + j]) : "memory");
  }
}
__device__ __forceinline__ void flat_copy(uint32_t step, const Bf16* row, int c, int tid, int H,
                                          const Bf16* end) {
  flat_piece(step + tid * 16, row, c, 8, H, end);
}
__device__ __forceinline__ void flat_copy(uint32_t step, const float* row, int c, int tid, int H,
                                          const float* end) {
  const int lane = tid & 31;
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // the layout of oct_copy
    const int piece = h * 32 + lane;
    flat_piece(step + (tid - lane) * 32 + (piece ^ ((piece >> 3) & 1)) * 16, row,
               c - lane * 8 + piece * 4, 4, H, end);
  }
}

// A weight vector whose type is known at run time only (bf16 or fp32).
struct WeightPtr {
  const void* p;
  bool f32;
  __device__ __forceinline__ float at(long c) const {
    return f32 ? __ldg(static_cast<const float*>(p) + c)
               : __uint_as_float(
                     static_cast<uint32_t>(__ldg(static_cast<const unsigned short*>(p) + c)) << 16);
  }
};

template <bool kWide>
__device__ __forceinline__ void load_weight8(float (&x)[8], const WeightPtr& w, long at0, int v,
                                             int tid, int n, int H) {
  if (kWide) {
    const int c = oct_col<true>(v, 0, tid, n);
    if (c >= H) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
    } else if (w.f32) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(w.p) + at0 + c);
      const float4 a = __ldg(q), b = __ldg(q + 1);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
      x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
      const uint4 a =
          __ldg(reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(w.p) + at0 + c));
      x[0] = bf16_lo(a.x), x[1] = bf16_hi(a.x), x[2] = bf16_lo(a.y), x[3] = bf16_hi(a.y);
      x[4] = bf16_lo(a.z), x[5] = bf16_hi(a.z), x[6] = bf16_lo(a.w), x[7] = bf16_hi(a.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = oct_col<false>(v, j, tid, n);
      x[j] = c < H ? w.at(at0 + c) : 0.f;
    }
  }
}

// The weights at0 + [c, c + 8); zeros outside the row.  wide: a whole octet is
// aligned.
__device__ __forceinline__ void load_weight_cols(float (&x)[8], const WeightPtr& w, long at0,
                                                 int c, int H, bool wide) {
  if (wide && oct_whole(c, H)) {
    load_weight8<true>(x, w, at0 + c, 0, 0, 1, 8);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = c + j >= 0 && c + j < H ? w.at(at0 + c + j) : 0.f;
}

// Sums over the threads of one row, every thread getting the totals.  kWarp:
// the row's threads are one warp.  Otherwise they are the block, `s` is
// kN * 32 floats of shared memory that the next call must not share with this
// one (two buffers alternate), and the order of the sum is fixed.
template <bool kWarp, int kN>
__device__ __forceinline__ void row_sum(float (&x)[kN], float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
  if (kWarp) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i * 32 + warp] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    x[i] = lane < nw ? s[i * 32 + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
  }
}

}  // namespace moe
