// Device pieces shared by the kernels of the 4-bit format (include/ec_mx.h)
// and of the token exchange (include/ec_experts.h).
#ifndef EC_MX_DEVICE_H
#define EC_MX_DEVICE_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ec_mx.h"

namespace ecmx {

using bf16_t = __bf16;
using f16_t = _Float16;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

inline size_t type_bytes(int type) { return type == EC_TYPE_F32 ? 4 : 2; }
inline bool type_known(int type) {
  return type == EC_TYPE_F32 || type == EC_TYPE_F16 || type == EC_TYPE_BF16;
}
inline bool aligned(const void* p, size_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
// Codes and scales that are written, and that are read: rows of scales start
// at multiples of 4 bytes, so a part of a tensor's rows may.
inline bool written_ok(const void* codes, const void* scales) {
  return codes && scales && aligned(codes, 16) && aligned(scales, 16);
}
inline bool read_ok(const void* codes, const void* scales) {
  return codes && scales && aligned(codes, 16) && aligned(scales, 4);
}
inline uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// A launch has less than 2^32 threads along x: with up to 512 threads a
// workgroup, their numbers past 22 bits go on along y. The last row may have
// more than there is work for: kernels check their numbers anyhow.
constexpr uint32_t kGridBits = 22;
constexpr uint64_t kMostBlocks = 0x7fffffffull;
inline dim3 grid_of(uint64_t blocks) {
  const uint64_t wide = 1ull << kGridBits;
  return blocks <= wide ? dim3((uint32_t)blocks)
                        : dim3((uint32_t)wide, (uint32_t)ceil_div(blocks, wide));
}
__device__ __forceinline__ uint32_t block_number() {
  return blockIdx.y << kGridBits | blockIdx.x;
}

template <typename To, typename From>
__device__ __forceinline__ To bits_as(From v) {
  static_assert(sizeof(To) == sizeof(From), "same size");
  To t;
  __builtin_memcpy(&t, &v, sizeof(t));
  return t;
}

// Eight consecutive elements of a row, as they lie in memory.
template <typename T>
struct Eight {
  static constexpr int kWords = 2 * (int)sizeof(T);
  uint32_t w[kWords];
};

// n of them hold elements of the row (the others read as zero).  The address
// has the alignment of an element: gfx950 takes 16-byte loads from there.
template <typename T>
__device__ __forceinline__ Eight<T> load_eight(const T* p, int64_t n) {
  Eight<T> v;
  if (n >= 8) {
    __builtin_memcpy(&v, p, sizeof(v));
  } else {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; i++) e[i] = i < n ? p[i] : (T)0.0f;
    __builtin_memcpy(&v, e, sizeof(v));
  }
  return v;
}

// Outputs that the caches cannot keep for who reads them are stored past them
// (`past`): lines that wait there only to be written back cost the reads. That
// is from the size of the last-level cache, 256 MiB, on, in rows of whole lines
// of 128 bytes. Measured with a kernel behind that reads the output, stored as
// usual and past: products 16384 x 512 x 16384 in bf16 (512 MiB) 363 and 340 us,
// of half the columns 171 and 173, 8192 x 512 x 8192 83 and 97; rows dispatched,
// 256 MiB of bf16, 160 and 146, 128 MiB 61 and 69. Where lines are in parts:
// 16384 x 512 x 8200 170 and 203, dispatched rows of 250 94 and 102.
inline bool past_caches(uint64_t bytes, uint64_t row_bytes) {
  return row_bytes % 128 == 0 && bytes >= 256ull << 20;
}

// 16 bytes to an address with the alignment of an element.
template <bool PAST, typename T>
__device__ __forceinline__ void store16(T* p, const void* v) {
  typedef int unaligned __attribute__((ext_vector_type(4), aligned(2)));
  unaligned w;
  __builtin_memcpy(&w, v, 16);
  if (PAST) __builtin_nontemporal_store(w, (unaligned*)p);
  else *(unaligned*)p = w;
}
// The same by a branch. The empty statements keep each store as it is: where two
// branches store alike, the compiler would make one store of both, without the
// hint, and of a whole piece and of a ragged one the shared last elements. (They
// also keep other memory operations on their side of the store.)
template <typename T>
__device__ __forceinline__ void store16(T* p, const void* v, bool past) {
  if (past) {
    asm volatile("");
    store16<true>(p, v);
    asm volatile("");
  } else {
    store16<false>(p, v);
    asm volatile("");
  }
}

template <typename T>
__device__ __forceinline__ void store_eight(T* p, int64_t n, const Eight<T>& v,
                                            bool past = false) {
  if (n >= 8) {
    // (two stores of a lane's 32 bytes leave gaps that only the caches close: a
    // dispatch of 16384 x 4 x 4096 fp32 takes 311 us, past them 479)
    store16(p, v.w, sizeof(T) == 2 && past);
    if constexpr (sizeof(T) == 4) store16(p + 4, v.w + 4, false);
  } else {
    T e[8];
    __builtin_memcpy(e, &v, sizeof(v));
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < n) p[i] = e[i];
  }
}

template <typename T>
__device__ __forceinline__ void widen(const Eight<T>& v, float (&f)[8]) {
  T e[8];
  __builtin_memcpy(e, &v, sizeof(v));
#pragma unroll
  for (int i = 0; i < 8; i++) f[i] = (float)e[i];
}

template <typename T>
__device__ __forceinline__ Eight<T> narrow(const float (&f)[8]) {
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; i++) e[i] = (T)f[i];  // to nearest, ties to even
  Eight<T> v;
  __builtin_memcpy(&v, e, sizeof(v));
  return v;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return bits_as<uint32_t>(__builtin_elementwise_max(bits_as<u16x2>(a), bits_as<u16x2>(b)));
}

// Largest magnitude of packed words as the bit pattern of T with the sign
// cleared: magnitudes order as their patterns do, NaN above infinity above
// all numbers, so one integer maximum also finds what is not finite.
template <typename T>
__device__ __forceinline__ uint32_t magnitude(uint32_t w) {
  return w & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu);
}
template <typename T>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  return sizeof(T) == 4 ? (a > b ? a : b) : max_u16x2(a, b);
}
// The two halves of a word of 16-bit magnitudes joined.
template <typename T>
__device__ __forceinline__ uint32_t joined(uint32_t m) {
  if (sizeof(T) == 4) return m;
  const uint32_t lo = m & 0xffffu, hi = m >> 16;
  return lo > hi ? lo : hi;
}

// Exponent field, as fp32 has it, of the magnitude with pattern m of type T.
template <typename T>
__device__ __forceinline__ uint32_t exponent_of(uint32_t m) {
  if constexpr (sizeof(T) == 4) {
    return m >> 23;
  } else if constexpr (__is_same(T, bf16_t)) {
    return m >> 7;
  } else {
    return bits_as<uint32_t>((float)bits_as<f16_t>((uint16_t)m)) >> 23;
  }
}

// A block's scale from the exponent field e of its largest magnitude: the
// byte, and the power of two that elements are divided by, 2^-127 at least.
// A block that is not finite takes 2^126, so that its codes are defined; they
// read as NaN by its byte.
struct Scale {
  uint32_t byte;
  float size;
};
__device__ __forceinline__ Scale scale_of(uint32_t e) {
  const uint32_t s = __builtin_elementwise_sub_sat(e, 2u), bits = s << 23;
  return {e == 255u ? 255u : s, bits_as<float>(bits > 0x00400000u ? bits : 0x00400000u)};
}

// Two elements into byte SEL of `old`.  The conversion instructions round to
// the nearest value, ties to the even code, saturate, take subnormal inputs
// and scales as they are, and turn NaN into 6: checked over all 16-bit
// patterns, and over fp32 values around every border, at 13 scales each.
template <typename T, int SEL>
__device__ __forceinline__ uint32_t code_two(uint32_t old, uint32_t pair, float scale) {
  if constexpr (__is_same(T, bf16_t))
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, bits_as<bf16x2>(pair), scale, SEL);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, bits_as<f16x2>(pair), scale, SEL);
}
template <int SEL>
__device__ __forceinline__ uint32_t code_two_f32(uint32_t old, uint32_t a, uint32_t b,
                                                 float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, bits_as<float>(a), bits_as<float>(b),
                                                  scale, SEL);
}

// Codes of eight elements, the first in the lowest four bits.
template <typename T>
__device__ __forceinline__ uint32_t code_eight(const Eight<T>& v, float scale) {
  uint32_t c = 0;
  if constexpr (sizeof(T) == 4) {
    c = code_two_f32<0>(c, v.w[0], v.w[1], scale);
    c = code_two_f32<1>(c, v.w[2], v.w[3], scale);
    c = code_two_f32<2>(c, v.w[4], v.w[5], scale);
    c = code_two_f32<3>(c, v.w[6], v.w[7], scale);
  } else {
    c = code_two<T, 0>(c, v.w[0], scale);
    c = code_two<T, 1>(c, v.w[1], scale);
    c = code_two<T, 2>(c, v.w[2], scale);
    c = code_two<T, 3>(c, v.w[3], scale);
  }
  return c;
}

template <typename T>
__device__ __forceinline__ uint32_t magnitude_of_eight(const Eight<T>& v) {
  uint32_t m = magnitude<T>(v.w[0]);
#pragma unroll
  for (int i = 1; i < Eight<T>::kWords; i++) m = larger<T>(m, magnitude<T>(v.w[i]));
  return joined<T>(m);
}

// Maximum over aligned groups of 4 or 8 lanes (all lanes get it).
__device__ __forceinline__ uint32_t max_of_4_lanes(uint32_t v) {
  uint32_t t = __builtin_amdgcn_mov_dpp(v, 0xb1, 0xf, 0xf, true);  // lanes 1 0 3 2
  v = v > t ? v : t;
  t = __builtin_amdgcn_mov_dpp(v, 0x4e, 0xf, 0xf, true);  // lanes 2 3 0 1
  return v > t ? v : t;
}
__device__ __forceinline__ uint32_t max_of_8_lanes(uint32_t v) {
  v = max_of_4_lanes(v);
  const uint32_t t = __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true);  // mirrored in 8
  return v > t ? v : t;
}

// Consecutive workgroups go to the 8 XCDs in turn; with this, each XCD takes a
// run of consecutive items, of each of `sets` sets in turn.  The grid is
// `items` rounded up to 8, times sets.
__device__ __forceinline__ bool dealt(uint32_t items, uint32_t sets, uint32_t& t, uint32_t& set) {
  const uint32_t run = (items + 7) / 8, i = block_number() >> 3;
  set = i / run;
  t = (blockIdx.x & 7) * run + (i - set * run);
  return set < sets && t < items;
}

// A group's rows, clamped to [0, rows] so that no offsets lead out of range.
__device__ __forceinline__ void group_rows(const int32_t* offsets, uint32_t g, uint64_t rows,
                                           uint64_t& first, uint64_t& count) {
  const int64_t r = (int64_t)rows;
  int64_t a = offsets[g], b = offsets[g + 1];
  a = a < 0 ? 0 : a > r ? r : a;
  b = b < a ? a : b > r ? r : b;
  first = (uint64_t)a;
  count = (uint64_t)(b - a);
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

struct GroupTile {
  uint32_t group;   // == groups: past the last group's tiles
  uint32_t local;   // the tile's number within its group (past the end: from 0 on)
  uint64_t first;   // the group's first row
  uint64_t count;   // its rows
};

// Which group the tile with number `tile` belongs to, where every group has
// ceil(rows / 2^shift) tiles.  Called by whole waves: lanes look at 64 groups
// at a time.
__device__ __forceinline__ GroupTile find_tile(const int32_t* offsets, uint32_t groups,
                                               uint64_t rows, uint32_t shift, uint32_t tile) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t before = 0;
  for (uint32_t base = 0; base < groups; base += 64) {
    const uint32_t g = base + lane;
    uint64_t first = 0, count = 0;
    if (g < groups) group_rows(offsets, g, rows, first, count);
    const uint32_t n = (uint32_t)((count + (1u << shift) - 1) >> shift);
    uint32_t upto = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t t = __shfl_up(upto, d);
      upto += lane >= (uint32_t)d ? t : 0;
    }
    const uint64_t hit = __ballot(before + upto > tile);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      GroupTile r;
      r.group = base + l;
      r.local = tile - before - (lane_value(upto, l) - lane_value(n, l));
      r.first = lane_value((uint32_t)first, l);  // rows are counted in 31 bits
      r.count = lane_value((uint32_t)count, l);
      return r;
    }
    before += lane_value(upto, 63);
  }
  return {groups, tile - before, 0, 0};
}

// Tiles of 2^shift rows that the groups have, and the rows of no group after them.
__device__ __forceinline__ uint32_t used_tiles(const int32_t* offsets, uint32_t groups,
                                               uint64_t rows, uint32_t shift) {
  const uint32_t lane = threadIdx.x & 63;
  uint64_t sum = 0;
  for (uint32_t g = lane; g < groups; g += 64) {
    uint64_t first, count;
    group_rows(offsets, g, rows, first, count);
    sum += (count + (1u << shift) - 1) >> shift;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  const int64_t end = offsets[groups];
  const uint64_t none = end < 0 ? rows : (uint64_t)end < rows ? rows - (uint64_t)end : 0;
  sum += (none + (1u << shift) - 1) >> shift;
  return (uint32_t)__builtin_amdgcn_readfirstlane(sum > 0x7fffffffull ? 0x7fffffff : (int)sum);
}

// Where group e's part of a transposed, padded row starts (in units of 128).
__device__ __forceinline__ uint32_t group_start(const int32_t* offsets, uint32_t e,
                                                uint64_t rows) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t sum = 0;
  for (uint32_t g = lane; g < e; g += 64) {
    uint64_t first, count;
    group_rows(offsets, g, rows, first, count);
    sum += (uint32_t)((count + 127) >> 7);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)sum);
}

}  // namespace ecmx

#endif  // EC_MX_DEVICE_H
