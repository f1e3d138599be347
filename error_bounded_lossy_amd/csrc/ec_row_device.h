// Device pieces shared by the kernels that work on whole rows: the 8-bit form
// (include/ec_i8.h) and the norm (include/ec_norm.h).
#ifndef EC_ROW_DEVICE_H
#define EC_ROW_DEVICE_H

#include "ec_lanes_device.h"

namespace ecmx {

// A row has 2^shift lanes of a workgroup of 256, or (kWhole) all threads of one of up
// to 512.  A lane has PIECES pieces of 8 elements in registers: piece i of a round is
// the row's chunk (round * PIECES + i) * lanes + lane.  Rows of more than one round are
// read again in each pass.
constexpr uint32_t kRowThreads = 256, kMostThreads = 512, kMostWaves = kMostThreads / 64;
constexpr uint32_t kWhole = 10;

struct RowShape {
  uint64_t rows;
  uint32_t cols, chunks, shift, rounds;
};

struct RowAt {
  uint64_t row;
  uint32_t lane, lanes;
};
__device__ __forceinline__ uint32_t row_slots(uint32_t shift) {
  return shift == kWhole ? 1 : kRowThreads >> shift;
}
__device__ __forceinline__ RowAt row_at(const RowShape& s, uint64_t block) {
  return {block * row_slots(s.shift) + (threadIdx.x >> s.shift),
          threadIdx.x & ((1u << s.shift) - 1), s.shift == kWhole ? blockDim.x : 1u << s.shift};
}

// Over the lanes of a row, from 0 on; all of them get the result.  `part` has
// kMostWaves words of LDS that no other reduction uses until a barrier.  Called by the
// whole workgroup.
template <typename V, typename F>
__device__ __forceinline__ V over_row(V v, uint32_t shift, V* part, F&& join) {
  v = join(v, shift < 6 ? shift : 6);
  if (shift > 6) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    const uint32_t waves = shift == kWhole ? blockDim.x / 64 : 1u << (shift - 6);
    const uint32_t first = (threadIdx.x >> shift) * waves, i = threadIdx.x & (kMostWaves - 1);
    v = i < waves ? part[first + i] : (V)0;
    v = join(v, 3);
  }
  return v;
}
__device__ __forceinline__ float sum_over_row(float v, uint32_t shift, float* part) {
  return over_row(v, shift, part, [](float x, uint32_t n) { return sum_of(x, n); });
}
__device__ __forceinline__ uint32_t max_over_row(uint32_t v, uint32_t shift, uint32_t* part) {
  return over_row(v, shift, part, [](uint32_t x, uint32_t n) { return max_of(x, n); });
}

// The scale of a row of the 8-bit form from the fp32 pattern of its largest
// magnitude, the number that its elements are divided by, and its reciprocal where
// that serves (0: divide).  A row that is not finite is divided by infinity: what
// is finite in it becomes 0, and so does what is NaN.
struct RowScale {
  float scale, by, inverse;
};
__device__ __forceinline__ RowScale row_scale(uint32_t pattern) {
  if (pattern >= 0x7f800000u) return {__builtin_nanf(""), __builtin_inff(), 0};
  const float s = bits_as<float>(pattern) / 127.0f;
  return {s, s > 0 ? s : __builtin_inff(), s >= 0x1p-100f ? 1.0f / s : 0};
}

// A code in the lowest byte: the quotient x / s, rounded to fp32, to a whole number.
// From a reciprocal that is rounded correctly, two steps q += (x - q s) / s give the
// correctly rounded quotient (the first makes it faithful; Markstein's theorem),
// where x - q s is exact: not for scales whose products leave fp32's range below.
// The last addition rounds to a whole number, ties to even, and leaves it in the
// lowest bits.  (The compiler's division takes twice as many instructions.)
__device__ __forceinline__ uint32_t code_of(float x, const RowScale& s) {
  float q = x * s.inverse;
  q = __builtin_fmaf(__builtin_fmaf(-q, s.by, x), s.inverse, q);
  q = __builtin_fmaf(__builtin_fmaf(-q, s.by, x), s.inverse, q);
  return bits_as<uint32_t>(q + 12582912.0f);
}
__device__ __forceinline__ uint32_t code_by_division(float x, const RowScale& s) {
  float q = __builtin_rintf(x / s.by);
  q = q == q ? q : 0.0f;
  return (uint32_t)(int)__builtin_fminf(__builtin_fmaxf(q, -127.0f), 127.0f);
}
__device__ __forceinline__ uint2 code_row_eight(const float (&f)[8], const RowScale& s) {
  uint32_t b[8];
  if (s.inverse != 0) {
#pragma unroll
    for (int i = 0; i < 8; i++) b[i] = code_of(f[i], s);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) b[i] = code_by_division(f[i], s);
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {  // the lowest bytes of four words
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0c0c0400);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x04000c0c);
    w[i] = lo | hi;
  }
  return make_uint2(w[0], w[1]);
}

// Largest magnitude of eight as an fp32 pattern.
__device__ __forceinline__ uint32_t magnitude_of_floats(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t b = bits_as<uint32_t>(f[i]) & 0x7fffffffu;
    m = m > b ? m : b;
  }
  return m;
}

// ---------------------------------------------------------------- host

// Lanes for a row of `chunks` pieces: a power of two while that makes up to 256
// threads of `each` pieces, then a workgroup of as many threads (a multiple of `unit`)
// as give a lane `most` pieces, then up to 512 threads of up to 4 (with most = 1: 512),
// then rounds.
inline RowShape row_shape(uint64_t rows, uint64_t cols, uint64_t chunks, uint32_t each,
                          uint32_t most, uint32_t unit, uint32_t& pieces, uint32_t& threads) {
  RowShape s{};
  s.rows = rows, s.cols = (uint32_t)cols, s.chunks = (uint32_t)chunks;
  s.shift = 4;
  while (s.shift < 8 && ((uint64_t)each << s.shift) < chunks) s.shift++;
  uint64_t lanes = 1ull << s.shift;
  threads = kRowThreads;
  if (each * lanes < chunks) {
    lanes = ceil_div(ceil_div(chunks, most), unit) * unit;
    if (lanes > kMostThreads && most > 1) lanes = ceil_div(ceil_div(chunks, 4), unit) * unit;
    if (lanes > kMostThreads) lanes = kMostThreads;
    s.shift = kWhole;
    threads = (uint32_t)lanes;
  }
  const uint64_t a_lane = ceil_div(chunks, lanes);
  pieces = (uint32_t)(a_lane < 4 ? a_lane : 4);
  s.rounds = (uint32_t)ceil_div(a_lane, pieces);
  return s;
}
inline uint64_t row_blocks(const RowShape& s, uint32_t threads) {
  return ceil_div(s.rows, s.shift == kWhole ? 1 : threads >> s.shift);
}

}  // namespace ecmx

#endif  // EC_ROW_DEVICE_H
