// Device pieces shared by the kernels that work on whole rows: the 8-bit form
// (include/ec_i8.h) and the norm (include/ec_norm.h).
#ifndef EC_ROW_DEVICE_H
#define EC_ROW_DEVICE_H

#include "ec_mx_device.h"

namespace ecmx {

// A workgroup of kRowThreads has 2^shift lanes along a row, a lane PIECES
// pieces of 8 elements in registers: piece i of a round is the row's chunk
// (round * PIECES + i) * lanes + lane.  Rows of more than one round are read
// again in each pass.
constexpr uint32_t kRowThreads = 256, kRowWaves = kRowThreads / 64;

struct RowShape {
  uint64_t rows;
  uint32_t cols, chunks, shift, rounds;
};

struct RowAt {
  uint64_t row;
  uint32_t slot, lane, lanes;
};
__device__ __forceinline__ RowAt row_at(const RowShape& s, uint64_t block) {
  const uint32_t slot = threadIdx.x >> s.shift;
  return {block * (kRowThreads >> s.shift) + slot, slot, threadIdx.x & ((1u << s.shift) - 1),
          1u << s.shift};
}

// Over the lanes of a row; all of them get the result.  `part` has kRowWaves
// words of LDS that no other reduction of the kernel uses.  Called by the whole
// workgroup.
template <typename V, typename F>
__device__ __forceinline__ V over_row(V v, uint32_t shift, V* part, F&& join) {
  const uint32_t lanes = 1u << shift, within = lanes < 64 ? lanes : 64;
  for (uint32_t m = within / 2; m > 0; m >>= 1) v = join(v, (V)__shfl_xor(v, m));
  if (lanes > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    const uint32_t waves = lanes / 64, w0 = (threadIdx.x >> shift) * waves;
    v = part[w0];
    for (uint32_t i = 1; i < waves; i++) v = join(v, part[w0 + i]);
  }
  return v;
}
__device__ __forceinline__ float sum_over_row(float v, uint32_t shift, float* part) {
  return over_row(v, shift, part, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ uint32_t max_over_row(uint32_t v, uint32_t shift, uint32_t* part) {
  return over_row(v, shift, part, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// The scale of a row of the 8-bit form from the fp32 pattern of its largest
// magnitude, and the number that its elements are divided by.
struct RowScale {
  float scale, by;
};
__device__ __forceinline__ RowScale row_scale(uint32_t pattern) {
  if (pattern >= 0x7f800000u) return {__builtin_nanf(""), __builtin_inff()};
  const float s = bits_as<float>(pattern) / 127.0f;
  return {s, s > 0 ? s : __builtin_inff()};
}
// A row that is not finite is divided by infinity: what is finite in it becomes
// 0, and so does what is NaN.
__device__ __forceinline__ int code_of(float x, float by) {
  float q = __builtin_rintf(x / by);
  q = q == q ? q : 0.0f;
  return (int)__builtin_fminf(__builtin_fmaxf(q, -127.0f), 127.0f);
}
__device__ __forceinline__ uint2 code_row_eight(const float (&f)[8], float by) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; i++) w[i / 4] |= (uint32_t)(code_of(f[i], by) & 255) << (8 * (i % 4));
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

// Lanes for a row of `chunks` pieces: two pieces a lane until 256 lanes, then
// up to 8, then rounds.  Calls go(PIECES).
inline RowShape row_shape(uint64_t rows, uint64_t cols, uint64_t chunks, uint32_t& pieces) {
  RowShape s{};
  s.rows = rows, s.cols = (uint32_t)cols, s.chunks = (uint32_t)chunks;
  s.shift = 4;
  while (s.shift < 8 && (2ull << s.shift) < chunks) s.shift++;
  const uint64_t each = ceil_div(chunks, 1ull << s.shift);
  pieces = each <= 1 ? 1 : each <= 2 ? 2 : each <= 4 ? 4 : 8;
  s.rounds = (uint32_t)ceil_div(each, pieces);
  return s;
}
inline uint64_t row_blocks(const RowShape& s) { return ceil_div(s.rows, kRowThreads >> s.shift); }

}  // namespace ecmx

#endif  // EC_ROW_DEVICE_H
