// Exchanges and reductions between the lanes of a wave.
#ifndef EC_LANES_DEVICE_H
#define EC_LANES_DEVICE_H

#include <type_traits>

#include "ec_mx_device.h"

namespace ecmx {

// A value of another lane, by a pattern within 4, 8 or 16 lanes.
template <int HOW>
__device__ __forceinline__ uint32_t moved(uint32_t v, std::integral_constant<int, HOW>) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, HOW, 0xf, 0xf, true);
}
template <int HOW>
__device__ __forceinline__ float moved(float v, std::integral_constant<int, HOW> how) {
  return bits_as<float>(moved(bits_as<uint32_t>(v), how));
}
template <int HOW>
__device__ __forceinline__ uint64_t moved(uint64_t v, std::integral_constant<int, HOW> how) {
  return (uint64_t)moved((uint32_t)(v >> 32), how) << 32 | moved((uint32_t)v, how);
}
template <int HOW>
__device__ __forceinline__ double moved(double v, std::integral_constant<int, HOW> how) {
  return bits_as<double>(moved(bits_as<uint64_t>(v), how));
}

// Over aligned runs of 2^shift lanes (1 to 64), by exchanges between registers; all
// lanes get the result.  join(v, other) is given the value of another lane.
template <typename F>
__device__ __forceinline__ uint32_t over_lanes(uint32_t v, uint32_t shift, F&& join) {
  using std::integral_constant;
  if (shift > 0) v = join(v, moved(v, integral_constant<int, 0xb1>{}));   // lanes 1 0 3 2
  if (shift > 1) v = join(v, moved(v, integral_constant<int, 0x4e>{}));   // lanes 2 3 0 1
  if (shift > 2) v = join(v, moved(v, integral_constant<int, 0x141>{}));  // mirrored in 8
  if (shift > 3) v = join(v, moved(v, integral_constant<int, 0x140>{}));  // mirrored in 16
  if (shift > 4) {
    const auto t = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = join(t[0], t[1]);
  }
  if (shift > 5) {
    const auto t = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = join(t[0], t[1]);
  }
  return v;
}
template <typename F>
__device__ __forceinline__ double over_lanes(double v, uint32_t shift, F&& join) {
  using std::integral_constant;
  if (shift > 0) v = join(v, moved(v, integral_constant<int, 0xb1>{}));
  if (shift > 1) v = join(v, moved(v, integral_constant<int, 0x4e>{}));
  if (shift > 2) v = join(v, moved(v, integral_constant<int, 0x141>{}));
  if (shift > 3) v = join(v, moved(v, integral_constant<int, 0x140>{}));
  if (shift > 4) v = join(v, (double)__shfl_xor(v, 16));
  if (shift > 5) v = join(v, (double)__shfl_xor(v, 32));
  return v;
}
__device__ __forceinline__ float max_of(float v, uint32_t shift) {
  return bits_as<float>(over_lanes(bits_as<uint32_t>(v), shift, [](uint32_t a, uint32_t b) {
    return bits_as<float>(b) > bits_as<float>(a) ? b : a;
  }));
}
__device__ __forceinline__ float sum_of(float v, uint32_t shift) {
  return bits_as<float>(over_lanes(bits_as<uint32_t>(v), shift, [](uint32_t a, uint32_t b) {
    return bits_as<uint32_t>(bits_as<float>(a) + bits_as<float>(b));
  }));
}
__device__ __forceinline__ uint32_t max_of(uint32_t v, uint32_t shift) {
  return over_lanes(v, shift, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ double max_of(double v, uint32_t shift) {
  return over_lanes(v, shift, [](double a, double b) { return b > a ? b : a; });
}
__device__ __forceinline__ double sum_of(double v, uint32_t shift) {
  return over_lanes(v, shift, [](double a, double b) { return a + b; });
}
// The high words decide but for ties.
__device__ __forceinline__ uint64_t max_of(uint64_t v, uint32_t shift) {
  const uint32_t hi = max_of((uint32_t)(v >> 32), shift);
  const uint32_t lo = max_of((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u, shift);
  return (uint64_t)hi << 32 | lo;
}

}  // namespace ecmx

#endif  // EC_LANES_DEVICE_H
