// Device pieces shared by the tile kernels of 4-bit and 8-bit products.
#ifndef EC_TILE_DEVICE_H
#define EC_TILE_DEVICE_H

#include "ec_mx_device.h"

namespace ecmx {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// 16 bytes a lane from base + lane_off + off straight to LDS, 1 KiB from `to` on.
__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t base, uint32_t lane_off,
                                         uint32_t off, uint8_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (__attribute__((address_space(3))) void*)to, 16,
                                           lane_off, off, 0, 0);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const uint8_t* p) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, 0xffffffffu, 0x00027000);
}

// Waits until at most N of this wave's loads are under way and its LDS reads
// have returned, then for the other waves.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(N < 64, "the counter's range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace ecmx

#endif  // EC_TILE_DEVICE_H
