// The 8-bit integer form (include/ec_i8.h): quantization along rows and its
// inverse.  Both are bound by memory: an element costs its own bytes and one.
#include "ec_i8.h"
#include "ec_row_device.h"

using namespace ecmx;

namespace {

// A row stays in registers between its magnitude and its codes (up to 16384
// elements; longer rows are read twice).  8192 x 8192 bf16: 39 us (5.2 TB/s of bytes
// read and written).
template <typename T, int PIECES>
__global__ __launch_bounds__(kMostThreads) void i8_rows(const T* __restrict__ x, RowShape s,
                                                       uint64_t stride, uint8_t* codes,
                                                       float* scales) {
  __shared__ uint32_t part[kMostWaves];
  const RowAt a = row_at(s, block_number());
  const bool here = a.row < s.rows;
  const T* from = x + (here ? a.row : s.rows - 1) * stride;
  Eight<T> v[PIECES];
  auto load = [&](uint32_t round) {
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      const uint32_t c = (round * PIECES + i) * a.lanes + a.lane;
      v[i] = load_eight(from + (uint64_t)c * 8, (int64_t)s.cols - (int64_t)c * 8);
    }
  };
  uint32_t m = 0;
  for (uint32_t round = 0; round < s.rounds; round++) {
    load(round);
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      float f[8];
      widen(v[i], f);
      const uint32_t n = magnitude_of_floats(f);
      m = m > n ? m : n;
    }
  }
  const RowScale r = row_scale(max_over_row(m, s.shift, part));
  if (!here) return;
  uint8_t* to = codes + a.row * s.chunks * 8;
  for (uint32_t round = 0; round < s.rounds; round++) {
    if (s.rounds > 1) load(round);
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      const uint32_t c = (round * PIECES + i) * a.lanes + a.lane;
      float f[8];
      widen(v[i], f);
      if (c < s.chunks)
        *reinterpret_cast<uint2*>(to + (uint64_t)c * 8) = code_row_eight(f, r);
    }
  }
  if (a.lane == 0) scales[a.row] = r.scale;
}

// 8200 x 5120 to bf16: 19 us (6.6 TB/s).
template <typename T>
__global__ __launch_bounds__(kMostThreads) void i8_values(const uint8_t* __restrict__ codes,
                                                         const float* __restrict__ scales,
                                                         RowShape s, uint64_t padded, T* y,
                                                         uint64_t stride) {
  const RowAt a = row_at(s, block_number());
  if (a.row >= s.rows) return;
  const float scale = scales[a.row];
  for (uint32_t c = a.lane; c < s.chunks; c += a.lanes) {
    const uint2 w = *reinterpret_cast<const uint2*>(codes + a.row * padded + (uint64_t)c * 8);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
      f[i] = in_fp32<T>(scale * (float)(int8_t)((i < 4 ? w.x : w.y) >> (8 * (i % 4))));
    store_eight(y + a.row * stride + (uint64_t)c * 8, (int64_t)s.cols - (int64_t)c * 8,
                narrow<T>(f));
  }
}

// ---------------------------------------------------------------- host

// Under as many rows, each has as many lanes as it can: what counts is when the
// last lane is done.
constexpr uint64_t kFewRows = 64;

ec_status launched() { return hipGetLastError() == hipSuccess ? EC_OK : EC_ERR_DEVICE; }

template <typename T>
ec_status rows_of(const void* x, uint64_t rows, uint64_t cols, uint64_t stride, void* codes,
                  void* scales, hipStream_t stream) {
  uint32_t pieces, threads;
  const bool few = rows < kFewRows;
  const RowShape s =
      row_shape(rows, cols, ec_mx_padded(cols) / 8, few ? 1 : 2, few ? 1 : 2, 64, pieces, threads);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid_of(row_blocks(s, threads)), dim3(threads), 0, stream,
                       (const T*)x, s, stride, (uint8_t*)codes, (float*)scales);
  };
  switch (pieces) {
    case 1: go(i8_rows<T, 1>); break;
    case 2: go(i8_rows<T, 2>); break;
    case 3: go(i8_rows<T, 3>); break;
    default: go(i8_rows<T, 4>);
  }
  return launched();
}

template <typename T>
ec_status values_of(const void* codes, const void* scales, uint64_t rows, uint64_t cols, void* y,
                    uint64_t stride, hipStream_t stream) {
  uint32_t pieces, threads;
  const bool few = rows < kFewRows;
  const RowShape s = row_shape(rows, cols, ceil_div(cols, 8), few ? 1 : 2, few ? 1 : 2, 64, pieces, threads);
  hipLaunchKernelGGL((i8_values<T>), grid_of(row_blocks(s, threads)), dim3(threads), 0, stream,
                     (const uint8_t*)codes, (const float*)scales, s, ec_mx_padded(cols), (T*)y,
                     stride);
  return launched();
}

ec_status check(const void* x, int type, uint64_t rows, uint64_t cols, uint64_t stride,
                const void* codes, const void* scales) {
  if (!type_known(type) || cols == 0 || stride < cols) return EC_ERR_INVALID;
  if (rows > EC_MX_MAX_ROWS || cols > EC_MX_MAX_DEPTH) return EC_ERR_UNSUPPORTED;
  if (rows == 0) return EC_OK;
  return x && aligned(x, type_bytes(type)) && read_ok(codes, scales) ? EC_OK : EC_ERR_INVALID;
}

}  // namespace

extern "C" {

ec_status ec_i8_quantize(const void* x, int type, uint64_t rows, uint64_t cols, uint64_t stride,
                         void* codes, void* scales, void* stream) {
  const ec_status st = check(x, type, rows, cols, stride, codes, scales);
  if (st != EC_OK || rows == 0) return st;
  hipStream_t s = (hipStream_t)stream;
  switch (type) {
    case EC_TYPE_F32: return rows_of<float>(x, rows, cols, stride, codes, scales, s);
    case EC_TYPE_F16: return rows_of<f16_t>(x, rows, cols, stride, codes, scales, s);
    default: return rows_of<bf16_t>(x, rows, cols, stride, codes, scales, s);
  }
}

ec_status ec_i8_dequantize(const void* codes, const void* scales, uint64_t rows, uint64_t cols,
                           void* y, int type, uint64_t stride, void* stream) {
  const ec_status st = check(y, type, rows, cols, stride, codes, scales);
  if (st != EC_OK || rows == 0) return st;
  hipStream_t s = (hipStream_t)stream;
  switch (type) {
    case EC_TYPE_F32: return values_of<float>(codes, scales, rows, cols, y, stride, s);
    case EC_TYPE_F16: return values_of<f16_t>(codes, scales, rows, cols, y, stride, s);
    default: return values_of<bf16_t>(codes, scales, rows, cols, y, stride, s);
  }
}

}  // extern "C"
