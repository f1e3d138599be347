// The microscaled 4-bit format (include/ec_mx.h): quantization along rows,
// along columns, along both in one pass, and its inverse.
//
// All of these are bound by memory: an element costs its own bytes and
// 17/32 of a byte, and a handful of instructions an element pair (the
// magnitude is an integer maximum on packed patterns, the rounding one
// conversion instruction for two elements).
#include <type_traits>

#include "ec_mx_device.h"

using namespace ecmx;

namespace {

constexpr uint32_t kThreads = 256;

// ---------------------------------------------------------------- rows

// A lane takes 8 consecutive elements (16 bytes of a 16-bit type), so a wave
// reads 1 KiB without gaps; 4 lanes share a block and find its magnitude with
// two lane exchanges.  tx lanes lie along a row, 256 / tx rows in a workgroup.
// ROWS rows a lane keep that many loads in flight.  Measured: 212992 x 128 fp32
// 19 us (6.5 TB/s of bytes read and written), 32768 x 4096 bf16 59 us (5.7
// TB/s; a copy of 1 GiB runs at 5.1).
template <typename T, int ROWS>
__global__ __launch_bounds__(kThreads) void mx_rows(const T* __restrict__ x, uint64_t rows,
                                                    uint32_t cols, uint64_t stride,
                                                    uint32_t padded, uint32_t tx_shift,
                                                    uint32_t col_tiles, uint8_t* codes,
                                                    uint8_t* scales) {
  const uint32_t tid = threadIdx.x, ty = kThreads >> tx_shift;
  const uint32_t block = block_number(), ct = block % col_tiles, rt = block / col_tiles;
  const uint32_t chunk = (ct << tx_shift) + (tid & ((1u << tx_shift) - 1));
  const uint64_t row0 = (uint64_t)rt * ty * ROWS + (tid >> tx_shift);
  if (chunk * 8 >= padded) return;  // whole quads of lanes: padded is a multiple of 128
  Eight<T> v[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; i++) {
    const uint64_t row = row0 + (uint64_t)i * ty;
    v[i] = load_eight(x + row * stride + chunk * 8, row < rows ? (int64_t)cols - chunk * 8 : 0);
  }
#pragma unroll
  for (int i = 0; i < ROWS; i++) {
    const uint64_t row = row0 + (uint64_t)i * ty;
    const Scale s = scale_of(exponent_of<T>(max_of_4_lanes(magnitude_of_eight(v[i]))));
    const uint32_t c = code_eight(v[i], s.size);
    if (row < rows) {
      *reinterpret_cast<uint32_t*>(codes + row * (padded / 2) + chunk * 4) = c;
      if ((tid & 3) == 0) scales[row * (padded / 32) + chunk / 4] = (uint8_t)s.byte;
    }
  }
}

// ---------------------------------------------------------------- rows and columns

// The 16 bytes without their first n (n < 16, even), zeros behind.
__device__ __forceinline__ void drop_bytes(uint32_t (&v)[4], uint32_t n) {
  if (n & 8) v[0] = v[2], v[1] = v[3], v[2] = 0, v[3] = 0;
  if (n & 4) v[0] = v[1], v[1] = v[2], v[2] = v[3], v[3] = 0;
  if (n & 2) {
    v[0] = v[0] >> 16 | v[1] << 16, v[1] = v[1] >> 16 | v[2] << 16;
    v[2] = v[2] >> 16 | v[3] << 16, v[3] = v[3] >> 16;
  }
}

// A wave takes 128 rows by 16 lanes of 16 bytes, a lane 32 rows of its 16
// bytes, all in registers (128 of them): the blocks of its columns are then
// its own, their magnitudes and codes need no exchange, and x is read once for
// both directions.  The 4 row blocks of a wave write 64 consecutive bytes of
// a column's codes, and a workgroup's waves (2 by 2) fill whole 128-byte
// lines together.  With two waves a vector unit, loads, some 1400 operations a
// lane and stores overlap only in part: 8200 x 5120 bf16 takes 33 us (3.9
// TB/s), 16 x 2048 x 2048 50 us (4.1 TB/s).  Half the rows a lane and twice
// the waves took 41 us for the first.
template <typename T, bool ROWS, bool COLS>
__global__ __launch_bounds__(kThreads, 2) void mx_both(
    const T* __restrict__ x, uint64_t rows, uint32_t cols, uint64_t batch_stride, uint64_t stride,
    const int32_t* __restrict__ offsets, uint32_t groups, uint32_t col_tiles, uint64_t row_tiles,
    uint8_t* row_codes, uint8_t* row_scales, uint8_t* col_codes, uint8_t* col_scales,
    uint32_t padded_cols, uint64_t padded_rows) {
  constexpr int E = 16 / sizeof(T);  // elements a lane has of a row
  constexpr int W = 16 * E;          // columns of a wave
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t cg = lane & 15, rb = lane >> 4;
  const uint32_t pairs = (col_tiles + 1) / 2;
  const uint32_t ct = 2 * (blockIdx.x % pairs) + (wave >> 1);
  const uint64_t rt = 2 * (uint64_t)(blockIdx.x / pairs) + (wave & 1);
  if (ct >= col_tiles || rt >= row_tiles) return;
  uint64_t first = rt * 128, last = rows;  // this wave's rows
  if (offsets) {
    const GroupTile t = find_tile(offsets, groups, rows, 7, (uint32_t)rt);
    if (t.group == groups) return;
    first = t.first + (uint64_t)t.local * 128;
    last = t.first + t.count;
  }
  x += (uint64_t)blockIdx.z * batch_stride;
  const uint32_t c0 = ct * W + cg * E;
  const uint64_t r0 = first + rb * 32;
  uint32_t v[32][4];
  if (c0 + E <= cols && r0 + 32 <= last) {
#pragma unroll
    for (int i = 0; i < 32; i++) __builtin_memcpy(v[i], x + (r0 + i) * stride + c0, 16);
  } else if (cols >= (uint32_t)E) {
    // An end of the rows or columns: whole pieces from inside the array, the
    // last one of a row from E elements before its end and moved down.
    const uint32_t c = min(c0, cols - E);
    const uint32_t past = (c0 - c) * sizeof(T);  // bytes to drop; 16 and more: all
    const T* from = x + min(r0, last - 1) * stride + c;
#pragma unroll
    for (int i = 0; i < 32; i++) {
      __builtin_memcpy(v[i], from, 16);
      from += r0 + i + 1 < last ? stride : 0;
    }
#pragma unroll
    for (int i = 0; i < 32; i++) {
      const bool none = r0 + i >= last || past >= 16;
      drop_bytes(v[i], past);
#pragma unroll
      for (int j = 0; j < 4; j++) v[i][j] = none ? 0 : v[i][j];
      asm volatile("" : "+v"(v[i][0]), "+v"(v[i][1]), "+v"(v[i][2]), "+v"(v[i][3]));
    }
  } else {
    // rows of less than 16 bytes: by elements, as whole words (as elements,
    // the compiler would carry halves of words to the end of this kernel)
#pragma unroll
    for (int i = 0; i < 32; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        uint32_t w = 0;
#pragma unroll
        for (int h = 0; h < 4 / (int)sizeof(T); h++) {
          const uint32_t col = c0 + j * (4 / sizeof(T)) + h;
          if (r0 + i < last && col < cols) {
            const T* from = x + (r0 + i) * stride + col;
            if constexpr (sizeof(T) == 4) w = *reinterpret_cast<const uint32_t*>(from);
            else w |= (uint32_t) * reinterpret_cast<const uint16_t*>(from) << (16 * h);
          }
        }
        v[i][j] = w;
      }
  }
  if (ROWS && c0 < padded_cols) {
    constexpr uint32_t kShare = 32 / E;  // lanes that share a block
    const uint64_t pitch = padded_cols / 2, spitch = padded_cols / 32;
    const uint32_t mine = lane & (kShare - 1);
    uint8_t* rc = row_codes + ((uint64_t)blockIdx.z * rows + r0) * pitch + c0 / 2;
    uint8_t* rs = row_scales + ((uint64_t)blockIdx.z * rows + r0 + mine) * spitch + c0 / 32;
    // Lanes that share a block store the scales of kShare rows in turn.  The
    // checks of whole tiles are left out: without branches, the rows' chains
    // of short operations overlap.
    auto all_rows = [&](auto whole) {
#pragma unroll
      for (int i0 = 0; i0 < 32; i0 += kShare) {
        uint32_t byte = 0;
#pragma unroll
        for (int k = 0; k < (int)kShare; k++) {
          const int i = i0 + k;
          uint32_t m = magnitude<T>(v[i][0]);
#pragma unroll
          for (int j = 1; j < 4; j++) m = larger<T>(m, magnitude<T>(v[i][j]));
          m = joined<T>(m);
          m = sizeof(T) == 4 ? max_of_8_lanes(m) : max_of_4_lanes(m);
          const Scale s = scale_of(exponent_of<T>(m));
          byte = mine == (uint32_t)k ? s.byte : byte;
          uint32_t c = 0;
          if constexpr (sizeof(T) == 4) {
            c = code_two_f32<0>(c, v[i][0], v[i][1], s.size);
            c = code_two_f32<1>(c, v[i][2], v[i][3], s.size);
          } else {
            c = code_two<T, 0>(c, v[i][0], s.size);
            c = code_two<T, 1>(c, v[i][1], s.size);
            c = code_two<T, 2>(c, v[i][2], s.size);
            c = code_two<T, 3>(c, v[i][3], s.size);
          }
          if (whole || r0 + i < last) {
            if constexpr (sizeof(T) == 4)
              *reinterpret_cast<uint16_t*>(rc + i * pitch) = (uint16_t)c;
            else
              *reinterpret_cast<uint32_t*>(rc + i * pitch) = c;
          }
        }
        if (whole || r0 + i0 + mine < last) rs[i0 * spitch] = (uint8_t)byte;
      }
    };
    if (first + 128 <= last) all_rows(std::true_type{});
    else all_rows(std::false_type{});
  }
  if (COLS && c0 < cols) {
    uint32_t m[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      m[j] = magnitude<T>(v[0][j]);
#pragma unroll
      for (int i = 1; i < 32; i++) m[j] = larger<T>(m[j], magnitude<T>(v[i][j]));
    }
    const uint64_t base = (uint64_t)blockIdx.z * cols + c0;
    uint8_t* cc = col_codes + base * (padded_rows / 2) + rt * 64 + rb * 16;
    uint8_t* cs = col_scales + base * (padded_rows / 32) + rt * 4 + rb;
#pragma unroll
    for (int j = 0; j < E; j++) {
      const int w = sizeof(T) == 4 ? j : j / 2, half = sizeof(T) == 4 ? 0 : j % 2;
      const uint32_t mj = sizeof(T) == 4 ? m[w] : (half ? m[w] >> 16 : m[w] & 0xffffu);
      const Scale s = scale_of(exponent_of<T>(mj));
      const float f = s.size;
      uint32_t c[4] = {0, 0, 0, 0};
      // elements 2i and 2i + 1 of the column side by side: one byte permute
      auto pair = [&](int i) {
        return __builtin_amdgcn_perm(v[i + 1][w], v[i][w], half ? 0x07060302u : 0x05040100u);
      };
#pragma unroll
      for (int q = 0; q < 4; q++) {
        if constexpr (sizeof(T) == 4) {
          c[q] = code_two_f32<0>(c[q], v[8 * q][w], v[8 * q + 1][w], f);
          c[q] = code_two_f32<1>(c[q], v[8 * q + 2][w], v[8 * q + 3][w], f);
          c[q] = code_two_f32<2>(c[q], v[8 * q + 4][w], v[8 * q + 5][w], f);
          c[q] = code_two_f32<3>(c[q], v[8 * q + 6][w], v[8 * q + 7][w], f);
        } else {
          c[q] = code_two<T, 0>(c[q], pair(8 * q), f);
          c[q] = code_two<T, 1>(c[q], pair(8 * q + 2), f);
          c[q] = code_two<T, 2>(c[q], pair(8 * q + 4), f);
          c[q] = code_two<T, 3>(c[q], pair(8 * q + 6), f);
        }
      }
      if (c0 + j < cols) {
        uint4 o = make_uint4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<uint4*>(cc + (uint64_t)j * (padded_rows / 2)) = o;
        cs[(uint64_t)j * (padded_rows / 32)] = (uint8_t)s.byte;
      }
    }
  }
}

// ---------------------------------------------------------------- the values again

// Values of byte SEL of the codes, rounded to T (exact but for fp16 out of its range).
template <typename T, int SEL>
__device__ __forceinline__ void two_values(uint32_t* to, uint32_t c, float f) {
  if constexpr (sizeof(T) == 4) {
    const f32x2 t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, f, SEL);
    to[2 * SEL] = bits_as<uint32_t>(t.x), to[2 * SEL + 1] = bits_as<uint32_t>(t.y);
  } else if constexpr (__is_same(T, bf16_t)) {
    to[SEL] = bits_as<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, SEL));
  } else {
    to[SEL] = bits_as<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, f, SEL));
  }
}

// A lane makes 16 bytes of a row, so that a wave's stores have no gaps (two
// stores of 16 bytes a lane: 29 us instead of 19 for 212992 x 128 fp32, which is
// 6.5 TB/s).
template <typename T, int ROWS>
__global__ __launch_bounds__(kThreads) void mx_values(const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales,
                                                      uint64_t rows, uint32_t cols,
                                                      uint32_t padded, T* y, uint64_t stride,
                                                      uint32_t tx_shift, uint32_t col_tiles,
                                                      bool past) {
  constexpr uint32_t E = 16 / sizeof(T);
  const uint32_t tid = threadIdx.x, ty = kThreads >> tx_shift;
  const uint32_t block = block_number(), ct = block % col_tiles, rt = block / col_tiles;
  const uint32_t c0 = ((ct << tx_shift) + (tid & ((1u << tx_shift) - 1))) * E;
  const uint64_t row0 = (uint64_t)rt * ty * ROWS + (tid >> tx_shift);
  if (c0 >= cols) return;
  uint32_t c[ROWS], s[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; i++) {
    const uint64_t row = row0 + (uint64_t)i * ty;
    c[i] = 0, s[i] = 0;
    if (row < rows) {
      const uint8_t* from = codes + row * (padded / 2) + c0 / 2;
      c[i] = E == 8 ? *reinterpret_cast<const uint32_t*>(from)
                    : *reinterpret_cast<const uint16_t*>(from);
      s[i] = scales[row * (padded / 32) + c0 / 32];
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; i++) {
    const uint64_t row = row0 + (uint64_t)i * ty;
    if (row >= rows) continue;
    const float f = bits_as<float>(s[i] == 0 ? 0x00400000u : s[i] << 23);
    uint32_t v[4];
    two_values<T, 0>(v, c[i], f);
    two_values<T, 1>(v, c[i], f);
    if constexpr (E == 8) {
      two_values<T, 2>(v, c[i], f);
      two_values<T, 3>(v, c[i], f);
    }
    if (s[i] == 255) {  // a block that is not finite
#pragma unroll
      for (int q = 0; q < 4; q++)
        v[q] = sizeof(T) == 4 ? 0x7fc00000u : __is_same(T, bf16_t) ? 0x7fc07fc0u : 0x7e007e00u;
    }
    T* to = y + row * stride + c0;
    if (c0 + E <= cols) {
      store16(to, v, past);
    } else {
      T e[E];
      __builtin_memcpy(e, v, 16);
#pragma unroll
      for (uint32_t j = 0; j < E; j++)
        if (c0 + j < cols) to[j] = e[j];
    }
  }
}

// Lanes along a row: the power of two that covers it, between 16 (128
// elements) and a whole workgroup.
uint32_t lanes_shift(uint64_t chunks) {
  uint32_t s = 4;
  while (s < 8 && (1ull << s) < chunks) s++;
  return s;
}

bool shape_ok(uint64_t rows, uint64_t cols) {
  return rows <= EC_MX_MAX_ROWS && ec_mx_padded(cols) <= EC_MX_MAX_DEPTH;
}

ec_status launched() { return hipGetLastError() == hipSuccess ? EC_OK : EC_ERR_DEVICE; }

// More than one row a lane only where the launch stays large: 4 waves on each
// of the 1024 vector units.  Quantizing bf16, one row and four: 512 x 4096 2.40
// and 2.58 us, 2048 x 4096 4.16 and 3.66, 32768 x 4096 60 and 57.
bool many(uint64_t lanes) { return lanes >= 4 * 1024 * 64 * 4; }

template <typename T>
ec_status rows_of(const void* x, uint64_t rows, uint64_t cols, uint64_t stride, void* codes,
                  void* scales, hipStream_t s) {
  const uint32_t padded = (uint32_t)ec_mx_padded(cols), sh = lanes_shift(padded / 8);
  const uint64_t tiles = ceil_div(padded / 8, 1ull << sh), ty = kThreads >> sh;
  const uint32_t per = many(rows * (padded / 8)) ? 4 : 1;
  const uint64_t blocks = tiles * ceil_div(rows, ty * per);
  if (blocks > kMostBlocks) return EC_ERR_UNSUPPORTED;
  if (per == 4)
    hipLaunchKernelGGL((mx_rows<T, 4>), grid_of(blocks), dim3(kThreads), 0, s,
                       (const T*)x, rows, (uint32_t)cols, stride, padded, sh, (uint32_t)tiles,
                       (uint8_t*)codes, (uint8_t*)scales);
  else
    hipLaunchKernelGGL((mx_rows<T, 1>), grid_of(blocks), dim3(kThreads), 0, s,
                       (const T*)x, rows, (uint32_t)cols, stride, padded, sh, (uint32_t)tiles,
                       (uint8_t*)codes, (uint8_t*)scales);
  return launched();
}

template <typename T>
ec_status both_of(const void* x, uint64_t batch, uint64_t rows, uint64_t cols,
                  uint64_t batch_stride, uint64_t stride, const int32_t* offsets, uint32_t groups,
                  void* rc, void* rs, void* cc, void* cs, hipStream_t s) {
  const uint32_t pc = (uint32_t)ec_mx_padded(cols);
  const uint64_t pr = offsets ? ec_mx_padded_groups(rows, groups) : ec_mx_padded(rows);
  const uint32_t width = 256 / sizeof(T);
  const uint32_t ct = (uint32_t)ceil_div(rc ? pc : cols, width);
  const uint64_t rt = pr / 128;
  const uint64_t blocks = ceil_div(ct, 2) * ceil_div(rt, 2);
  // (an array of 2^24 - 1 workgroups would have 2^40 elements)
  if (blocks * kThreads >> 32) return EC_ERR_UNSUPPORTED;
  const dim3 grid((uint32_t)blocks, 1, (uint32_t)batch), block(kThreads);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, s, (const T*)x, rows, (uint32_t)cols, batch_stride,
                       stride, offsets, groups, ct, rt, (uint8_t*)rc, (uint8_t*)rs, (uint8_t*)cc,
                       (uint8_t*)cs, pc, pr);
  };
  if (rc && cc) go(mx_both<T, true, true>);
  else if (rc) go(mx_both<T, true, false>);
  else go(mx_both<T, false, true>);
  return launched();
}

template <typename T>
ec_status values_of(const void* codes, const void* scales, uint64_t rows, uint64_t cols, void* y,
                    uint64_t stride, hipStream_t s) {
  const uint32_t padded = (uint32_t)ec_mx_padded(cols), E = 16 / sizeof(T);
  const uint32_t sh = lanes_shift(ceil_div(cols, E));
  const uint64_t tiles = ceil_div(ceil_div(cols, E), 1ull << sh), ty = kThreads >> sh;
  const uint32_t per = many(rows * (padded / E)) ? 4 : 1;
  const uint64_t blocks = tiles * ceil_div(rows, ty * per);
  if (blocks > kMostBlocks) return EC_ERR_UNSUPPORTED;
  // Past the caches from 32 MiB on, what the L2 caches hold, where the pieces of
  // 16 bytes are aligned: 212992 x 128 fp32 (104 MiB), quantized and back, 41 us,
  // stored as usual 48; a kernel behind that reads 8192 x 4096 fp32 is done after
  // 57 with it and 51, of 16384 x 4096 (256 MiB) after 108 and 129. Rows of 989
  // and of 6498 fp32 took 42 and 56 so, and take 31 and 41.
  const bool past = stride * sizeof(T) % 16 == 0 && rows * cols * sizeof(T) > (32ull << 20);
  if (per == 4)
    hipLaunchKernelGGL((mx_values<T, 4>), grid_of(blocks), dim3(kThreads), 0, s,
                       (const uint8_t*)codes, (const uint8_t*)scales, rows, (uint32_t)cols, padded,
                       (T*)y, stride, sh, (uint32_t)tiles, past);
  else
    hipLaunchKernelGGL((mx_values<T, 1>), grid_of(blocks), dim3(kThreads), 0, s,
                       (const uint8_t*)codes, (const uint8_t*)scales, rows, (uint32_t)cols, padded,
                       (T*)y, stride, sh, (uint32_t)tiles, past);
  return launched();
}

ec_status both(const void* x, int type, uint64_t batch, uint64_t rows, uint64_t cols,
               uint64_t batch_stride, uint64_t stride, const int32_t* offsets, uint32_t groups,
               void* rc, void* rs, void* cc, void* cs, void* stream) {
  if (!type_known(type) || cols == 0 || stride < cols || (!rc) != (!rs) || (!cc) != (!cs) ||
      (!rc && !cc))
    return EC_ERR_INVALID;
  if ((rc && !written_ok(rc, rs)) || (cc && !written_ok(cc, cs))) return EC_ERR_INVALID;
  if (!shape_ok(rows, cols) || !shape_ok(cols, rows) || batch > EC_MX_MAX_GROUPS)
    return EC_ERR_UNSUPPORTED;
  if (batch * rows == 0) return EC_OK;
  if (!x || !aligned(x, type_bytes(type))) return EC_ERR_INVALID;
  hipStream_t s = (hipStream_t)stream;
  switch (type) {
    case EC_TYPE_F32:
      return both_of<float>(x, batch, rows, cols, batch_stride, stride, offsets, groups, rc, rs,
                            cc, cs, s);
    case EC_TYPE_F16:
      return both_of<f16_t>(x, batch, rows, cols, batch_stride, stride, offsets, groups, rc, rs,
                            cc, cs, s);
    default:
      return both_of<bf16_t>(x, batch, rows, cols, batch_stride, stride, offsets, groups, rc, rs,
                             cc, cs, s);
  }
}

}  // namespace

extern "C" {

uint64_t ec_mx_padded(uint64_t cols) { return (cols + 127) / 128 * 128; }

uint64_t ec_mx_padded_groups(uint64_t rows, uint32_t groups) {
  const uint64_t used = groups < rows ? groups : rows;
  return (rows + 127 * used) / 128 * 128;
}

ec_status ec_mx_quantize(const void* x, int type, uint64_t rows, uint64_t cols, uint64_t stride,
                         void* codes, void* scales, void* stream) {
  if (!type_known(type) || cols == 0 || stride < cols) return EC_ERR_INVALID;
  if (!shape_ok(rows, cols)) return EC_ERR_UNSUPPORTED;
  if (rows == 0) return EC_OK;
  if (!x || !aligned(x, type_bytes(type)) || !written_ok(codes, scales)) return EC_ERR_INVALID;
  hipStream_t s = (hipStream_t)stream;
  switch (type) {
    case EC_TYPE_F32: return rows_of<float>(x, rows, cols, stride, codes, scales, s);
    case EC_TYPE_F16: return rows_of<f16_t>(x, rows, cols, stride, codes, scales, s);
    default: return rows_of<bf16_t>(x, rows, cols, stride, codes, scales, s);
  }
}

ec_status ec_mx_quantize_both(const void* x, int type, uint64_t batch, uint64_t rows,
                              uint64_t cols, uint64_t batch_stride, uint64_t stride,
                              void* row_codes, void* row_scales, void* col_codes,
                              void* col_scales, void* stream) {
  return both(x, type, batch, rows, cols, batch_stride, stride, nullptr, 0, row_codes, row_scales,
              col_codes, col_scales, stream);
}

ec_status ec_mx_quantize_groups(const void* x, int type, uint64_t rows, uint64_t cols,
                                uint64_t stride, const int32_t* offsets, uint32_t groups,
                                void* row_codes, void* row_scales, void* col_codes,
                                void* col_scales, void* stream) {
  if (!offsets || !aligned(offsets, 4) || groups == 0) return EC_ERR_INVALID;
  if (groups > EC_MX_MAX_GROUPS) return EC_ERR_UNSUPPORTED;
  return both(x, type, 1, rows, cols, 0, stride, offsets, groups, row_codes, row_scales, col_codes,
              col_scales, stream);
}

ec_status ec_mx_dequantize(const void* codes, const void* scales, uint64_t rows, uint64_t cols,
                           void* y, int type, uint64_t stride, void* stream) {
  if (!type_known(type) || cols == 0 || stride < cols) return EC_ERR_INVALID;
  if (!shape_ok(rows, cols)) return EC_ERR_UNSUPPORTED;
  if (rows == 0) return EC_OK;
  if (!read_ok(codes, scales) || !y || !aligned(y, type_bytes(type))) return EC_ERR_INVALID;
  hipStream_t s = (hipStream_t)stream;
  switch (type) {
    case EC_TYPE_F32: return values_of<float>(codes, scales, rows, cols, y, stride, s);
    case EC_TYPE_F16: return values_of<f16_t>(codes, scales, rows, cols, y, stride, s);
    default: return values_of<bf16_t>(codes, scales, rows, cols, y, stride, s);
  }
}

}  // extern "C"
