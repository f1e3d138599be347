// The root-mean-square norm with the residual's addition (include/ec_norm.h),
// its output in x's type or in the 8-bit form, and its gradients.  All of it is
// bound by memory.
#include <cmath>

#include "ec_norm.h"
#include "ec_row_device.h"

using namespace ecmx;

namespace {

// Eight weights from element c on; those past the row's end are zero.
__device__ __forceinline__ void weights_at(const void* w, int type, uint64_t c, int64_t n,
                                           float (&f)[8]) {
  if (type == EC_TYPE_F32) widen(load_eight((const float*)w + c, n), f);
  else if (type == EC_TYPE_F16) widen(load_eight((const f16_t*)w + c, n), f);
  else widen(load_eight((const bf16_t*)w + c, n), f);
}

struct Norm {
  const void *x, *residual, *weight;
  uint64_t stride, residual_stride;
  int wtype;
  float eps;
  void *h, *y;      // y: rows of x's type, or codes
  float* scales;    // of codes
  float* rstd;
};

// One pass over x and the residual: the row stays in registers (up to 16384
// elements; longer rows are read again from h, or x, in each pass).  The weights
// are asked for before the sum is known (one row of 8192 into 8 bits: 4.1 us, 6.3
// with them behind the sum and 256 lanes).  Bound by memory: 16384 x 4096 bf16 with
// residual 86 us (6.2 TB/s of bytes read and written; a copy of 1 GiB 5.1), 8200 x
// 5120 into 8 bits 61 us (4.8 TB/s).
template <typename T, int PIECES, bool EIGHT_BITS>
__global__ __launch_bounds__(kMostThreads) void rms_norm(const Norm p, RowShape s) {
  __shared__ float sums[kMostWaves];
  __shared__ uint32_t tops[kMostWaves];
  const RowAt a = row_at(s, block_number());
  const bool here = a.row < s.rows;
  const uint64_t row = here ? a.row : s.rows - 1;
  const T* x = (const T*)p.x + row * p.stride;
  const T* residual = p.residual ? (const T*)p.residual + row * p.residual_stride : nullptr;
  T* h = p.h ? (T*)p.h + row * s.cols : nullptr;
  auto chunk = [&](uint32_t round, int i) { return (round * PIECES + i) * a.lanes + a.lane; };
  auto left = [&](uint32_t c) { return (int64_t)s.cols - (int64_t)c * 8; };
  Eight<T> v[PIECES];
  float w[PIECES][8];
  auto load_weights = [&](uint32_t round) {
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      const uint32_t c = chunk(round, i);
      weights_at(p.weight, p.wtype, (uint64_t)c * 8, left(c), w[i]);
    }
  };
  float sum = 0;
  for (uint32_t round = 0; round < s.rounds; round++) {
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      const uint32_t c = chunk(round, i);
      v[i] = load_eight(x + (uint64_t)c * 8, left(c));
    }
    if (residual) {
      Eight<T> r[PIECES];
#pragma unroll
      for (int i = 0; i < PIECES; i++) {
        const uint32_t c = chunk(round, i);
        r[i] = load_eight(residual + (uint64_t)c * 8, left(c));
      }
      if (s.rounds == 1) load_weights(0);
#pragma unroll
      for (int i = 0; i < PIECES; i++) {
        const uint32_t c = chunk(round, i);
        float f[8], g[8];
        widen(v[i], f);
        widen(r[i], g);
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] += g[j];
        v[i] = narrow<T>(f);
        if (here) store_eight(h + (uint64_t)c * 8, left(c), v[i]);
      }
    } else if (s.rounds == 1) {
      load_weights(0);
    }
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      float f[8];
      widen(v[i], f);
#pragma unroll
      for (int j = 0; j < 8; j++) sum += f[j] * f[j];
    }
  }
  sum = sum_over_row(sum, s.shift, sums);
  const float rstd = 1.0f / __builtin_sqrtf(sum / (float)s.cols + p.eps);
  if (here && p.rstd && a.lane == 0) p.rstd[row] = rstd;
  const T* again = residual ? h : x;
  auto normed = [&](uint32_t round, int i, float (&f)[8]) {
    const uint32_t c = chunk(round, i);
    if (s.rounds > 1) {
      weights_at(p.weight, p.wtype, (uint64_t)c * 8, left(c), w[i]);
      v[i] = load_eight(again + (uint64_t)c * 8, left(c));
    }
    widen(v[i], f);
#pragma unroll
    for (int j = 0; j < 8; j++) f[j] = f[j] * rstd * w[i][j];
  };
  if constexpr (!EIGHT_BITS) {
    T* y = (T*)p.y + row * s.cols;
    for (uint32_t round = 0; round < s.rounds; round++)
#pragma unroll
      for (int i = 0; i < PIECES; i++) {
        const uint32_t c = chunk(round, i);
        float f[8];
        normed(round, i, f);
        if (here) store_eight(y + (uint64_t)c * 8, left(c), narrow<T>(f));
      }
  } else {
    uint32_t m = 0;
    for (uint32_t round = 0; round < s.rounds; round++)
#pragma unroll
      for (int i = 0; i < PIECES; i++) {
        float f[8];
        normed(round, i, f);
        const uint32_t n = magnitude_of_floats(f);
        m = m > n ? m : n;
        if (s.rounds == 1)  // the products take the weights' place
#pragma unroll
          for (int j = 0; j < 8; j++) w[i][j] = f[j];
      }
    const RowScale r = row_scale(max_over_row(m, s.shift, tops));
    if (!here) return;
    uint8_t* codes = (uint8_t*)p.y + row * s.chunks * 8;
    for (uint32_t round = 0; round < s.rounds; round++)
#pragma unroll
      for (int i = 0; i < PIECES; i++) {
        const uint32_t c = chunk(round, i);
        float f[8];
        if (s.rounds > 1) normed(round, i, f);
        if (c < s.chunks)
          *reinterpret_cast<uint2*>(codes + (uint64_t)c * 8) =
              code_row_eight(s.rounds > 1 ? f : w[i], r);
      }
    if (a.lane == 0) p.scales[row] = r.scale;
  }
}

// ---------------------------------------------------------------- gradients

struct Back {
  const void *dy, *h, *dh, *weight;
  const float* rstd;
  int wtype;
  void* dx;
  float* parts;  // dweight's parts [gridDim * slots][cols]; NULL: another kernel sums it
};

// Rows that a lane adds up one after the other, before their sum is added to what
// those before gave: however long a batch is, it is off by 256 roundings and one for each
// run (of 64 rows, the way through memory costs 3 %: 131072 x 4096 bf16 694 us for 672).
constexpr uint32_t kRun = 256;

// dx = rstd (w dy - n mean(w dy n)) + dh with n = h rstd: the mean is one sum over the
// row.  A workgroup takes every gridDim-th set of rows and adds up what they give to
// dweight in registers; the next set's rows are on their way while it works on one
// (without: 16384 x 4096 bf16 141 us, with the column sums, for 114).  Bound by memory:
// 117 us of it in this kernel among others, 4.6 TB/s.
template <typename T, int PIECES>
__global__ __launch_bounds__(kMostThreads) void rms_norm_back(const Back p, RowShape s) {
  __shared__ float sums[2][kMostWaves];
  // (of four pieces, and of three in fp32, the registers hold one row: 2000 x 16384 bf16
  // 45 us, else 67; 8200 x 5120 fp32 100, else 155)
  constexpr bool kAhead = PIECES <= (sizeof(T) == 4 ? 2 : 3);
  const uint64_t sets = (s.rows + row_slots(s.shift) - 1) / row_slots(s.shift);
  struct Row {
    Eight<T> dy[PIECES], h[PIECES], dh[PIECES];
    float rstd;
  };
  auto chunk = [&](const RowAt& a, uint32_t round, int i) {
    return (round * PIECES + i) * a.lanes + a.lane;
  };
  auto left = [&](uint32_t c) { return (int64_t)s.cols - (int64_t)c * 8; };
  auto load = [&](uint64_t set, uint32_t round, Row& r) {
    const RowAt a = row_at(s, set);
    const bool here = a.row < s.rows;
    const uint64_t row = here ? a.row : s.rows - 1;
    r.rstd = p.rstd[row];
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      const uint32_t c = chunk(a, round, i);
      const uint64_t at = row * s.cols + (uint64_t)c * 8;
      const int64_t n = here ? left(c) : 0;
      r.dy[i] = load_eight((const T*)p.dy + at, n);
      r.h[i] = load_eight((const T*)p.h + at, n);
      if (p.dh) r.dh[i] = load_eight((const T*)p.dh + at, n);
    }
  };
  float w[PIECES][8], dw[PIECES][8] = {};
  auto load_weights = [&](uint32_t round) {
    const RowAt a = row_at(s, 0);
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      const uint32_t c = chunk(a, round, i);
      weights_at(p.weight, p.wtype, (uint64_t)c * 8, left(c), w[i]);
    }
  };
  // What the lane has summed goes to this slot's part, on top of what is there already,
  // and the lane begins anew.
  auto put = [&](bool first) {
    const RowAt a = row_at(s, blockIdx.x);
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      const uint32_t c = chunk(a, 0, i);
      float* to = p.parts + a.row * s.cols + (uint64_t)c * 8;
      if (!first) {
        float f[8];
        widen(load_eight(to, left(c)), f);
#pragma unroll
        for (int j = 0; j < 8; j++) dw[i][j] += f[j];
      }
      store_eight(to, left(c), narrow<float>(dw[i]));
#pragma unroll
      for (int j = 0; j < 8; j++) dw[i][j] = 0;
    }
  };
  Row now, next;
  if (s.rounds == 1) load_weights(0);
  load(blockIdx.x, 0, now);
  uint64_t set = blockIdx.x;
  uint32_t turn = 0;
  for (bool first = true; set < sets; first = false) {
    const uint64_t run = set + (uint64_t)gridDim.x * kRun, end = run < sets ? run : sets;
    for (; set < end; set += gridDim.x, turn ^= 1) {
      const RowAt a = row_at(s, set);
      const bool more = set + gridDim.x < sets;
      float dot = 0;
      for (uint32_t round = 0; round < s.rounds; round++) {
        if (s.rounds > 1) {
          load(set, round, now);
          load_weights(round);
        } else if (kAhead && more) {
          load(set + gridDim.x, 0, next);
        }
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
          float f[8], g[8];
          widen(now.dy[i], f);
          widen(now.h[i], g);
#pragma unroll
          for (int j = 0; j < 8; j++) {
            const float n = g[j] * now.rstd;
            dot += f[j] * w[i][j] * n;
            dw[i][j] += f[j] * n;
          }
        }
      }
      // two sets of words in turn: a wave may be one row ahead of another
      dot = sum_over_row(dot, s.shift, sums[turn]) / (float)s.cols;
      if (a.row < s.rows)
        for (uint32_t round = 0; round < s.rounds; round++) {
          if (s.rounds > 1) {
            load(set, round, now);
            load_weights(round);
          }
#pragma unroll
          for (int i = 0; i < PIECES; i++) {
            const uint32_t c = chunk(a, round, i);
            float f[8], g[8], o[8] = {};
            widen(now.dy[i], f);
            widen(now.h[i], g);
            if (p.dh) widen(now.dh[i], o);
#pragma unroll
            for (int j = 0; j < 8; j++)
              o[j] += now.rstd * (f[j] * w[i][j] - g[j] * now.rstd * dot);
            store_eight((T*)p.dx + a.row * s.cols + (uint64_t)c * 8, left(c), narrow<T>(o));
          }
        }
      if (s.rounds == 1 && more) {
        if (kAhead) now = next;
        else load(set + gridDim.x, 0, now);
      }
    }
    if (p.parts) put(first);
  }
}

constexpr uint32_t kSumCols = 32, kSumSlices = 32, kSumAhead = 8;

// Column sums of [parts][cols]: 32 columns a workgroup, their rows in 32 slices
// that are joined in order, 8 rows of a slice on their way at a time (512 x 4096: 4.9
// us; one at a time, of 1024 parts, 13).  In 64 bits, which costs nothing beside the
// loads: 1001 x 1111 fp32 is off by 7.0e-8 then, 1.5e-7 in 32.
struct PartRows {
  const float* parts;
  uint64_t rows;
  uint32_t cols;
  __device__ float at(uint64_t r, uint32_t c) const { return parts[r * cols + c]; }
};
// The same of dy times n, where a row is too long for one workgroup's registers.
template <typename T>
struct GradientRows {
  const T *dy, *h;
  const float* rstd;
  uint64_t rows;
  uint32_t cols;
  __device__ float at(uint64_t r, uint32_t c) const {
    return (float)dy[r * cols + c] * ((float)h[r * cols + c] * rstd[r]);
  }
};
template <typename F>
__global__ __launch_bounds__(kSumCols* kSumSlices) void column_sums(const F from, void* to,
                                                                    int type) {
  __shared__ double part[kSumSlices][kSumCols + 1];
  const uint32_t col = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
  const uint64_t c = (uint64_t)blockIdx.x * kSumCols + col;
  double sum = 0;
  if (c < from.cols)
    for (uint64_t r0 = slice; r0 < from.rows; r0 += kSumSlices * kSumAhead) {
      // (rows past the end read the last one: of a load behind a branch, the conversion
      // to 64 bits would wait there, 6.4 us)
      float v[kSumAhead];
#pragma unroll
      for (int i = 0; i < (int)kSumAhead; i++) {
        const uint64_t r = r0 + i * kSumSlices;
        v[i] = from.at(r < from.rows ? r : from.rows - 1, (uint32_t)c);
      }
#pragma unroll
      for (int i = 0; i < (int)kSumAhead; i++)
        sum += r0 + i * kSumSlices < from.rows ? (double)v[i] : 0.0;
    }
  part[slice][col] = sum;
  __syncthreads();
  if (slice || c >= from.cols) return;
  sum = 0;
  for (uint32_t i = 0; i < kSumSlices; i++) sum += part[i][col];
  if (type == EC_TYPE_F32) ((float*)to)[c] = (float)sum;
  else if (type == EC_TYPE_F16) ((f16_t*)to)[c] = (f16_t)(float)sum;
  else ((bf16_t*)to)[c] = (bf16_t)(float)sum;
}

// ---------------------------------------------------------------- host

ec_status launched() { return hipGetLastError() == hipSuccess ? EC_OK : EC_ERR_DEVICE; }
bool fine(const void* p, size_t to) { return p && aligned(p, to); }

// What forward and backward ask of sizes and types.
ec_status check(int type, int wtype, uint64_t rows, uint64_t cols) {
  if (!type_known(type) || !type_known(wtype) || cols == 0) return EC_ERR_INVALID;
  return rows > EC_MX_MAX_ROWS || cols > EC_MX_MAX_DEPTH ? EC_ERR_UNSUPPORTED : EC_OK;
}

ec_status check_norm(const Norm& p, int type, uint64_t rows, uint64_t cols) {
  const ec_status st = check(type, p.wtype, rows, cols);
  if (st != EC_OK) return st;
  if (p.stride < cols || (!p.residual) != (!p.h) || (p.residual && p.residual_stride < cols) ||
      !(p.eps > 0) || !std::isfinite(p.eps))
    return EC_ERR_INVALID;
  if (rows == 0) return EC_OK;
  const size_t b = type_bytes(type);
  return fine(p.x, b) && aligned(p.residual, b) && aligned(p.h, b) &&
                 fine(p.weight, type_bytes(p.wtype)) && aligned(p.rstd, 4)
             ? EC_OK
             : EC_ERR_INVALID;
}

// Under as many rows, each has as many lanes as it can: what counts is when the
// last lane is done.
constexpr uint64_t kFewRows = 64;

template <typename T, bool EIGHT_BITS>
ec_status norm_as(const Norm& p, uint64_t rows, uint64_t cols, hipStream_t stream) {
  uint32_t pieces, threads;
  const bool few = rows < kFewRows;
  const RowShape s = row_shape(rows, cols, EIGHT_BITS ? ec_mx_padded(cols) / 8 : ceil_div(cols, 8),
                               few ? 1 : 2, few ? 1 : 2, 64, pieces, threads);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid_of(row_blocks(s, threads)), dim3(threads), 0, stream, p, s);
  };
  switch (pieces) {
    case 1: go(rms_norm<T, 1, EIGHT_BITS>); break;
    case 2: go(rms_norm<T, 2, EIGHT_BITS>); break;
    case 3: go(rms_norm<T, 3, EIGHT_BITS>); break;
    default: go(rms_norm<T, 4, EIGHT_BITS>);
  }
  return launched();
}
template <bool EIGHT_BITS>
ec_status norm(const Norm& p, int type, uint64_t rows, uint64_t cols, hipStream_t s) {
  switch (type) {
    case EC_TYPE_F32: return norm_as<float, EIGHT_BITS>(p, rows, cols, s);
    case EC_TYPE_F16: return norm_as<f16_t, EIGHT_BITS>(p, rows, cols, s);
    default: return norm_as<bf16_t, EIGHT_BITS>(p, rows, cols, s);
  }
}

// Whole workgroups of 256 or 512 threads (a unit holds two of 256: one of 320 leaves
// it half empty), with two pieces a lane where that makes a row: two rows and
// dweight's sums fit its registers.
RowShape back_shape(uint64_t rows, uint64_t cols, uint32_t& pieces, uint32_t& threads) {
  return row_shape(rows, cols, ceil_div(cols, 8), 2, 3, kRowThreads, pieces, threads);
}
uint32_t slots_of(const RowShape& s, uint32_t threads) {
  return s.shift == kWhole ? 1 : threads >> s.shift;
}
// Workgroups of the backward pass: as many as the units hold at a time, and two rows
// a slot at least, so that dweight's parts stay below half of dy's elements.
uint32_t back_blocks(const RowShape& s, uint32_t threads) {
  const uint64_t n = ceil_div(row_blocks(s, threads), 2), most = 512 * kRowThreads / threads;
  return (uint32_t)(n > most ? most : n);
}

template <typename T>
ec_status back_as(Back p, uint64_t rows, uint64_t cols, void* dweight, void* workspace,
                  hipStream_t stream) {
  uint32_t pieces, threads;
  const RowShape s = back_shape(rows, cols, pieces, threads);
  p.parts = s.rounds == 1 ? (float*)workspace : nullptr;
  const uint32_t blocks = back_blocks(s, threads);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(threads), 0, stream, p, s);
  };
  if (rows) {
    switch (pieces) {
      case 1: go(rms_norm_back<T, 1>); break;
      case 2: go(rms_norm_back<T, 2>); break;
      case 3: go(rms_norm_back<T, 3>); break;
      default: go(rms_norm_back<T, 4>);
    }
  }
  const dim3 grid((uint32_t)ceil_div(cols, kSumCols)), block(kSumCols * kSumSlices);
  if (p.parts || !rows) {
    const PartRows f{p.parts, rows ? blocks * (uint64_t)slots_of(s, threads) : 0, s.cols};
    hipLaunchKernelGGL((column_sums<PartRows>), grid, block, 0, stream, f, dweight, p.wtype);
  } else {
    const GradientRows<T> f{(const T*)p.dy, (const T*)p.h, p.rstd, rows, s.cols};
    hipLaunchKernelGGL((column_sums<GradientRows<T>>), grid, block, 0, stream, f, dweight,
                       p.wtype);
  }
  return launched();
}

}  // namespace

extern "C" {

ec_status ec_rms_norm(const void* x, uint64_t stride, const void* residual,
                      uint64_t residual_stride, int type, uint64_t rows, uint64_t cols,
                      const void* weight, int wtype, float eps, void* h, void* y, float* rstd,
                      void* stream) {
  const Norm p{x, residual, weight, stride, residual_stride, wtype, eps, h, y, nullptr, rstd};
  const ec_status st = check_norm(p, type, rows, cols);
  if (st != EC_OK || rows == 0) return st;
  if (!fine(y, type_bytes(type))) return EC_ERR_INVALID;
  return norm<false>(p, type, rows, cols, (hipStream_t)stream);
}

ec_status ec_rms_norm_i8(const void* x, uint64_t stride, const void* residual,
                         uint64_t residual_stride, int type, uint64_t rows, uint64_t cols,
                         const void* weight, int wtype, float eps, void* h, void* codes,
                         void* scales, void* stream) {
  const Norm p{x,   residual, weight, stride,         residual_stride, wtype,
               eps, h,        codes,  (float*)scales, nullptr};
  const ec_status st = check_norm(p, type, rows, cols);
  if (st != EC_OK || rows == 0) return st;
  if (!read_ok(codes, scales)) return EC_ERR_INVALID;
  return norm<true>(p, type, rows, cols, (hipStream_t)stream);
}

size_t ec_rms_norm_backward_workspace_bytes(uint64_t rows, uint64_t cols) {
  if (rows == 0 || cols == 0) return 0;
  uint32_t pieces, threads;
  const RowShape s = back_shape(rows, cols, pieces, threads);
  return s.rounds > 1 ? 0 : (size_t)back_blocks(s, threads) * slots_of(s, threads) * cols * 4;
}

ec_status ec_rms_norm_backward(const void* dy, const void* h, const void* dh, int type,
                               uint64_t rows, uint64_t cols, const float* rstd, const void* weight,
                               int wtype, void* dx, void* dweight, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const ec_status st = check(type, wtype, rows, cols);
  if (st != EC_OK) return st;
  const size_t b = type_bytes(type), wb = type_bytes(wtype);
  if (!fine(dweight, wb)) return EC_ERR_INVALID;
  if (rows && (!fine(dy, b) || !fine(h, b) || !aligned(dh, b) || !fine(rstd, 4) ||
               !fine(weight, wb) || !fine(dx, b)))
    return EC_ERR_INVALID;
  const size_t need = ec_rms_norm_backward_workspace_bytes(rows, cols);
  if (need && !fine(workspace, 16)) return EC_ERR_INVALID;
  if (workspace_bytes < need) return EC_ERR_CAPACITY;
  const Back p{dy, h, dh, weight, rstd, wtype, dx, nullptr};
  hipStream_t s = (hipStream_t)stream;
  switch (type) {
    case EC_TYPE_F32: return back_as<float>(p, rows, cols, dweight, workspace, s);
    case EC_TYPE_F16: return back_as<f16_t>(p, rows, cols, dweight, workspace, s);
    default: return back_as<bf16_t>(p, rows, cols, dweight, workspace, s);
  }
}

}  // extern "C"
