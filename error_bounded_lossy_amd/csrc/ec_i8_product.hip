// Products of operands in the 8-bit integer form (include/ec_i8.h) on the
// matrix cores' integer instructions: y = (a b^T) times the rows' and the
// columns' scales, both operands stored along the contraction.
#include <type_traits>

#include "ec_i8.h"
#include "ec_tile_device.h"

using namespace ecmx;

namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));

enum { kDense = 0, kExperts = 1 };

struct Operand {
  const uint8_t* codes;
  const float* scales;
};

struct Product {
  Operand a, b;
  void* y;
  const int32_t* offsets;
  uint64_t rows;   // of y (kExperts: of all groups)
  uint32_t cols;   // of y
  uint32_t depth;  // codes of a stored row
  uint32_t experts;
  uint32_t m_tiles, n_tiles;
};

// ---------------------------------------------------------------- tiles

// One workgroup of 2 by 2 waves computes a tile of 64 FM rows by 64 FN columns,
// a wave 32 FM by 32 FN of it with 32x32x32 instructions.  With FM = FN = 4 a
// wave's sums fill half of its 512 registers, and an operand byte read from LDS
// is used 128 times.
//
// A stage is 64 codes of every row of both operands, brought to LDS without
// passing registers.  Four stages are in LDS: one is multiplied while the loads
// of the next three fly, with one barrier a stage, placed before the last
// multiplications so that they cover the first reads of the next stage.
//
// The order within the contraction is free as long as both operands agree, so
// lane group g of instruction step s takes the 16-byte chunk 2 g + s of a row.
// Chunks are stored at their number xor bits 1 and 2 of the row, so that 8 lanes
// of consecutive rows read 8 different 16-byte columns of 128.
template <int BM, int BN>
struct Stage {
  uint8_t a[BM * 64];
  uint8_t b[BN * 64];
};

template <int FM, int FN>
struct Fragments {
  i32x4 a[FM], b[FN];
};

// Where this lane reads in a stage: step 0's chunk of its first rows.
struct Lane {
  uint32_t a, b;
};

template <int BM, int BN, int FM, int FN>
__device__ __forceinline__ void read(const Stage<BM, BN>& st, const Lane& at, int step,
                                     Fragments<FM, FN>& f) {
  // chunk 2 g + 1 lies at the place of chunk 2 g with the lowest bit turned
#pragma unroll
  for (int i = 0; i < FN; i++)
    f.b[i] = *reinterpret_cast<const i32x4*>(st.b + (at.b ^ (step << 4)) + i * 2048);
#pragma unroll
  for (int i = 0; i < FM; i++)
    f.a[i] = *reinterpret_cast<const i32x4*>(st.a + (at.a ^ (step << 4)) + i * 2048);
}

// `between(i)` issues what goes between the rows of multiplications; nothing
// else is moved there.
template <int FM, int FN, typename F>
__device__ __forceinline__ void multiply(const Fragments<FM, FN>& f, i32x16 (&acc)[FM][FN],
                                         F&& between) {
#pragma unroll
  for (int i = 0; i < FM; i++) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < FN; j++)
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    between(i);
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <int FM, int FN, typename T, int MODE, bool PAST>
__global__ __launch_bounds__(256, FM * FN > 8 ? 1 : 2) void i8_tiles(const Product p) {
  constexpr int BM = 64 * FM, BN = 64 * FN, kWaves = 4;
  using St = Stage<BM, BN>;
  constexpr uint32_t kShift = FM == 1 ? 6 : FM == 2 ? 7 : 8;
  static_assert((1u << kShift) == BM, "tile rows");
  // four variables, not an array: the compiler then knows which loads a read waits for
  __shared__ __attribute__((aligned(16))) St st0, st1, st2, st3;
  __shared__ __attribute__((aligned(16))) float scales[BM + BN];  // of a's rows, then of b's
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t wm = wave & 1, wn = wave >> 1;

  // the tiles that groups have, not the most they could have: each XCD gets its share
  uint32_t m_tiles = p.m_tiles;
  if (MODE == kExperts) m_tiles = min(m_tiles, used_tiles(p.offsets, p.experts, p.rows, kShift));
  uint32_t t, set = 0;
  if (!dealt(m_tiles * p.n_tiles, 1, t, set)) return;
  // in an XCD's run, 8 tiles along the rows share a column tile
  const uint32_t width = 8 * p.n_tiles, band = t / width;
  const uint32_t high = min(m_tiles - band * 8, 8u);
  const uint32_t tm = band * 8 + (t - band * width) % high;
  const uint32_t tn = (t - band * width) / high;

  // this tile's rows [m0, m_end) of a and y, and its columns
  uint64_t m0 = (uint64_t)tm * BM, m_end = p.rows;
  const uint32_t n0 = tn * BN;
  T* y = (T*)p.y;
  const uint8_t* bc = p.b.codes;
  const float* bs = p.b.scales;
  if (MODE == kExperts) {
    const GroupTile gt = find_tile(p.offsets, p.experts, p.rows, kShift, tm);
    if (gt.group == p.experts) {  // rows of no group: zeros
      int64_t first = p.offsets[p.experts];
      first = first < 0 ? 0 : first;
      m0 = (uint64_t)first + (uint64_t)gt.local * BM;
      const uint64_t end = min(m0 + BM, p.rows);
      for (uint64_t r = m0 + wave; r < end; r += kWaves)
        for (uint32_t c = n0 + lane; c < min(n0 + (uint32_t)BN, p.cols); c += 64)
          y[r * p.cols + c] = (T)0.0f;
      return;
    }
    m0 = gt.first + (uint64_t)gt.local * BM;
    m_end = gt.first + gt.count;
    if (m0 >= m_end) return;  // only with offsets out of order
    bc += (uint64_t)gt.group * p.cols * p.depth;
    bs += (uint64_t)gt.group * p.cols;
  }

  // What this lane loads: of instruction q of an operand, row 16 q + lane / 4
  // and chunk (lane & 3) xor bits 1 and 2 of the row.  Rows past the end read
  // the last one: they only reach results that are not stored.
  const uint32_t pitch = p.depth;
  const uint32_t m_last = (uint32_t)(m_end - m0) - 1, n_last = p.cols - n0 - 1;
  const uint32_t chunk = (lane & 3) ^ ((lane >> 3) & 3);
  // offsets from the tile's first row: at most 256 rows of 2^17 bytes
  constexpr int LA = BM / 16 / kWaves, LB = BN / 16 / kWaves;  // a wave's loads of a stage
  uint32_t oa[LA], ob[LB];
#pragma unroll
  for (int i = 0; i < LA; i++)
    oa[i] = min((wave * LA + i) * 16 + (lane >> 2), m_last) * pitch + chunk * 16;
#pragma unroll
  for (int i = 0; i < LB; i++)
    ob[i] = min((wave * LB + i) * 16 + (lane >> 2), n_last) * pitch + chunk * 16;
  constexpr int kLoads = LA + LB;
  const uint32_t stages = __builtin_amdgcn_readfirstlane(p.depth / 64), fours = stages / 4;
  // Past the last stage it is loaded again, so that every turn below does the
  // same and waits for the same number of loads.  Part i of FM.
  const __amdgpu_buffer_rsrc_t ra = buffer_at(p.a.codes + m0 * pitch);
  const __amdgpu_buffer_rsrc_t rb = buffer_at(bc + (uint64_t)n0 * pitch);
  auto load = [&](St& st, uint32_t stage, int part) {
    const uint32_t c = __builtin_amdgcn_readfirstlane(min(stage, stages - 1)) * 64;
#pragma unroll
    for (int i = part * LA / FM; i < (part + 1) * LA / FM; i++)
      to_lds16(ra, oa[i], c, st.a + (wave * LA + i) * 1024);
#pragma unroll
    for (int i = part * LB / FM; i < (part + 1) * LB / FM; i++)
      to_lds16(rb, ob[i], c, st.b + (wave * LB + i) * 1024);
  };
  auto load_all = [&](St& st, uint32_t stage) {
#pragma unroll
    for (int i = 0; i < FM; i++) load(st, stage, i);
  };

  const uint32_t r = lane & 31, g = lane >> 5;
  Lane at;
  at.a = (wm * 32 * FM + r) * 64 + ((2 * g) ^ ((r >> 1) & 3)) * 16;
  at.b = (wn * 32 * FN + r) * 64 + ((2 * g) ^ ((r >> 1) & 3)) * 16;

  for (uint32_t i = threadIdx.x; i < BM + BN; i += 256)
    scales[i] = i < BM ? p.a.scales[m0 + min(i, m_last)] : bs[n0 + min(i - BM, n_last)];

  i32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) acc[i][j] = i32x16{};

  load_all(st0, 0);
  load_all(st1, 1);
  load_all(st2, 2);
  wait_and_meet<2 * kLoads>();
  Fragments<FM, FN> f0, f1;
  read(st0, at, 0, f0);
  // Stage s is in `now`, its first fragments are in registers.  The last stages
  // (`more` false) load nothing.
  auto turn = [&](uint32_t s, auto more, const St& now, const St& next, St& free) {
    read(now, at, 1, f1);
    multiply<FM, FN>(f0, acc, [&](int i) {
      if (more) load(free, s + 3, i);
    });
    if (more) wait_and_meet<2 * kLoads>();
    else wait_and_meet<0>();
    read(next, at, 0, f0);
    multiply<FM, FN>(f1, acc, [](int) {});
  };
  constexpr std::true_type more;
  constexpr std::false_type last;
  for (uint32_t u = 0; u < fours; u++) {
    turn(4 * u, more, st0, st1, st3);
    turn(4 * u + 1, more, st1, st2, st0);
    turn(4 * u + 2, more, st2, st3, st1);
    turn(4 * u + 3, more, st3, st0, st2);
  }
  if (stages & 2) {  // stages are pairs: rows are padded to 128 codes
    turn(4 * fours, last, st0, st1, st3);
    turn(4 * fours + 1, last, st1, st2, st0);
  }
  wait_and_meet<0>();  // the stages' memory is used again below

  // A lane has row lane & 31 of y and 4 consecutive columns in each quarter
  // of a result: 32 rows at a time go through LDS (this wave's own part) and
  // leave as whole 16-byte pieces.  Sums become floats, are scaled and rounded
  // once, here.
  constexpr uint32_t kRow = 32 * FN * sizeof(T), kPitch = kRow + 16;
  static_assert(32 * kPitch <= sizeof(St), "the stage holds the results");
  uint8_t* out = reinterpret_cast<uint8_t*>(wave == 0   ? &st0
                                             : wave == 1 ? &st1
                                             : wave == 2 ? &st2
                                                         : &st3);
  const uint32_t nw = n0 + wn * 32 * FN;
#pragma unroll
  for (int i = 0; i < FM; i++) {
    const float sa = scales[wm * 32 * FM + i * 32 + r];
#pragma unroll
    for (int j = 0; j < FN; j++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const uint32_t col = j * 32 + q * 8 + g * 4;
        float sb[4];
        __builtin_memcpy(sb, __builtin_assume_aligned(scales + BM + wn * 32 * FN + col, 16), 16);
        T v[4];
#pragma unroll
        for (int u = 0; u < 4; u++) v[u] = (T)in_fp32<T>((float)acc[i][j][4 * q + u] * sa * sb[u]);
        __builtin_memcpy(out + r * kPitch + col * sizeof(T), v, sizeof(v));
      }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr uint32_t kLanes = kRow / 16, kTogether = 64 / kLanes, kE = 16 / sizeof(T);
#pragma unroll
    for (uint32_t q = 0; q < 32 / kTogether; q++) {
      const uint32_t row = q * kTogether + lane / kLanes, col = (lane % kLanes) * kE;
      const uint64_t m = m0 + wm * 32 * FM + i * 32 + row;
      T v[kE];
      __builtin_memcpy(v, __builtin_assume_aligned(out + row * kPitch + col * sizeof(T), 16), 16);
      if (m < m_end) {
        T* to = y + m * p.cols + nw + col;
        if (nw + col + kE <= p.cols) {
          store16<PAST>(to, v);
        } else {
#pragma unroll
          for (uint32_t u = 0; u < kE; u++)
            if (nw + col + u < p.cols) to[u] = v[u];
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------------- few rows

// Up to 16 rows (of a group) against 16 columns a workgroup: what counts is
// reading b once, at full bandwidth.  The waves divide the contraction in pieces
// of 256 codes; a lane loads 16 bytes of a row of b and an instruction's 4 lanes
// of a row 64 bytes, straight into registers, two pieces ahead.
constexpr uint32_t kFewCols = 16, kFewRows = 16, kFewWaves = 8, kPiece = 256;
constexpr int kSteps = kPiece / 64, kSets = 2;

template <typename T>
__global__ __launch_bounds__(64 * kFewWaves, 4) void i8_few(const Product p) {
  __shared__ __attribute__((aligned(16))) int part[kFewWaves][256];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t waves = blockDim.x >> 6;
  const uint32_t r = lane & 15, g = lane >> 4;
  const uint32_t block = block_number(), tn = block % p.n_tiles;
  const uint32_t n0 = tn * kFewCols;
  uint64_t row0 = 0;
  uint32_t here = (uint32_t)p.rows;
  T* y = (T*)p.y;
  const uint8_t* bc = p.b.codes;
  const float* bs = p.b.scales;
  if (p.experts) {
    const GroupTile gt = find_tile(p.offsets, p.experts, p.rows, 4, block / p.n_tiles);
    const uint64_t skip = (uint64_t)gt.local * kFewRows;
    if (gt.group == p.experts) {  // rows of no group: zeros
      const int64_t f = p.offsets[p.experts];
      const uint64_t m0 = (f < 0 ? 0 : f) + skip, end = min(m0 + kFewRows, p.rows);
      const uint32_t col = n0 + threadIdx.x % kFewCols;
      if (col < p.cols)
        for (uint64_t m = m0 + threadIdx.x / kFewCols; m < end; m += blockDim.x / kFewCols)
          y[m * p.cols + col] = (T)0.0f;
      return;
    }
    if (skip >= gt.count) return;  // only with offsets out of order
    row0 = gt.first + skip;
    here = (uint32_t)min((uint64_t)kFewRows, gt.count - skip);
    bc += (uint64_t)gt.group * p.cols * p.depth;
    bs += (uint64_t)gt.group * p.cols;
  } else if (block >= p.n_tiles) {
    return;
  }
  const uint32_t steps = p.depth / 64, pieces = (steps + kSteps - 1) / kSteps;
  const uint8_t* gb = bc + (uint64_t)min(n0 + r, p.cols - 1) * p.depth + g * 16;
  const uint8_t* ga = p.a.codes + (row0 + min(r, here - 1)) * p.depth + g * 16;
  struct Piece {
    i32x4 b[kSteps];
  };
  auto load = [&](Piece& f, uint32_t at) {
#pragma unroll
    for (int s = 0; s < kSteps; s++)  // steps past the end read the last one
      f.b[s] = *reinterpret_cast<const i32x4*>(gb + min(at * kSteps + s, steps - 1) * 64);
  };
  Piece f[kSets];
#pragma unroll
  for (int i = 0; i < kSets; i++)
    if (wave + i * waves < pieces) load(f[i], wave + i * waves);
  i32x4 acc = {};
  for (uint32_t piece = wave; piece < pieces; piece += kSets * waves) {
#pragma unroll
    for (int i = 0; i < kSets; i++) {
      const uint32_t now = piece + i * waves;
      if (now >= pieces) break;
#pragma unroll
      for (int s = 0; s < kSteps; s++) {
        const uint32_t step = now * kSteps + s;
        if (step < steps) {
          const i32x4 fa = *reinterpret_cast<const i32x4*>(ga + step * 64);
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(f[i].b[s], fa, acc, 0, 0, 0);
        }
      }
      if (now + kSets * waves < pieces) load(f[i], now + kSets * waves);
    }
  }
  // a lane has row r of y and columns 4 g .. 4 g + 3
  *reinterpret_cast<i32x4*>(&part[wave][r * 16 + g * 4]) = acc;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < here * 16; i += blockDim.x) {
    int sum = 0;
    for (uint32_t w = 0; w < waves; w++) sum += part[w][i];
    const uint32_t col = n0 + i % 16;
    const uint64_t row = row0 + i / 16;
    if (col < p.cols) y[row * p.cols + col] = (T)in_fp32<T>((float)sum * p.a.scales[row] * bs[col]);
  }
}

// ---------------------------------------------------------------- host

ec_status launched() { return hipGetLastError() == hipSuccess ? EC_OK : EC_ERR_DEVICE; }

template <int FM, int FN, typename T, int MODE>
ec_status tiles_as(Product p, hipStream_t s) {
  p.n_tiles = (uint32_t)ceil_div(p.cols, 64 * FN);
  uint64_t m = ceil_div(p.rows, 64 * FM);
  // groups round up each, and the rows of no group once more
  if (MODE == kExperts) m += (p.experts < p.rows ? p.experts : p.rows) + 1;
  const uint64_t tiles = ceil_div(m * p.n_tiles, 8) * 8;
  if (tiles > kMostBlocks) return EC_ERR_UNSUPPORTED;
  p.m_tiles = (uint32_t)m;
  const uint64_t row = p.cols * sizeof(T), bytes = p.rows * row;
  if (FM > 1 && past_caches(bytes, row)) {
    hipLaunchKernelGGL((i8_tiles<FM, FN, T, MODE, true>), grid_of(tiles), dim3(256), 0, s, p);
    return launched();
  }
  hipLaunchKernelGGL((i8_tiles<FM, FN, T, MODE, false>), grid_of(tiles), dim3(256), 0, s, p);
  return launched();
}

// Rows and columns of a tile.
uint32_t side_of(int mode, uint64_t rows, uint64_t cols, uint64_t groups) {
  const uint64_t extra = mode == kExperts ? groups / 2 : 0;  // half a tile more for each
  const uint64_t large = (ceil_div(rows, 256) + extra) * ceil_div(cols, 256);
  const uint64_t small = (ceil_div(rows, 128) + extra) * ceil_div(cols, 128);
  return large >= 192 ? 256 : small >= 128 ? 128 : 64;
}

// Whether the kernel for few rows runs.
bool few_rows(uint64_t rows, uint64_t experts) {
  return (experts ? ceil_div(rows, experts) : rows) <= kFewRows;
}

template <typename T>
ec_status product_as(Product p, hipStream_t s) {
  if (few_rows(p.rows, p.experts)) {
    p.n_tiles = (uint32_t)ceil_div(p.cols, kFewCols);
    // groups round up each, and the rows of no group once more
    const uint64_t m = p.experts ? ceil_div(p.rows, kFewRows) +
                                       (p.experts < p.rows ? p.experts : p.rows) + 1
                                 : 1;
    const uint64_t blocks = p.n_tiles * m;
    if (blocks > kMostBlocks) return EC_ERR_UNSUPPORTED;
    const uint32_t pieces = (p.depth + kPiece - 1) / kPiece;
    const uint32_t waves = pieces < kFewWaves ? pieces : kFewWaves;
    hipLaunchKernelGGL((i8_few<T>), grid_of(blocks), dim3(64 * waves), 0, s, p);
    return launched();
  }
  const uint32_t side = side_of(p.experts ? kExperts : kDense, p.rows, p.cols, p.experts);
  if (p.experts) {
    if (side == 256) return tiles_as<4, 4, T, kExperts>(p, s);
    if (side == 128) return tiles_as<2, 2, T, kExperts>(p, s);
    return tiles_as<1, 1, T, kExperts>(p, s);
  }
  if (side == 256) return tiles_as<4, 4, T, kDense>(p, s);
  if (side == 128) return tiles_as<2, 2, T, kDense>(p, s);
  return tiles_as<1, 1, T, kDense>(p, s);
}

ec_status product(const Product& p, int type, hipStream_t s) {
  switch (type) {
    case EC_TYPE_F32: return product_as<float>(p, s);
    case EC_TYPE_F16: return product_as<f16_t>(p, s);
    default: return product_as<bf16_t>(p, s);
  }
}

ec_status check(const void* a, const void* sa, uint64_t rows, const void* b, const void* sb,
                uint64_t cols, uint64_t depth, const void* y, int type) {
  if (!type_known(type) || cols == 0 || depth == 0 || depth % 128 != 0) return EC_ERR_INVALID;
  if (rows > EC_MX_MAX_ROWS || cols > EC_MX_MAX_ROWS || depth > EC_I8_MAX_DEPTH)
    return EC_ERR_UNSUPPORTED;
  if (rows == 0) return EC_OK;
  if (!y || !aligned(y, type_bytes(type)) || !read_ok(b, sb) || !read_ok(a, sa))
    return EC_ERR_INVALID;
  return EC_OK;
}

ec_status check_groups(const int32_t* offsets, uint32_t groups) {
  if (!offsets || !aligned(offsets, 4) || groups == 0) return EC_ERR_INVALID;
  return groups > EC_MX_MAX_GROUPS ? EC_ERR_UNSUPPORTED : EC_OK;
}

Product product_of(const void* a_codes, const void* a_scales, uint64_t rows, const void* b_codes,
                   const void* b_scales, uint64_t cols, uint64_t depth, const int32_t* offsets,
                   uint32_t experts, void* y) {
  Product p{};
  p.a = {(const uint8_t*)a_codes, (const float*)a_scales};
  p.b = {(const uint8_t*)b_codes, (const float*)b_scales};
  p.y = y, p.rows = rows, p.cols = (uint32_t)cols, p.depth = (uint32_t)depth;
  p.offsets = offsets, p.experts = experts;
  return p;
}

// Codes of the workspace of a linear layer; the scales are behind them.
uint64_t code_bytes(uint64_t rows, uint64_t depth) { return rows * ec_mx_padded(depth); }

}  // namespace

extern "C" {

ec_status ec_i8_product(const void* a_codes, const void* a_scales, uint64_t rows,
                        const void* b_codes, const void* b_scales, uint64_t cols, uint64_t depth,
                        void* y, int type, void* stream) {
  const ec_status st = check(a_codes, a_scales, rows, b_codes, b_scales, cols, depth, y, type);
  if (st != EC_OK || rows == 0) return st;
  return product(product_of(a_codes, a_scales, rows, b_codes, b_scales, cols, depth, nullptr, 0, y),
                 type, (hipStream_t)stream);
}

ec_status ec_i8_product_experts(const void* a_codes, const void* a_scales, uint64_t rows,
                                const void* b_codes, const void* b_scales, uint64_t cols,
                                uint64_t depth, const int32_t* offsets, uint32_t experts, void* y,
                                int type, void* stream) {
  ec_status st = check_groups(offsets, experts);
  if (st == EC_OK) st = check(a_codes, a_scales, rows, b_codes, b_scales, cols, depth, y, type);
  if (st != EC_OK || rows == 0) return st;
  return product(product_of(a_codes, a_scales, rows, b_codes, b_scales, cols, depth, offsets,
                            experts, y),
                 type, (hipStream_t)stream);
}

uint32_t ec_i8_product_tile(uint64_t rows, uint64_t cols, uint64_t depth, int type,
                            uint32_t experts) {
  if (!type_known(type) || rows == 0 || cols == 0 || depth == 0) return 0;
  if (few_rows(rows, experts)) return kFewRows;
  return side_of(experts ? kExperts : kDense, rows, cols, experts);
}

size_t ec_i8_linear_workspace_bytes(uint64_t rows, uint64_t depth, uint64_t cols,
                                    uint32_t experts) {
  (void)cols;
  (void)experts;
  return code_bytes(rows, depth) + rows * 4;
}

ec_status ec_i8_linear(const void* x, int type, uint64_t rows, uint64_t depth, uint64_t stride,
                       const void* w_codes, const void* w_scales, uint64_t cols,
                       const int32_t* offsets, uint32_t experts, void* y, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!type_known(type) || depth == 0 || cols == 0 || stride < depth || (!offsets) != (!experts))
    return EC_ERR_INVALID;
  if (experts > EC_MX_MAX_GROUPS || rows > EC_MX_MAX_ROWS || cols > EC_MX_MAX_ROWS ||
      depth > EC_I8_MAX_DEPTH)
    return EC_ERR_UNSUPPORTED;
  if (rows == 0) return EC_OK;
  if (!x || !aligned(x, type_bytes(type)) || !y || !aligned(y, type_bytes(type)) ||
      !read_ok(w_codes, w_scales) || !aligned(offsets, 4) || !aligned(workspace, 16))
    return EC_ERR_INVALID;
  const size_t need = ec_i8_linear_workspace_bytes(rows, depth, cols, experts);
  if (need && !workspace) return EC_ERR_INVALID;
  if (workspace_bytes < need) return EC_ERR_CAPACITY;
  uint8_t* codes = (uint8_t*)workspace;
  void* scales = codes + code_bytes(rows, depth);
  const ec_status st = ec_i8_quantize(x, type, rows, depth, stride, codes, scales, stream);
  if (st != EC_OK) return st;
  return product(product_of(codes, scales, rows, w_codes, w_scales, cols, ec_mx_padded(depth),
                            offsets, experts, y),
                 type, (hipStream_t)stream);
}

}  // extern "C"
