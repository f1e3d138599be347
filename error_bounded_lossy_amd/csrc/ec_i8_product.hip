// Products of operands in the 8-bit integer form (include/ec_i8.h) on the
// matrix cores' integer instructions: y = (a b^T) times the rows' and the
// columns' scales, both operands stored along the contraction.
#include <type_traits>

#include "ec_i8.h"
#include "ec_row_device.h"
#include "ec_tile_device.h"

using namespace ecmx;

namespace {

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
  uint32_t parts;  // of the contraction, of T = int32_t
};

// ---------------------------------------------------------------- tiles

// One workgroup of 2 by 2 waves computes a tile of 64 FM rows by 64 FN columns,
// a wave 32 FM by 32 FN of it with 16x16x64 instructions, which on random codes
// reach 4.0 POP/s where those of 32x32x32 reach 3.3 (the clock falls with the
// power; 4.9 and 4.6 on zeros).  With FM = FN = 4 a wave's sums fill half of its
// 512 registers, and an operand byte read from LDS is used 128 times.
//
// A stage is 128 codes of every row of both operands, a line of the caches, so
// that a line is asked for once.  It is brought to LDS without passing registers,
// while the stage before is multiplied (of small tiles, the three before), with
// one barrier a stage, placed between its two steps so that the second covers the
// first reads of the next stage.
//
// The order within the contraction is free as long as both operands agree, so
// lane group g of step s takes the 16-byte chunk 4 s + g of a row.
// Chunks are stored at their number xor the row's lowest three bits, so that 8
// lanes of consecutive rows read 8 different 16-byte columns of 128.
template <int BM, int BN>
struct Stage {
  uint8_t a[BM * 128];
  uint8_t b[BN * 128];
};

// Where this lane reads in a stage: step 0's chunk of its first rows.
struct Lane {
  uint32_t a, b;
};

// Fragment i of a step.
template <typename St>
__device__ __forceinline__ i32x4 read_a(const St& st, const Lane& at, int step, int i) {
  return *reinterpret_cast<const i32x4*>(st.a + (at.a ^ (step << 6)) + i * 2048);
}
template <int N, typename St>
__device__ __forceinline__ void read_b(const St& st, const Lane& at, int step, i32x4 (&b)[N]) {
#pragma unroll
  for (int i = 0; i < N; i++)
    b[i] = *reinterpret_cast<const i32x4*>(st.b + (at.b ^ (step << 6)) + i * 2048);
}

// `between(i)` issues what goes behind row i of the multiplications, when a[i] is
// free; nothing else is moved there.
//
// The sums of the largest tile (64 results) are held in the accumulation registers
// by the instruction's own operands: from the builtin, the compiler moves most of
// them to other registers and back in every round of the loop (8192^3 625 us).
// What it does not see are the waits between the instruction and what uses its
// result: none are due among multiplications, 64 of which are between two of one
// result; the barrier is between the zeros and the first of them, and finished()
// waits before the results are read.  So the loop has to stay one piece of code whose
// sums leave these registers nowhere: its functions are always inlined, and a test
// looks at the compiled code.
__device__ __forceinline__ void multiply_held(i32x4& acc, const i32x4& b, const i32x4& a) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}
template <int M, int N>
__device__ __forceinline__ void hold(i32x4 (&acc)[M][N]) {  // keeps its place among such statements
#pragma unroll
  for (int i = 0; i < M; i++)
#pragma unroll
    for (int j = 0; j < N; j++) asm volatile("" : "+a"(acc[i][j]));
}
template <int M, int N>
__device__ __forceinline__ void finished(i32x4 (&acc)[M][N]) {
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  hold(acc);
}

template <int M, int N, typename F>
__device__ __forceinline__ void multiply(const i32x4 (&a)[M], const i32x4 (&b)[N],
                                         i32x4 (&acc)[M][N], F&& between) {
#pragma unroll
  for (int i = 0; i < M; i++) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < N; j++) {
      if constexpr (M * N == 64) multiply_held(acc[i][j], b[j], a[i]);
      else acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[j], a[i], acc[i][j], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    between(i);
  }
  __builtin_amdgcn_sched_barrier(0);
}

__host__ __device__ uint32_t part_pitch(uint32_t cols) { return (cols + 63) / 64 * 64; }

// With T = int32_t, a workgroup takes one of p.parts parts of the contraction, and y
// [parts][rows][part_pitch(cols)] holds the parts' sums, which i8_join adds: the same
// whole numbers in any order.
//
// STAGES: 2 of the largest tile (of one line each they fill LDS) and where two
// workgroups share a unit; 4 where there is a unit for each (512 x 8192 x 8192 as tiles
// of 128 41 us, with 2 stages 45; 2048 x 4096 x 4096 45 and 36), or the tile is small (8
// stages of tiles of 64, 17 x 1000 x 300: 4.2 us, 4: 3.7; 64 x 16384 x 4096 39.1 and
// 39.9).
template <int FM, int FN, int STAGES, typename T, int MODE, bool PAST>
__global__ __launch_bounds__(256, STAGES * FM * FN >= 16 ? 1 : 2) void i8_tiles(const Product p) {
  constexpr int BM = 64 * FM, BN = 64 * FN, kWaves = 4;
  using St = Stage<BM, BN>;
  constexpr uint32_t kShift = FM == 1 ? 6 : FM == 2 ? 7 : 8;
  static_assert((1u << kShift) == BM, "tile rows");
  // (variables, not an array: the compiler then knows which loads a read waits for)
  __shared__ __attribute__((aligned(16))) St st0, st1;
  __shared__ __attribute__((aligned(16))) std::conditional_t<STAGES == 4, St, int> st2, st3;
  __shared__ __attribute__((aligned(16))) float scales[BM + BN];  // of a's rows, then of b's
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t wm = wave & 1, wn = wave >> 1;

  // the tiles that groups have, not the most they could have: each XCD gets its share
  uint32_t m_tiles = p.m_tiles;
  if (MODE == kExperts) m_tiles = min(m_tiles, used_tiles(p.offsets, p.experts, p.rows, kShift));
  constexpr bool kParts = std::is_same_v<T, int32_t>;
  uint32_t t, set = 0;
  if (!dealt(m_tiles * p.n_tiles, kParts ? p.parts : 1, t, set)) return;
  // in an XCD's run, 8 tiles along the rows share a column tile
  const uint32_t width = 8 * p.n_tiles, band = t / width;
  const uint32_t high = min(m_tiles - band * 8, 8u);
  // (as scalars: a buffer whose address is in vector registers costs a loop a load)
  const uint32_t tm = __builtin_amdgcn_readfirstlane(band * 8 + (t - band * width) % high);
  const uint32_t tn = __builtin_amdgcn_readfirstlane((t - band * width) / high);

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

  // What this lane loads: of instruction q of an operand, row 8 q + lane / 8 and
  // chunk (lane & 7) xor the row's lowest three bits.  Rows past the end read the
  // last one: they only reach results that are not stored.
  const uint32_t pitch = p.depth;
  const uint32_t m_last = (uint32_t)(m_end - m0) - 1, n_last = p.cols - n0 - 1;
  const uint32_t chunk = (lane & 7) ^ (lane >> 3);
  // offsets from the tile's first row: at most 256 rows of 2^17 bytes
  constexpr int LA = BM / 8 / kWaves, LB = BN / 8 / kWaves;  // a wave's loads of a stage
  uint32_t oa[LA], ob[LB];
#pragma unroll
  for (int i = 0; i < LA; i++)
    oa[i] = min((wave * LA + i) * 8 + (lane >> 3), m_last) * pitch + chunk * 16;
#pragma unroll
  for (int i = 0; i < LB; i++)
    ob[i] = min((wave * LB + i) * 8 + (lane >> 3), n_last) * pitch + chunk * 16;
  constexpr int kLoads = LA + LB;
  uint32_t stages = __builtin_amdgcn_readfirstlane(p.depth / 128), begin = 0;
  uint32_t y_pitch = p.cols, y_cols = p.cols;
  if constexpr (kParts) {
    const uint32_t each = (stages + p.parts - 1) / p.parts;  // the last one may have fewer
    begin = __builtin_amdgcn_readfirstlane(set * each);
    stages = min(each, stages - begin);
    y_pitch = y_cols = part_pitch(p.cols);
    y += set * p.rows * y_pitch;
  }
  // Past the last stage it is loaded again, so that every turn below does the
  // same and waits for the same number of loads.  Part i of 2 FM: two loads behind every row
  // of multiplications (8192^3: 494 us; four behind the first half of them 509, eight
  // behind the first quarter 530).
  const __amdgpu_buffer_rsrc_t ra = buffer_at(p.a.codes + m0 * pitch + begin * 128);
  const __amdgpu_buffer_rsrc_t rb = buffer_at(bc + (uint64_t)n0 * pitch + begin * 128);
  auto load = [&](St& st, uint32_t stage, int part) __attribute__((always_inline)) {
    const uint32_t c = __builtin_amdgcn_readfirstlane(min(stage, stages - 1)) * 128;
#pragma unroll
    for (int i = part * LA / (2 * FM); i < (part + 1) * LA / (2 * FM); i++)
      to_lds16(ra, oa[i], c, st.a + (wave * LA + i) * 1024);
#pragma unroll
    for (int i = part * LB / (2 * FM); i < (part + 1) * LB / (2 * FM); i++)
      to_lds16(rb, ob[i], c, st.b + (wave * LB + i) * 1024);
  };
  auto load_all = [&](St& st, uint32_t stage) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2 * FM; i++) load(st, stage, i);
  };

  const uint32_t r = lane & 15, g = lane >> 4;
  Lane at;
  at.a = (wm * 32 * FM + r) * 128 + (g ^ (r & 7)) * 16;
  at.b = (wn * 32 * FN + r) * 128 + (g ^ (r & 7)) * 16;

  if constexpr (!kParts)
    for (uint32_t i = threadIdx.x; i < BM + BN; i += 256)
      scales[i] = i < BM ? p.a.scales[m0 + min(i, m_last)] : bs[n0 + min(i - BM, n_last)];

  i32x4 acc[2 * FM][2 * FN];
#pragma unroll
  for (int i = 0; i < 2 * FM; i++)
#pragma unroll
    for (int j = 0; j < 2 * FN; j++) acc[i][j] = i32x4{};
  if constexpr (FM * FN == 16) hold(acc);  // written before the barrier below

  load_all(st0, 0);
  if constexpr (STAGES == 4) {
    load_all(st1, 1);
    load_all(st2, 2);
    wait_and_meet<2 * kLoads>();
  } else {
    wait_and_meet<0>();
    load_all(st1, 1);
  }
  // A step's fragments of b are read a step ahead, those of a as the multiplications
  // free them: both twice would not fit the registers beside the sums.
  i32x4 fa[2 * FM], b0[2 * FN], b1[2 * FN];
  read_b(st0, at, 0, b0);
#pragma unroll
  for (int i = 0; i < 2 * FM; i++) fa[i] = read_a(st0, at, 0, i);
  // Stage s is in `now`, its first fragments are in registers.  With two stages,
  // the loads of stage s + 2 begin behind the barrier, into `now`, which all waves
  // have read; with four, those of stage s + 3 go into the stage before.
  auto turn = [&](uint32_t s, St& now, St& next, St& free) __attribute__((always_inline)) {
    read_b(now, at, 1, b1);
    multiply(fa, b0, acc, [&](int i) {
      fa[i] = read_a(now, at, 1, i);
      if (STAGES == 4) load(free, s + 3, i);
    });
    wait_and_meet<STAGES == 4 ? 2 * kLoads : 0>();
    read_b(next, at, 0, b0);
    multiply(fa, b1, acc, [&](int i) {
      fa[i] = read_a(next, at, 0, i);
      if (STAGES == 2) load(now, s + 2, i);
    });
  };
  uint32_t s = 0;
  if constexpr (STAGES == 4) {
    for (; s + 4 <= stages; s += 4) {
      turn(s, st0, st1, st3);
      turn(s + 1, st1, st2, st0);
      turn(s + 2, st2, st3, st1);
      turn(s + 3, st3, st0, st2);
    }
    if (s < stages) turn(s, st0, st1, st3);
    if (s + 1 < stages) turn(s + 1, st1, st2, st0);
    if (s + 2 < stages) turn(s + 2, st2, st3, st1);
  } else {
    for (; s + 2 <= stages; s += 2) {
      turn(s, st0, st1, st1);
      turn(s + 1, st1, st0, st0);
    }
    if (s < stages) turn(s, st0, st1, st1);
  }
  wait_and_meet<0>();  // the stages' memory is used again below
  if constexpr (FM * FN == 16) finished(acc);

  // A lane has row lane & 15 of y and 4 consecutive columns of a result: 32 rows at
  // a time go through LDS (this wave's own part) and leave as whole 16-byte pieces.
  // Sums become floats, are scaled and rounded once, here.
  constexpr uint32_t kRow = 32 * FN * sizeof(T), kPitch = kRow + 16;
  static_assert(2 * 32 * kPitch <= sizeof(St), "a stage holds the results of two waves");
  uint8_t* out = reinterpret_cast<uint8_t*>(wave & 1 ? &st1 : &st0) + (wave >> 1) * 32 * kPitch;
  const uint32_t nw = n0 + wn * 32 * FN;
#pragma unroll
  for (int i = 0; i < FM; i++) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const float sa = scales[wm * 32 * FM + i * 32 + h * 16 + r];
#pragma unroll
      for (int j = 0; j < 2 * FN; j++) {
        const uint32_t col = j * 16 + g * 4;
        float sb[4];
        __builtin_memcpy(sb, __builtin_assume_aligned(scales + BM + wn * 32 * FN + col, 16), 16);
        T v[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
          if constexpr (kParts) v[u] = acc[2 * i + h][j][u];
          else v[u] = (T)in_fp32<T>((float)acc[2 * i + h][j][u] * sa * sb[u]);
        }
        __builtin_memcpy(out + (h * 16 + r) * kPitch + col * sizeof(T), v, sizeof(v));
      }
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
        T* to = y + m * y_pitch + nw + col;
        if (nw + col + kE <= y_cols) {
          store16<PAST>(to, v);
        } else {
#pragma unroll
          for (uint32_t u = 0; u < kE; u++)
            if (nw + col + u < y_cols) to[u] = v[u];
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// What the parts of a contraction sum to, scaled and rounded as a tile's results are;
// a thread takes four columns of a row.
template <typename T>
__global__ __launch_bounds__(256) void i8_join(const Product p, T* y) {
  const uint32_t pitch = part_pitch(p.cols), quads = pitch / 4;
  const uint64_t i = (uint64_t)block_number() * 256 + threadIdx.x;
  if (i >= p.rows * quads) return;
  const uint64_t row = i / quads;
  const uint32_t col = (uint32_t)(i - row * quads) * 4;
  const i32x4* from = (const i32x4*)p.y + i;
  i32x4 sum = {};
#pragma unroll 4
  for (uint32_t s = 0; s < p.parts; s++) sum += from[s * p.rows * quads];
  const float sa = p.a.scales[row];
#pragma unroll
  for (int u = 0; u < 4; u++)
    if (col + u < p.cols)
      y[row * p.cols + col + u] = (T)in_fp32<T>((float)sum[u] * sa * p.b.scales[col + u]);
}

// ---------------------------------------------------------------- few rows

// Up to 16 rows against 16 columns a workgroup: what counts is reading b once, at
// full bandwidth.  The waves divide the contraction in pieces of 256 codes; a lane
// loads 16 bytes of a row of b and an instruction's 4 lanes of a row 64 bytes,
// straight into registers, SETS pieces ahead: 4 where a wave has as many (1 x 8192 x
// 8192: 15.8 us with 4, 17.1 with 2; 1 x 4096 x 4096: 6.6 and 6.4).
//
// With x unquantized (CHUNKS > 0), the workgroup quantizes its rows into LDS first,
// while its first loads of b are in flight.
//
// (Rows of experts all go to the tiles, whose loads go past the registers: 128 rows
// of 32 experts of 1024 x 2048 16.2 us there and 17.7 here, 512 rows 18.6 and 27.9.)
constexpr uint32_t kFewCols = 16, kFewRows = 16, kFewWaves = 8, kPiece = 256;
constexpr int kSteps = kPiece / 64;
// Elements that the workgroup quantizes: CHUNKS pieces of 8 a thread, 2 or 4, with
// SETS = 2 where it is 4 (both do not fit 128 registers).
constexpr uint32_t kFewElements = 4 * 8 * 64 * kFewWaves;

struct Few {
  Product p;
  const void* x;
  uint64_t stride;
  uint32_t raw_depth;  // elements of a row of x
};

template <typename T, int CHUNKS, int SETS>  // CHUNKS = 0: x is in the 8-bit form
__global__ __launch_bounds__(64 * kFewWaves, 4) void i8_few(const Few few) {
  extern __shared__ __attribute__((aligned(16))) uint8_t codes[];
  __shared__ __attribute__((aligned(16))) int part[kFewWaves][256];
  __shared__ uint32_t tops[kFewRows];
  const Product& p = few.p;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t waves = blockDim.x >> 6;
  const uint32_t r = lane & 15, g = lane >> 4, rows = (uint32_t)p.rows;
  const uint32_t block = block_number(), n0 = block * kFewCols;
  if (block >= p.n_tiles) return;
  const uint32_t steps = p.depth / 64, pieces = (steps + kSteps - 1) / kSteps;
  const uint8_t* gb = p.b.codes + (uint64_t)min(n0 + r, p.cols - 1) * p.depth + g * 16;
  struct Piece {
    i32x4 b[kSteps];
  };
  auto load = [&](Piece& f, uint32_t at) {
#pragma unroll
    for (int s = 0; s < kSteps; s++)  // steps past the end read the last one
      f.b[s] = *reinterpret_cast<const i32x4*>(gb + min(at * kSteps + s, steps - 1) * 64);
  };
  Piece f[SETS];
#pragma unroll
  for (int i = 0; i < SETS; i++)
    if (wave + i * waves < pieces) load(f[i], wave + i * waves);
  const uint32_t lr = min(r, rows - 1);
  const uint8_t* ga;
  if constexpr (CHUNKS > 0) {
    const uint32_t chunks = p.depth / 8, total = rows * chunks, pitch = p.depth + 16;
    if (threadIdx.x < kFewRows) tops[threadIdx.x] = 0;
    __syncthreads();
    Eight<T> v[CHUNKS];
    uint32_t row[CHUNKS], c[CHUNKS];
#pragma unroll
    for (int q = 0; q < CHUNKS; q++) {
      const uint32_t i = threadIdx.x + q * blockDim.x;
      if (q * blockDim.x >= total) break;
      row[q] = i / chunks, c[q] = i - row[q] * chunks;
      v[q] = load_eight((const T*)few.x + row[q] * few.stride + c[q] * 8,
                        i < total ? (int64_t)few.raw_depth - c[q] * 8 : 0);
    }
#pragma unroll
    for (int q = 0; q < CHUNKS; q++) {
      if (q * blockDim.x >= total) break;
      float e[8];
      widen(v[q], e);
      // 16 lanes share a row
      uint32_t m = max_of_8_lanes(magnitude_of_floats(e));
      const uint32_t t = __builtin_amdgcn_mov_dpp(m, 0x140, 0xf, 0xf, true);
      m = m > t ? m : t;
      if (r == 0 && threadIdx.x + q * blockDim.x < total) atomicMax(&tops[row[q]], m);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < CHUNKS; q++) {
      if (threadIdx.x + q * blockDim.x >= total) break;
      float e[8];
      widen(v[q], e);
      *reinterpret_cast<uint2*>(codes + row[q] * pitch + c[q] * 8) =
          code_row_eight(e, row_scale(tops[row[q]]));
    }
    __syncthreads();
    ga = codes + lr * pitch + g * 16;
  } else {
    ga = p.a.codes + lr * p.depth + g * 16;
  }
  i32x4 acc = {};
  for (uint32_t piece = wave; piece < pieces; piece += SETS * waves) {
#pragma unroll
    for (int i = 0; i < SETS; i++) {
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
      if (now + SETS * waves < pieces) load(f[i], now + SETS * waves);
    }
  }
  // a lane has row r of y and columns 4 g .. 4 g + 3
  *reinterpret_cast<i32x4*>(&part[wave][r * 16 + g * 4]) = acc;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < rows * 16; i += blockDim.x) {
    int sum = 0;
    for (uint32_t w = 0; w < waves; w++) sum += part[w][i];
    const uint32_t col = n0 + i % 16;
    float scale;
    if constexpr (CHUNKS > 0) scale = row_scale(tops[i / 16]).scale;
    else scale = p.a.scales[i / 16];
    if (col < p.cols)
      ((T*)p.y)[(uint64_t)(i / 16) * p.cols + col] =
          (T)in_fp32<T>((float)sum * scale * p.b.scales[col]);
  }
}

// ---------------------------------------------------------------- host

ec_status launched() { return hipGetLastError() == hipSuccess ? EC_OK : EC_ERR_DEVICE; }

template <int FM, int FN, int STAGES, typename T, int MODE>
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
    hipLaunchKernelGGL((i8_tiles<FM, FN, STAGES, T, MODE, true>), grid_of(tiles), dim3(256), 0, s, p);
    return launched();
  }
  hipLaunchKernelGGL((i8_tiles<FM, FN, STAGES, T, MODE, false>), grid_of(tiles), dim3(256), 0, s, p);
  return launched();
}

// Which tile: by what a round of workgroups costs, in us times 1024: large ones
// fill the 256 units one by one, of the others two share a unit.  Measured, us, as
// tiles of 256, 128 and 64 (outputs, contraction, bf16):
//   8192 x 8192, 512: 66, 58, 95; 4096 x 4096, 2048: 39, 41, 57; 8192: 105, 119, 187;
//   2048 x 4096, 4096: 49, 33, 50; 1024 x 4096, 4096: 48, 21, 26; 500 x 4096, 4096:
//   47, 19, 14; 200 x 8192, 8192: 82, 31, 26; 100 x 4096, 4096: 45, 17, 6.8.
// Experts' weights are read anew by every group's tiles: 32768 rows, 64 experts,
// 2048 outputs, contraction 4096: 349, 377, 529; 1024: 147, 134, 204; 2048 rows, 32
// experts, 1024 outputs, 2048: 31, 27, 20.  Outputs in fp32 cost their stores: 8192 x
// 8192, 512: 93, 76, 106.
struct Tiles {
  uint64_t large, small, least;  // how many of 256, 128 and 64
  uint64_t cost[3];
};
Tiles tiles_for(int mode, uint64_t rows, uint64_t cols, uint64_t depth, uint64_t groups,
                size_t bytes) {
  const uint64_t extra = mode == kExperts ? groups / 2 : 0;  // half a tile more for each
  auto tiles = [&](uint64_t side) { return (ceil_div(rows, side) + extra) * ceil_div(cols, side); };
  const bool experts = mode == kExperts, wide = bytes == 4;
  // a round of `at_once`, a last one that is at most half full as half of one
  auto cost = [&](uint64_t n, uint64_t at_once, uint64_t start, uint64_t per8) {
    const uint64_t halves = ceil_div(2 * n, at_once);
    return (halves < 2 ? 2 : halves) * (start * 1024 + depth * per8 / 8) / 2;
  };
  Tiles t{tiles(256), tiles(128), tiles(64), {}};
  t.cost[0] = ceil_div(t.large, 256) *
              ((experts ? 16 : wide ? 18 : 12) * 1024 + depth * (experts ? 108 : 86) / 8);
  t.cost[1] = t.small <= 256 ? cost(t.small, 256, experts ? 7 : 5, experts ? 48 : 32)
                             : cost(t.small, 512, experts ? 6 : wide ? 7 : 5, experts ? 72 : 52);
  t.cost[2] = t.least <= 256 ? cost(t.least, 256, 2, experts ? 16 : 10)
                             : cost(t.least, 512, wide ? 3 : 2, experts ? 26 : 24);
  return t;
}
// Rows and columns of a tile.
uint32_t side_of(const Tiles& t) {
  if (t.cost[0] <= t.cost[1] && t.cost[0] <= t.cost[2]) return 256;
  return t.cost[1] <= t.cost[2] ? 128 : 64;
}

// Rows (a multiple of 256) that go first as large tiles where the rest would begin
// another round, and costs less in a launch of its own: 4100 x 4096 x 4096 (rows,
// contraction, columns) takes 80 us in one, as tiles of 128.
uint64_t rows_first(uint64_t rows, uint64_t cols, uint64_t depth, size_t bytes) {
  auto cost = [&](uint64_t n) {
    if (n <= 16) return 3 * 1024 + (cols * depth >> 12);
    const Tiles t = tiles_for(kDense, n, cols, depth, 1, bytes);
    const uint64_t least = t.cost[1] < t.cost[2] ? t.cost[1] : t.cost[2];
    return t.cost[0] < least ? t.cost[0] : least;
  };
  const uint64_t main = rows / 256 * 256;
  if (main == 0 || main == rows) return 0;
  const Tiles t = tiles_for(kDense, main, cols, depth, 1, bytes);
  return t.cost[0] + 6 * 1024 + cost(rows - main) < cost(rows) ? main : 0;
}

// Parts of the contraction, 1: the tiles take it whole.  A workgroup of a small tile
// gets a stage of 128 codes in 0.22 to 0.27 us however few of them there are, so with
// few tiles the units that are left take parts of it: as many as fill all once, of one
// row tile, whose parts are small, twice, with 8 stages at least.  The sums' way through
// memory and the second kernel cost 4 us, and 5 of the host, so 32 stages have to be
// saved.  Rows x contraction x columns, us in a graph, whole and in parts, weights out of
// memory:
//   32 x 16384 x 4096: 36.4, 19.5; 64: 40.0, 22.2; 128: 39.9, 29.6
//   32 x 8192 x 8192: 22.8, 19.6; 32 x 8192 x 1024: 13.1, 8.1; 256: 13.6, 10.7
//   32 x 5120 x 2048: 12.6, 8.5; 4096 x 4096 (24 saved): 12.0, 10.1, but 11.7, 15.2 eager
//   128 x 4096 x 4096 (16 saved): 12.9, 13.7; twice full, 128 x 8192 x 8192: 24.5, 30.3;
//   4 stages at least, 32 x 4096 x 4096: 12.3
// Up to 16 rows, the kernel for them is as fast up to a contraction of 12288:
//   1 x 8192 x 8192: 16.0 there, 17.2 in parts; 16 x 8192 x 4096: 12.4, 13.0; 1 x 10240 x
//   4096: 13.5, 13.7; 1 x 12288 x 2048: 13.6, 11.9; 16: 16.0, 12.5; 1 x 16384 x 4096: 21.1,
//   17.8; 16: 23.2, 18.4; 1 x 16384 x 8192: 33.4, 35.1; 16: 39.7, 36.5; 1 x 32768 x 2048:
//   35.2, 20.1
uint32_t parts_of(uint64_t rows, uint64_t cols, uint64_t depth) {
  if (rows == 0 || rows > EC_I8_MOST_PARTS_ROWS || cols == 0 || cols > EC_MX_MAX_ROWS)
    return 1;
  const uint64_t tiles = ceil_div(rows, 64) * ceil_div(cols, 64), stages = depth / 128;
  if (rows <= kFewRows && stages < 96) return 1;
  uint64_t most = (rows <= 64 ? 512 : 256) / tiles;
  if (most > stages / 8) most = stages / 8;
  if (most < 2) return 1;
  const uint64_t each = ceil_div(stages, most);
  if (stages - each < 32) return 1;
  return (uint32_t)ceil_div(stages, each);  // none is empty
}
uint64_t part_bytes(uint64_t rows, uint64_t cols, uint64_t depth) {
  const uint32_t parts = parts_of(rows, cols, depth);
  return parts > 1 ? parts * rows * part_pitch((uint32_t)cols) * 4 : 0;
}

template <typename T>
ec_status join_as(const Product& p, void* y, hipStream_t s) {
  const uint64_t blocks = ceil_div(p.rows * (part_pitch(p.cols) / 4), 256);
  hipLaunchKernelGGL((i8_join<T>), grid_of(blocks), dim3(256), 0, s, p, (T*)y);
  return launched();
}
ec_status product_in_parts(Product p, int type, void* workspace, hipStream_t s) {
  void* y = p.y;
  p.y = workspace, p.parts = parts_of(p.rows, p.cols, p.depth);
  p.n_tiles = (uint32_t)ceil_div(p.cols, 64), p.m_tiles = (uint32_t)ceil_div(p.rows, 64);
  const uint64_t blocks = ceil_div((uint64_t)p.m_tiles * p.n_tiles, 8) * 8 * p.parts;
  hipLaunchKernelGGL((i8_tiles<1, 1, 4, int32_t, kDense, false>), grid_of(blocks), dim3(256), 0, s, p);
  const ec_status st = launched();
  if (st != EC_OK) return st;
  switch (type) {
    case EC_TYPE_F32: return join_as<float>(p, y, s);
    case EC_TYPE_F16: return join_as<f16_t>(p, y, s);
    default: return join_as<bf16_t>(p, y, s);
  }
}

template <typename T, int MODE>
ec_status tiles_of(const Product& p, hipStream_t s) {
  const Tiles t = tiles_for(MODE, p.rows, p.cols, p.depth, p.experts, sizeof(T));
  switch (side_of(t)) {
    case 256: return tiles_as<4, 4, 2, T, MODE>(p, s);
    case 128:
      return t.small <= 256 ? tiles_as<2, 2, 4, T, MODE>(p, s) : tiles_as<2, 2, 2, T, MODE>(p, s);
    default: return tiles_as<1, 1, 4, T, MODE>(p, s);
  }
}

// Whether the kernel for few rows runs, and whether it quantizes the rows itself.
bool few_rows(uint64_t rows, uint64_t experts) { return !experts && rows <= kFewRows; }
bool few_quantizing(uint64_t rows, uint64_t padded, uint64_t experts) {
  const uint64_t pieces = (padded + kPiece - 1) / kPiece;  // a short row has fewer waves
  return few_rows(rows, experts) &&
         rows * padded <= (pieces < kFewWaves ? pieces * 4 * 512 : kFewElements);
}

template <typename T, int CHUNKS, int SETS>
ec_status few_sets(const Few& f, uint32_t waves, hipStream_t s) {
  const uint32_t lds = CHUNKS ? (uint32_t)f.p.rows * (f.p.depth + 16) : 0;
  hipLaunchKernelGGL((i8_few<T, CHUNKS, SETS>), grid_of(f.p.n_tiles), dim3(64 * waves), lds, s, f);
  return launched();
}
template <typename T>
ec_status few_of(Few f, bool quantize, hipStream_t s) {
  f.p.n_tiles = (uint32_t)ceil_div(f.p.cols, kFewCols);
  const uint32_t pieces = (f.p.depth + kPiece - 1) / kPiece;
  const uint32_t waves = pieces < kFewWaves ? pieces : kFewWaves;
  const uint64_t chunks = quantize ? ceil_div(f.p.rows * f.p.depth, 512 * waves) : 0;
  if (chunks > 2) return few_sets<T, 4, 2>(f, waves, s);
  const bool deep = pieces >= 4 * kFewWaves;
  if (quantize) return deep ? few_sets<T, 2, 4>(f, waves, s) : few_sets<T, 2, 2>(f, waves, s);
  return deep ? few_sets<T, 0, 4>(f, waves, s) : few_sets<T, 0, 2>(f, waves, s);
}

template <typename T>
ec_status product_as(const Product& p, hipStream_t s) {
  if (few_rows(p.rows, p.experts)) return few_of<T>(Few{p, nullptr, 0, 0}, false, s);
  return p.experts ? tiles_of<T, kExperts>(p, s) : tiles_of<T, kDense>(p, s);
}

ec_status product(Product p, int type, void* workspace, hipStream_t s) {
  if (workspace && !p.experts && parts_of(p.rows, p.cols, p.depth) > 1)
    return product_in_parts(p, type, workspace, s);
  const size_t bytes = type_bytes(type);
  if (const uint64_t first = p.experts ? 0 : rows_first(p.rows, p.cols, p.depth, bytes)) {
    Product rest = p;
    rest.a = {p.a.codes + first * p.depth, p.a.scales + first};
    rest.y = (uint8_t*)p.y + first * p.cols * bytes;
    rest.rows = p.rows - first;
    const ec_status st = product(rest, type, nullptr, s);
    if (st != EC_OK) return st;
    p.rows = first;
  }
  switch (type) {
    case EC_TYPE_F32: return product_as<float>(p, s);
    case EC_TYPE_F16: return product_as<f16_t>(p, s);
    default: return product_as<bf16_t>(p, s);
  }
}

// Sizes and type that a product takes.
ec_status check_sizes(uint64_t rows, uint64_t cols, uint64_t depth, int type) {
  if (!type_known(type) || cols == 0 || depth == 0 || depth % 128 != 0) return EC_ERR_INVALID;
  return rows > EC_MX_MAX_ROWS || cols > EC_MX_MAX_ROWS || depth > EC_I8_MAX_DEPTH
             ? EC_ERR_UNSUPPORTED
             : EC_OK;
}
bool is_product(uint64_t rows, uint64_t cols, uint64_t depth, int type) {
  return check_sizes(rows, cols, depth, type) == EC_OK;
}

ec_status check(const void* a, const void* sa, uint64_t rows, const void* b, const void* sb,
                uint64_t cols, uint64_t depth, const void* y, int type) {
  const ec_status st = check_sizes(rows, cols, depth, type);
  if (st != EC_OK || rows == 0) return st;
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

// Codes of the workspace of a linear layer; the scales are behind them, then the sums of
// the contraction's parts.
uint64_t code_bytes(uint64_t rows, uint64_t depth) { return rows * ec_mx_padded(depth); }
uint64_t parts_begin(uint64_t rows, uint64_t depth) {
  return code_bytes(rows, depth) + ceil_div(rows * 4, 16) * 16;
}

}  // namespace

extern "C" {

ec_status ec_i8_product(const void* a_codes, const void* a_scales, uint64_t rows,
                        const void* b_codes, const void* b_scales, uint64_t cols, uint64_t depth,
                        void* y, int type, void* stream) {
  const ec_status st = check(a_codes, a_scales, rows, b_codes, b_scales, cols, depth, y, type);
  if (st != EC_OK || rows == 0) return st;
  return product(product_of(a_codes, a_scales, rows, b_codes, b_scales, cols, depth, nullptr, 0, y),
                 type, nullptr, (hipStream_t)stream);
}

size_t ec_i8_product_parts_bytes(uint64_t rows, uint64_t cols, uint64_t depth) {
  if (depth % 128 != 0 || depth > EC_I8_MAX_DEPTH) return 0;  // no such product
  return part_bytes(rows, cols, depth);
}

ec_status ec_i8_product_parts(const void* a_codes, const void* a_scales, uint64_t rows,
                              const void* b_codes, const void* b_scales, uint64_t cols,
                              uint64_t depth, void* y, int type, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const ec_status st = check(a_codes, a_scales, rows, b_codes, b_scales, cols, depth, y, type);
  if (st != EC_OK || rows == 0) return st;
  const size_t need = part_bytes(rows, cols, depth);
  if (!aligned(workspace, 16) || (need && !workspace)) return EC_ERR_INVALID;
  if (workspace_bytes < need) return EC_ERR_CAPACITY;
  return product(product_of(a_codes, a_scales, rows, b_codes, b_scales, cols, depth, nullptr, 0, y),
                 type, workspace, (hipStream_t)stream);
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
                 type, nullptr, (hipStream_t)stream);
}

uint32_t ec_i8_product_tile(uint64_t rows, uint64_t cols, uint64_t depth, int type,
                            uint32_t experts) {
  if (rows == 0 || !is_product(rows, cols, depth, type) || experts > EC_MX_MAX_GROUPS) return 0;
  if (few_rows(rows, experts)) return kFewRows;
  return side_of(tiles_for(experts ? kExperts : kDense, rows, cols, depth, experts,
                           type_bytes(type)));
}

uint64_t ec_i8_product_rows_first(uint64_t rows, uint64_t cols, uint64_t depth, int type) {
  return is_product(rows, cols, depth, type) ? rows_first(rows, cols, depth, type_bytes(type)) : 0;
}

size_t ec_i8_linear_workspace_bytes(uint64_t rows, uint64_t depth, uint64_t cols,
                                    uint32_t experts) {
  const uint64_t padded = ec_mx_padded(depth);
  if (few_quantizing(rows, padded, experts)) return 0;
  const uint64_t parts = experts ? 0 : part_bytes(rows, cols, padded);
  return parts ? parts_begin(rows, depth) + parts : code_bytes(rows, depth) + rows * 4;
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
  const uint64_t padded = ec_mx_padded(depth);
  if (few_quantizing(rows, padded, experts)) {
    const Few f{product_of(nullptr, nullptr, rows, w_codes, w_scales, cols, padded, nullptr, 0, y),
                x, stride, (uint32_t)depth};
    hipStream_t s = (hipStream_t)stream;
    switch (type) {
      case EC_TYPE_F32: return few_of<float>(f, true, s);
      case EC_TYPE_F16: return few_of<f16_t>(f, true, s);
      default: return few_of<bf16_t>(f, true, s);
    }
  }
  uint8_t* codes = (uint8_t*)workspace;
  void* scales = codes + code_bytes(rows, depth);
  const ec_status st = ec_i8_quantize(x, type, rows, depth, stride, codes, scales, stream);
  if (st != EC_OK) return st;
  return product(product_of(codes, scales, rows, w_codes, w_scales, cols, padded, offsets, experts,
                            y),
                 type, codes + parts_begin(rows, depth), (hipStream_t)stream);
}

}  // extern "C"
