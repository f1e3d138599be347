// Products of operands in the microscaled 4-bit format (include/ec_mx.h) on
// the matrix cores' scaled instructions: y = a b^T with both operands stored
// along the contraction, blocks of 32 sharing a scale.
#include <type_traits>

#include "ec_mx_device.h"

using namespace ecmx;

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFp4 = 4;  // the instructions' code of the element type

enum { kDense = 0, kExperts = 1, kTokens = 2 };

struct Operand {
  const uint8_t* codes;
  const uint8_t* scales;
};

struct Product {
  Operand a, b;
  void* y;
  const int32_t* offsets;
  uint64_t rows;     // of y (kExperts: of all groups; kTokens: of one expert's y)
  uint32_t cols;     // of y
  uint32_t depth;    // elements of a stored row
  uint32_t experts;
  uint32_t m_tiles, n_tiles;
  uint64_t tokens;   // kTokens: rows that the groups divide
};

// ---------------------------------------------------------------- tiles

// One workgroup of 2 by 2 waves computes a tile of 64 FM rows by 64 FN columns,
// a wave 32 FM by 32 FN of it with 32x32x64 instructions, whose rate measured
// 8.6 PFLOP/s against 6.8 of the 16x16x128 ones.  With FM = FN = 4 a wave's
// results fill half of its 512 registers, and an operand byte read from LDS is
// used 128 times.
//
// A stage is 128 elements (64 bytes) of every row of both operands, brought to
// LDS without passing registers.  Four stages are in LDS: one is multiplied
// while the loads of the next three fly, with one barrier a stage, placed
// before the last multiplications so that they cover the first reads of the
// next stage.
//
// The order within the contraction is free as long as both operands agree, so
// lane group g of instruction step s takes the 16-byte chunk 2 g + s of a
// row: a lane's two scale bytes of a stage are then one half word, and the
// step selects its byte in the instruction.  Chunks are stored at their number
// xor bits 1 and 2 of the row, so that 8 lanes of consecutive rows read 8
// different 16-byte columns of 128.
//
// 8192 x 8192 x 8192 in bf16: 310 us in a loop of its own (3.5 PFLOP/s; 326 to
// 341 among other kernels, fp32 362), of which the instructions alone take 270 at
// the clock that random codes leave (202 on zeros); loads and LDS reads alone
// take 220.
//
// Scales come 16 bytes a row, once in four stages, through registers: 4 bytes
// a row and stage would be as many requests of the caches as the codes are
// (half of the L2 cache's requests, measured).
template <int BM, int BN>
struct Stage {
  uint8_t a[BM * 64];
  uint8_t b[BN * 64];
};

// 16 bytes a lane from base + lane_off + off straight to LDS, 1 KiB from `to` on.
__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t base, uint32_t lane_off,
                                         uint32_t off, uint8_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (__attribute__((address_space(3))) void*)to, 16,
                                           lane_off, off, 0, 0);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const uint8_t* p) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, 0xffffffffu, 0x00027000);
}

__device__ __forceinline__ i32x8 widened(const i32x4& v) {
  return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0};  // 4-bit operands use half
}

template <int FM, int FN>
struct Fragments {
  i32x4 a[FM], b[FN];
};
template <int FM, int FN>
struct Scales {
  int a[FM], b[FN];
};

// Where this lane reads in a stage.
struct Lane {
  uint32_t a, b, sa, sb;  // step 0's chunk of its first rows; its scales
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
// of stage q of the four
template <int FM, int FN>
__device__ __forceinline__ void read(const uint8_t* scales, const Lane& at, int q,
                                     Scales<FM, FN>& f) {
#pragma unroll
  for (int i = 0; i < FM; i++)
    f.a[i] = *reinterpret_cast<const uint16_t*>(scales + at.sa + i * 512 + q * 4);
#pragma unroll
  for (int i = 0; i < FN; i++)
    f.b[i] = *reinterpret_cast<const uint16_t*>(scales + at.sb + i * 512 + q * 4);
}

// `between(i)` issues what goes between the rows of multiplications; nothing
// else is moved there.
template <int FM, int FN, int STEP, typename F>
__device__ __forceinline__ void multiply(const Fragments<FM, FN>& f, const Scales<FM, FN>& s,
                                         f32x16 (&acc)[FM][FN], F&& between) {
#pragma unroll
  for (int i = 0; i < FM; i++) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < FN; j++)
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          widened(f.b[j]), widened(f.a[i]), acc[i][j], kFp4, kFp4, STEP, s.b[j], STEP, s.a[i]);
    __builtin_amdgcn_sched_barrier(0);
    between(i);
  }
  __builtin_amdgcn_sched_barrier(0);
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

// PAST: results are stored past the caches (a branch at each store costs 1 us of
// 45 for 4096 x 4096 x 4096).
template <int FM, int FN, typename T, int MODE, bool PAST>
__global__ __launch_bounds__(256, FM * FN > 8 ? 1 : 2) void mx_tiles(const Product p) {
  constexpr int BM = 64 * FM, BN = 64 * FN, kWaves = 4;
  using St = Stage<BM, BN>;
  constexpr uint32_t kShift = FM == 1 ? 6 : FM == 2 ? 7 : 8;
  static_assert((1u << kShift) == BM, "tile rows");
  // four variables, not an array: the compiler then knows which loads a read waits for
  __shared__ __attribute__((aligned(16))) St st0, st1, st2, st3;
  __shared__ __attribute__((aligned(16))) uint8_t scales[2][(BM + BN) * 16];  // of a, then of b
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t wm = wave & 1, wn = wave >> 1;

  // the tiles that groups have, not the most they could have: each XCD gets its share
  uint32_t m_tiles = p.m_tiles;
  if (MODE == kExperts) m_tiles = min(m_tiles, used_tiles(p.offsets, p.experts, p.rows, kShift));
  // (an expert's tiles cost what it has of tokens: each XCD gets a share of
  // every expert, not some experts whole)
  uint32_t t, e = 0;
  if (!dealt(m_tiles * p.n_tiles, MODE == kTokens ? p.experts : 1, t, e)) return;
  // in an XCD's run, 8 tiles along the rows share a column tile
  const uint32_t width = 8 * p.n_tiles, band = t / width;
  const uint32_t high = min(m_tiles - band * 8, 8u);
  uint32_t tm = band * 8 + (t - band * width) % high;
  const uint32_t tn = (t - band * width) / high;

  // this tile's rows [m0, m_end) of a and y, its columns, its contraction
  uint64_t m0 = (uint64_t)tm * BM, m_end = p.rows;
  const uint32_t n0 = tn * BN;
  uint64_t k0 = 0;        // first element of the contraction in a stored row
  uint32_t k_len = p.depth;
  T* y = (T*)p.y;
  const uint8_t *bc = p.b.codes, *bs = p.b.scales;
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
    bc += (uint64_t)gt.group * p.cols * (p.depth / 2);
    bs += (uint64_t)gt.group * p.cols * (p.depth / 32);
  }
  if (MODE == kTokens) {
    uint64_t first, count;
    group_rows(p.offsets, e, p.tokens, first, count);
    k0 = (uint64_t)group_start(p.offsets, e, p.tokens) * 128;
    k_len = (uint32_t)((count + 127) / 128 * 128);
    if (k0 >= p.depth) k_len = 0;  // only with offsets out of order
    else if (k0 + k_len > p.depth) k_len = p.depth - (uint32_t)k0;
    if (k_len == 0) k0 = 0;
    y += (uint64_t)e * p.rows * p.cols;
  }

  // What this lane loads: of instruction q of an operand, row 16 q + lane / 4
  // and chunk (lane & 3) xor bits 1 and 2 of the row.  Rows past the end read
  // the last one: they only reach results that are not stored.
  const uint32_t pitch = p.depth / 2, spitch = p.depth / 32;
  const uint32_t m_last = (uint32_t)(m_end - m0) - 1, n_last = p.cols - n0 - 1;
  const uint8_t* ga = p.a.codes + m0 * pitch + k0 / 2;
  const uint8_t* gsa = p.a.scales + m0 * spitch + k0 / 32;
  const uint8_t* gb = bc + (uint64_t)n0 * pitch + k0 / 2;
  const uint8_t* gsb = bs + (uint64_t)n0 * spitch + k0 / 32;
  const uint32_t chunk = (lane & 3) ^ ((lane >> 3) & 3);
  // offsets from the tile's first row: at most 256 rows of 2^23 bytes
  constexpr int LA = BM / 16 / kWaves, LB = BN / 16 / kWaves;  // a wave's loads of a stage
  uint32_t oa[LA], ob[LB];
#pragma unroll
  for (int i = 0; i < LA; i++)
    oa[i] = min((wave * LA + i) * 16 + (lane >> 2), m_last) * pitch + chunk * 16;
#pragma unroll
  for (int i = 0; i < LB; i++)
    ob[i] = min((wave * LB + i) * 16 + (lane >> 2), n_last) * pitch + chunk * 16;
  constexpr int kLoads = LA + LB;
  const uint32_t stages = __builtin_amdgcn_readfirstlane(k_len / 128);
  // Scales of stages 4 u .. 4 u + 3: a thread has a row (two rows).  The last
  // stages may be fewer than four: theirs are loaded first, into `tail`, and
  // the loop below stays without branches (with them, the compiler moved the
  // results between registers every turn).  Where there are no four stages at
  // all, it loads codes that nothing uses.
  constexpr int kRows = (BM + BN + 255) / 256;
  const uint32_t fours = stages / 4;
  const uint8_t* scale_row[kRows];
  uint4 held[kRows], tail[kRows];
#pragma unroll
  for (int i = 0; i < kRows; i++) {
    const uint32_t row = min(threadIdx.x + i * 256, (uint32_t)(BM + BN - 1));
    scale_row[i] = row < BM ? gsa + min(row, m_last) * spitch
                            : gsb + min(row - BM, n_last) * spitch;
    const uint32_t n = stages & 3;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(scale_row[i]) + fours * 4;
    tail[i] = make_uint4(n > 0 ? w[0] : 0, n > 1 ? w[1] : 0, n > 2 ? w[2] : 0, 0);
    if (fours == 0) scale_row[i] = p.a.codes;
  }
  auto load_scales = [&](uint32_t u) {
    const uint32_t at = fours ? min(u, fours - 1) * 16 : 0;
#pragma unroll
    for (int i = 0; i < kRows; i++) __builtin_memcpy(&held[i], scale_row[i] + at, 16);
  };
  auto keep_scales = [&](uint32_t u) {
#pragma unroll
    for (int i = 0; i < kRows; i++) {
      const uint32_t row = threadIdx.x + i * 256;
      const uint4 v = u < fours ? held[i] : tail[i];
      if (kRows * 256 == BM + BN || row < BM + BN)
        *reinterpret_cast<uint4*>(&scales[u & 1][row * 16]) = v;
    }
  };
  // Past the last stage it is loaded again, so that every turn below does the
  // same and waits for the same number of loads.  Part i of FM.
  const __amdgpu_buffer_rsrc_t ra = buffer_at(ga), rb = buffer_at(gb);
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
  at.sa = (wm * 32 * FM + r) * 16 + g * 2;
  at.sb = (BM + wn * 32 * FN + r) * 16 + g * 2;

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) acc[i][j] = f32x16{};

  if (stages > 0) {
    load_scales(0);
    load_all(st0, 0);
    load_all(st1, 1);
    load_all(st2, 2);
    keep_scales(0);
    wait_and_meet<2 * kLoads>();
    Fragments<FM, FN> f0, f1;
    Scales<FM, FN> sc;
    read(scales[0], at, 0, sc);
    read(st0, at, 0, f0);
    // Stage s = 4 u + q is in `now`; its first fragments and scales are in
    // registers.  The scales of the next four are loaded at q = 0 and in LDS
    // before the barrier of q = 3; the waits count them as if they were stage
    // loads, which waits for two more at most.  The last stages (`more`
    // false) load nothing.
    auto turn = [&](uint32_t u, auto q, auto more, const St& now, const St& next, St& free) {
      if (more && q == 3) keep_scales(u + 1);
      read(now, at, 1, f1);
      if (more && q == 0) load_scales(u + 1);
      multiply<FM, FN, 0>(f0, sc, acc, [&](int i) {
        if (more) load(free, 4 * u + q + 3, i);
      });
      if (more) wait_and_meet<2 * kLoads>();
      else wait_and_meet<0>();
      Scales<FM, FN> snext;
      read(scales[(q == 3 ? u + 1 : u) & 1], at, (q + 1) & 3, snext);
      read(next, at, 0, f0);
      multiply<FM, FN, 1>(f1, sc, acc, [](int) {});
      sc = snext;
    };
    using std::integral_constant;
    constexpr integral_constant<int, 0> q0;
    constexpr integral_constant<int, 1> q1;
    constexpr integral_constant<int, 2> q2;
    constexpr integral_constant<int, 3> q3;
    constexpr std::true_type more;
    constexpr std::false_type last;
    for (uint32_t u = 0; u < fours; u++) {
      turn(u, q0, more, st0, st1, st3);
      turn(u, q1, more, st1, st2, st0);
      turn(u, q2, more, st2, st3, st1);
      turn(u, q3, more, st3, st0, st2);
    }
    if (stages & 3) turn(fours, q0, last, st0, st1, st3);
    if ((stages & 3) > 1) turn(fours, q1, last, st1, st2, st0);
    if ((stages & 3) > 2) turn(fours, q2, last, st2, st3, st1);
    wait_and_meet<0>();  // the stages' memory is used again below
  }

  // A lane has row lane & 31 of y and 4 consecutive columns in each quarter
  // of a result: 32 rows at a time go through LDS (this wave's own part) and
  // leave as whole 16-byte pieces.  Results are rounded once, here.
  constexpr uint32_t kRow = 32 * FN * sizeof(T), kPitch = kRow + 16;
  static_assert(32 * kPitch <= sizeof(St), "the stage holds the results");
  uint8_t* out = reinterpret_cast<uint8_t*>(wave == 0   ? &st0
                                             : wave == 1 ? &st1
                                             : wave == 2 ? &st2
                                                         : &st3);
  const uint32_t nw = n0 + wn * 32 * FN;
#pragma unroll
  for (int i = 0; i < FM; i++) {
#pragma unroll
    for (int j = 0; j < FN; j++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        T v[4];
#pragma unroll
        for (int u = 0; u < 4; u++) v[u] = (T)acc[i][j][4 * q + u];
        __builtin_memcpy(out + r * kPitch + (j * 32 + q * 8 + g * 4) * sizeof(T), v, sizeof(v));
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

// Up to 16 rows (of a group) against 16 NT columns a workgroup: what counts is
// reading b once, at full bandwidth.  The waves divide the contraction in
// pieces of 512 elements; a lane loads 16 bytes of a row of b and an
// instruction's 4 lanes of a row 64 bytes, straight into registers.
// With x unquantized (T), the workgroup quantizes its rows into LDS first,
// while the first loads of b are in flight.
//
// A wave keeps two loads of 4 KiB and more in flight: the pieces of two rounds
// (SETS = 2) where it has several, else those of two column tiles (NT = 2).
// One row by 8192 x 8192: 8.7 us, 4.1 TB/s of the weights.  Rows of an expert
// past 16 go to other workgroups, so that a crowded expert does not wait.
constexpr uint32_t kFewCols = 16, kFewRows = 16, kFewWaves = 8;
constexpr uint32_t kPiece = 512;

__device__ __forceinline__ f32x4 multiply16(const i32x4& b, const i32x4& a, f32x4 acc, int sb,
                                            int sa) {
  const i32x8 wb = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  const i32x8 wa = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wb, wa, acc, kFp4, kFp4, 0, sb, 0, sa);
}

struct Few {
  const void* x;
  uint64_t stride;
  uint32_t raw_depth;  // elements of a row of x
  Operand a;           // x in the 4-bit form, where it is
  Operand b;
  void* y;
  const int32_t* offsets;
  uint64_t rows;
  uint32_t cols, depth, n_tiles;
  uint32_t experts;      // of x unquantized; 0: none
  uint32_t held, shift;  // rows of a workgroup: up to held, of groups 2^shift = held
};

// A piece of b: 4 steps of 128 elements, and their scale bytes, whole words
// (a lane's byte is the one with its group's number).
template <int NT>
struct Piece {
  i32x4 b[NT][4];
  uint32_t s[NT][4];
};

template <typename T, bool QUANTIZE, int NT, int SETS>
__global__ __launch_bounds__(64 * kFewWaves, 4) void mx_few(const Few p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ float part[kFewWaves][256 * NT];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t waves = blockDim.x >> 6;
  const uint32_t r = lane & 15, g = lane >> 4;
  const uint32_t block = block_number(), tn = block % p.n_tiles;
  const uint32_t n0 = tn * kFewCols * NT;
  // (experts' rows come unquantized: in the 4-bit form they go to the tiles)
  const uint32_t experts = QUANTIZE ? p.experts : 0;
  uint64_t row0 = 0;
  uint32_t here = (uint32_t)p.rows;
  T* y = (T*)p.y;
  const uint8_t *bc = p.b.codes, *bs = p.b.scales;
  if (experts) {
    const GroupTile gt = find_tile(p.offsets, experts, p.rows, p.shift, block / p.n_tiles);
    const uint64_t skip = (uint64_t)gt.local << p.shift;
    if (gt.group == experts) {  // rows of no group: zeros
      const int64_t f = p.offsets[experts];
      const uint64_t m0 = (f < 0 ? 0 : f) + skip, end = min(m0 + p.held, p.rows);
      const uint32_t col = n0 + threadIdx.x % (kFewCols * NT);
      if (col < p.cols)
        for (uint64_t m = m0 + threadIdx.x / (kFewCols * NT); m < end;
             m += blockDim.x / (kFewCols * NT))
          y[m * p.cols + col] = (T)0.0f;
      return;
    }
    if (skip >= gt.count) return;  // only with offsets out of order
    row0 = gt.first + skip;
    here = (uint32_t)min((uint64_t)p.held, gt.count - skip);
    bc += (uint64_t)gt.group * p.cols * (p.depth / 2);
    bs += (uint64_t)gt.group * p.cols * (p.depth / 32);
  } else if (block >= p.n_tiles) {
    return;
  }
  const uint32_t pitch = p.depth / 2, spitch = p.depth / 32;
  const uint32_t steps = p.depth / 128, pieces = (steps + 3) / 4;
  const uint8_t *gb[NT], *gsb[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) {
    const uint32_t n = min(n0 + t * kFewCols + r, p.cols - 1);
    gb[t] = bc + (uint64_t)n * pitch + g * 16;
    gsb[t] = bs + (uint64_t)n * spitch;
  }
  const uint32_t lpitch = pitch + 16;  // rows of LDS start 4 banks apart
  uint8_t* lscales = lds + (uint32_t)min((uint64_t)p.held, p.rows) * lpitch;

  auto load = [&](Piece<NT>& f, uint32_t at) {
#pragma unroll
    for (int t = 0; t < NT; t++) {
#pragma unroll
      for (int s = 0; s < 4; s++)  // steps past the end read the last one
        f.b[t][s] = *reinterpret_cast<const i32x4*>(gb[t] + min(at * 4 + s, steps - 1) * 64);
      if (at * 4 + 4 <= steps) {
        __builtin_memcpy(f.s[t], gsb[t] + at * 16, 16);
      } else {
#pragma unroll
        for (int s = 0; s < 4; s++)
          __builtin_memcpy(&f.s[t][s], gsb[t] + min(at * 4 + s, steps - 1) * 4, 4);
      }
    }
  };

  Piece<NT> f[SETS];
#pragma unroll
  for (int i = 0; i < SETS; i++)
    if (wave + i * waves < pieces) load(f[i], wave + i * waves);
  const uint32_t lr = min(r, here - 1);
  const uint8_t *ga, *gsa;
  if constexpr (QUANTIZE) {
    const uint32_t chunks = p.depth / 8, total = here * chunks;
    constexpr int Q = 4;  // loads in flight
    for (uint32_t i0 = threadIdx.x; i0 < total; i0 += Q * blockDim.x) {
      Eight<T> v[Q];
      uint32_t row[Q], c[Q];
#pragma unroll
      for (int q = 0; q < Q; q++) {  // quads of lanes share a block
        const uint32_t i = i0 + q * blockDim.x;
        row[q] = i / chunks, c[q] = i - row[q] * chunks;
        v[q] = load_eight((const T*)p.x + (row0 + row[q]) * p.stride + c[q] * 8,
                          i < total ? (int64_t)p.raw_depth - c[q] * 8 : 0);
      }
#pragma unroll
      for (int q = 0; q < Q; q++) {
        if (i0 + q * blockDim.x >= total) break;
        const Scale s = scale_of(exponent_of<T>(max_of_4_lanes(magnitude_of_eight(v[q]))));
        *reinterpret_cast<uint32_t*>(lds + row[q] * lpitch + c[q] * 4) = code_eight(v[q], s.size);
        if ((c[q] & 3) == 0) lscales[row[q] * spitch + c[q] / 4] = (uint8_t)s.byte;
      }
    }
    __syncthreads();
    ga = lds + lr * lpitch + g * 16;
    gsa = lscales + lr * spitch + g;
  } else {
    ga = p.a.codes + (row0 + lr) * pitch + g * 16;
    gsa = p.a.scales + (row0 + lr) * spitch + g;
  }
  f32x4 acc[NT] = {};
  for (uint32_t piece = wave; piece < pieces; piece += SETS * waves) {
#pragma unroll
    for (int i = 0; i < SETS; i++) {
      const uint32_t now = piece + i * waves;
      if (now >= pieces) break;
#pragma unroll
      for (int s = 0; s < 4; s++) {
        const uint32_t step = now * 4 + s;
        if (step < steps) {
          const i32x4 fa = *reinterpret_cast<const i32x4*>(ga + step * 64);
          const int sa = gsa[step * 4];
#pragma unroll
          for (int t = 0; t < NT; t++)
            acc[t] = multiply16(f[i].b[t][s], fa, acc[t], (int)(f[i].s[t][s] >> (8 * g)), sa);
        }
      }
      if (now + SETS * waves < pieces) load(f[i], now + SETS * waves);
    }
  }
  // a lane has row r of y and columns 4 g .. 4 g + 3 of a tile; the waves'
  // parts are added in their order
#pragma unroll
  for (int t = 0; t < NT; t++)
    *reinterpret_cast<f32x4*>(&part[wave][(r * NT + t) * 16 + g * 4]) = acc[t];
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < here * 16 * NT; i += blockDim.x) {
    float sum = 0;
    for (uint32_t w = 0; w < waves; w++) sum += part[w][i];
    const uint32_t col = n0 + i % (16 * NT);
    if (col < p.cols) y[(row0 + i / (16 * NT)) * p.cols + col] = (T)sum;
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
  const uint64_t tiles = ceil_div(m * p.n_tiles, 8) * 8 * (MODE == kTokens ? p.experts : 1);
  if (tiles > kMostBlocks) return EC_ERR_UNSUPPORTED;
  p.m_tiles = (uint32_t)m;
  // Weights' gradients are read after the whole backward pass, when no cache has
  // them: past what the L2 caches hold, 32 MiB, in whole lines (16 x 2048 x 2048
  // fp32 stored as usual 115 us, past 101; 64 x 4096 x 2048 bf16 575 and 435; not
  // in rows of 1304 bf16 58 and 70, of 366 fp32 52 and 87). Ragged rows of other
  // products fill most of their lines as large tiles: from 512 MiB on (32768 x 512
  // x 16389 bf16 491 and 393; as tiles of 128, 6013 x 384 x 52412, 238 and 346).
  const uint64_t bytes = p.rows * p.cols * sizeof(T) * (MODE == kTokens ? p.experts : 1);
  const uint64_t row = p.cols * sizeof(T);
  if constexpr (FM > 1) {  // under 128 tiles of 128, where those of 64 run, is 8 MiB at most
    if (MODE == kTokens ? row % 128 == 0 && bytes > (32ull << 20)
                        : past_caches(bytes, row) || (FM == 4 && bytes >= (512ull << 20))) {
      hipLaunchKernelGGL((mx_tiles<FM, FN, T, MODE, true>), grid_of(tiles), dim3(256), 0, s, p);
      return launched();
    }
  }
  hipLaunchKernelGGL((mx_tiles<FM, FN, T, MODE, false>), grid_of(tiles), dim3(256), 0, s, p);
  return launched();
}

// The larger tile reads less and keeps the matrix units busier, but the last
// round of its workgroups (one a unit, 256 in all) may be nearly empty, and
// nothing hides where it starts and ends; of the tiles of 128, two workgroups
// share a unit.  Measured for 8192 x 8192 outputs in bf16, a contraction of
// 128, 512, 1024, 2048, 4096, 8192, us: large 37, 49, 64, 101, 166, 288, small
// 31, 47, 76, 122, 216, 388: about 8 and 8 more for each 1024 a round of 256,
// and 3.5 and 5.5 more a round of 512.  Finding a group's rows adds 5 to a
// round of large ones and tokens' parts 3 (16 groups, 16384 x 2048 x 2048:
// large 62 and 85 us, small 59 and 79; tokens of 4 groups, 4096 x 4096 x 4096:
// large 71, small 77).  A round's stores are half of what does not grow with
// the contraction: a dense product in fp32 stores twice as much, and costs 17
// and 9, and 5 and 5.5, there (8192 x 8192 outputs, contractions of 512, 2048,
// 4096 and 8192: large 94, 143, 216, 362 us, small 62, 117, 207, 409; experts
// and tokens in fp32 are within 9% of the better tile with the costs of bf16).
// Costs in us times 1024.
//
// Tiles of 64 where fewer than 128 of 128 would run: 1024 x 4096 x 4096 takes
// 22 us with tiles of 128 and 30 with 64, 64 x 4096 x 4096 10.4 with 64.
struct Tiles {
  uint64_t large, small;            // how many
  uint64_t cost_large, cost_small;  // too few large ones: more than anything
  uint64_t round_small;             // what 512 small ones cost
};
Tiles tiles_for(int mode, uint64_t rows, uint64_t cols, uint64_t depth, uint64_t groups,
                size_t bytes) {
  const uint64_t extra = mode == kExperts ? groups / 2 : 0;  // half a tile more for each
  const uint64_t sets = mode == kTokens ? groups : 1;
  Tiles t;
  t.large = (ceil_div(rows, 256) + extra) * ceil_div(cols, 256) * sets;
  t.small = (ceil_div(rows, 128) + extra) * ceil_div(cols, 128) * sets;
  const bool twice = mode == kDense && bytes == 4;
  const uint64_t start = mode == kDense ? (twice ? 17 : 8) : mode == kExperts ? 13 : 11;
  t.round_small = (twice ? 5120 : 3584) + depth * 11 / 2;
  t.cost_large = t.large < 192 ? ~0ull >> 1
                               : ceil_div(t.large, 256) * (start * 1024 + depth * (twice ? 9 : 8));
  t.cost_small = ceil_div(t.small, 512) * t.round_small;
  return t;
}

// Rows and columns of a tile.
uint32_t side_of(const Tiles& t) {
  return t.cost_large <= t.cost_small ? 256 : t.small >= 128 ? 128 : 64;
}
// The contraction that the costs go by: a stored row, or an expert's mean part of it.
uint64_t mean_depth(int mode, uint64_t depth, uint64_t tokens, uint32_t experts) {
  return mode == kTokens ? tokens / experts : depth;
}

template <typename T, int MODE>
ec_status tiles_of(const Product& p, hipStream_t s) {
  switch (side_of(tiles_for(MODE, p.rows, p.cols,
                            mean_depth(MODE, p.depth, p.tokens, p.experts), p.experts,
                            sizeof(T)))) {
    case 256: return tiles_as<4, 4, T, MODE>(p, s);
    case 128: return tiles_as<2, 2, T, MODE>(p, s);
    default: return tiles_as<1, 1, T, MODE>(p, s);
  }
}

// What a product of under 256 rows costs, by the way that it takes (us, contractions
// of 1024, 4096, 8192): 16 rows by 4096 columns 3.7, 5.6, 8.8, by 57344 11.6, 35, 82;
// 250 by 4096 (256 tiles of 64) 4.6, 8.8, 14, by 16384 (256 of 128) 7.2, 17, 27, by
// 57344 (224 of 256) 18.5, 43, 85.
uint64_t cost_of_few(uint64_t rows, uint64_t cols, uint64_t depth, size_t bytes) {
  if (rows <= kFewRows) return 3 * 1024 + (cols * depth * 10 >> 16);
  const Tiles t = tiles_for(kDense, rows, cols, depth, 1, bytes);
  if (t.cost_large <= t.cost_small) return t.cost_large + 4 * 1024;
  if (t.small >= 128) return ceil_div(t.small, 256) * (3 * 1024 + depth * 3);
  return ceil_div(ceil_div(rows, 64) * ceil_div(cols, 64), 256) * (3 * 1024 + depth * 3 / 2);
}

// Rows (a multiple of 256) whose large tiles go first where the rest, which
// would begin another round, goes to a launch of its own, which costs 6 us
// beside its work.  A last round of small tiles that is at most half full costs
// half of one (2112 tiles 4.2 rounds, 1056 2.5).  Measured in one launch and in
// two: 4100 x 4096 x 4096 (rows, contraction, columns) 66 and 52 us, 4346 x
// 2048 x 16384 114 and 107; in one by this rule: 4100 x 1024 x 8190 38 and 44,
// 506 x 8192 x 57344 152 and 166.  Of 390 products that it sends in two, 363
// were faster for it (9% on average) and the others up to 10% slower.
uint64_t rows_first(uint64_t rows, uint64_t cols, uint64_t depth, size_t bytes) {
  const uint64_t main = rows / 256 * 256;
  if (main == 0 || main == rows) return 0;
  const Tiles all = tiles_for(kDense, rows, cols, depth, 1, bytes);
  const Tiles t = tiles_for(kDense, main, cols, depth, 1, bytes);
  const uint64_t small = ceil_div(all.small, 256) * all.round_small / 2;
  const uint64_t best = all.cost_large < small ? all.cost_large : small;
  const uint64_t rest = cost_of_few(rows - main, cols, depth, bytes);
  return t.cost_large + 6 * 1024 + rest < best ? main : 0;
}

template <int MODE>
ec_status tiles(const Product& p, int type, hipStream_t s) {
  switch (type) {
    case EC_TYPE_F32: return tiles_of<float, MODE>(p, s);
    case EC_TYPE_F16: return tiles_of<f16_t, MODE>(p, s);
    default: return tiles_of<bf16_t, MODE>(p, s);
  }
}

template <typename T, int NT, int SETS>
ec_status few_as(Few p, bool quantize, uint32_t waves, hipStream_t s) {
  p.n_tiles = (uint32_t)ceil_div(p.cols, kFewCols * NT);
  if (!quantize) p.held = kFewRows;
  p.shift = __builtin_ctz(p.held);
  // groups round up each, and the rows of no group once more
  const uint64_t m =
      p.experts ? ceil_div(p.rows, p.held) + (p.experts < p.rows ? p.experts : p.rows) + 1 : 1;
  const uint64_t blocks = p.n_tiles * m;
  if (blocks > kMostBlocks) return EC_ERR_UNSUPPORTED;
  const uint32_t rows = p.rows < p.held ? (uint32_t)p.rows : p.held;  // what LDS has to hold
  const uint32_t lds = quantize ? rows * (p.depth / 2 + 16 + p.depth / 32) : 0;
  if (quantize)
    hipLaunchKernelGGL((mx_few<T, true, NT, SETS>), grid_of(blocks), dim3(64 * waves), lds,
                       s, p);
  else
    hipLaunchKernelGGL((mx_few<T, false, NT, SETS>), grid_of(blocks), dim3(64 * waves), lds,
                       s, p);
  return launched();
}

template <typename T>
ec_status few_of(const Few& p, bool quantize, hipStream_t s) {
  const uint32_t pieces = (p.depth + kPiece - 1) / kPiece;
  const uint32_t waves = pieces < kFewWaves ? pieces : kFewWaves;
  const uint64_t columns = (uint64_t)p.cols * (p.experts ? p.experts : 1);
  // two column tiles where a wave has one piece and 512 workgroups remain: 4
  // rows for each of 32 experts of 1024 x 2048 take 11.0 us, with one 12.4
  if (pieces <= kFewWaves && columns >= 512 * 2 * kFewCols)
    return few_as<T, 2, 1>(p, quantize, waves, s);
  return few_as<T, 1, 2>(p, quantize, waves, s);
}

ec_status few(const Few& p, int type, bool quantize, hipStream_t s) {
  switch (type) {
    case EC_TYPE_F32: return few_of<float>(p, quantize, s);
    case EC_TYPE_F16: return few_of<f16_t>(p, quantize, s);
    default: return few_of<bf16_t>(p, quantize, s);
  }
}

// The limit of a row's length holds for `row`, depth without what groups add to it (the
// kernels' offsets within a tile hold up to 2^25 elements).
ec_status check(const void* a, const void* sa, uint64_t rows, const void* b, const void* sb,
                uint64_t cols, uint64_t depth, uint64_t row, const void* y, int type) {
  if (!type_known(type) || cols == 0 || depth % 128 != 0) return EC_ERR_INVALID;
  if (rows > EC_MX_MAX_ROWS || cols > EC_MX_MAX_ROWS || row > EC_MX_MAX_DEPTH)
    return EC_ERR_UNSUPPORTED;
  if (rows == 0) return EC_OK;
  if (!y || !aligned(y, type_bytes(type))) return EC_ERR_INVALID;
  if (depth && (!read_ok(b, sb) || !read_ok(a, sa))) return EC_ERR_INVALID;
  return EC_OK;
}

ec_status check_groups(const int32_t* offsets, uint32_t groups) {
  if (!offsets || !aligned(offsets, 4) || groups == 0) return EC_ERR_INVALID;
  return groups > EC_MX_MAX_GROUPS ? EC_ERR_UNSUPPORTED : EC_OK;
}

// How ec_mx_linear goes.  Measured with the quantization, us a call on the
// GPU, for 1, 4, 8, 16 rows: 8192 x 8192 dense, quantizing in the product 8.7,
// 10.9, 15.3, 16.7, before it 10.8, 12.2, 13.6, 16.2, tiles 16.4 each; 32
// experts of 1024 x 2048 (rows of each) 10.8, 11.0, 13.1, 23, before it 12.5,
// 12.9, 13.6, 15.8, tiles 12.0, 11.9, 12.0, 12.3.
enum Way { kFewQuantizing, kFewStored, kTiled };
constexpr uint32_t kFewLds = 48 * 1024;

// Rows that fit, a power of two (0: none).
uint32_t held_rows(uint64_t padded) {
  const uint64_t each = padded / 2 + 16 + padded / 32;
  uint32_t n = kFewRows;
  while (n && n * each > kFewLds) n /= 2;
  return n;
}

Way way_of(uint64_t rows, uint64_t padded, uint32_t experts) {
  const uint64_t mean = experts ? ceil_div(rows, experts) : rows;
  if (mean <= 4 && held_rows(padded) >= mean) return kFewQuantizing;
  return !experts && rows <= kFewRows ? kFewStored : kTiled;
}

}  // namespace

extern "C" {

ec_status ec_mx_product(const void* a_codes, const void* a_scales, uint64_t rows,
                        const void* b_codes, const void* b_scales, uint64_t cols, uint64_t depth,
                        void* y, int type, void* stream) {
  ec_status st = check(a_codes, a_scales, rows, b_codes, b_scales, cols, depth, depth, y, type);
  if (st != EC_OK || rows == 0) return st;
  if (depth == 0) return EC_ERR_INVALID;
  if (const uint64_t first = rows_first(rows, cols, depth, type_bytes(type))) {
    st = ec_mx_product((const uint8_t*)a_codes + first * (depth / 2),
                       (const uint8_t*)a_scales + first * (depth / 32), rows - first, b_codes,
                       b_scales, cols, depth, (uint8_t*)y + first * cols * type_bytes(type), type,
                       stream);
    if (st != EC_OK) return st;
    rows = first;
  }
  if (rows <= kFewRows) {
    Few f{};
    f.a = {(const uint8_t*)a_codes, (const uint8_t*)a_scales};
    f.b = {(const uint8_t*)b_codes, (const uint8_t*)b_scales};
    f.y = y, f.rows = rows, f.cols = (uint32_t)cols, f.depth = (uint32_t)depth;
    return few(f, type, false, (hipStream_t)stream);
  }
  Product p{};
  p.a = {(const uint8_t*)a_codes, (const uint8_t*)a_scales};
  p.b = {(const uint8_t*)b_codes, (const uint8_t*)b_scales};
  p.y = y, p.rows = rows, p.cols = (uint32_t)cols, p.depth = (uint32_t)depth;
  return tiles<kDense>(p, type, (hipStream_t)stream);
}

ec_status ec_mx_product_experts(const void* a_codes, const void* a_scales, uint64_t rows,
                                const void* b_codes, const void* b_scales, uint64_t cols,
                                uint64_t depth, const int32_t* offsets, uint32_t experts, void* y,
                                int type, void* stream) {
  ec_status st = check_groups(offsets, experts);
  if (st != EC_OK) return st;
  st = check(a_codes, a_scales, rows, b_codes, b_scales, cols, depth, depth, y, type);
  if (st != EC_OK || rows == 0) return st;
  if (depth == 0) return EC_ERR_INVALID;
  Product p{};
  p.a = {(const uint8_t*)a_codes, (const uint8_t*)a_scales};
  p.b = {(const uint8_t*)b_codes, (const uint8_t*)b_scales};
  p.y = y, p.rows = rows, p.cols = (uint32_t)cols, p.depth = (uint32_t)depth;
  p.offsets = offsets, p.experts = experts;
  return tiles<kExperts>(p, type, (hipStream_t)stream);
}

ec_status ec_mx_product_tokens(const void* a_codes, const void* a_scales, uint64_t rows,
                               const void* b_codes, const void* b_scales, uint64_t cols,
                               uint64_t tokens, const int32_t* offsets, uint32_t experts, void* y,
                               int type, void* stream) {
  ec_status st = check_groups(offsets, experts);
  if (st != EC_OK) return st;
  if (tokens > EC_MX_MAX_ROWS) return EC_ERR_UNSUPPORTED;
  const uint64_t depth = ec_mx_padded_groups(tokens, experts);
  st = check(a_codes, a_scales, rows, b_codes, b_scales, cols, depth, ec_mx_padded(tokens), y,
             type);
  if (st != EC_OK || rows == 0) return st;
  Product p{};
  p.a = {(const uint8_t*)a_codes, (const uint8_t*)a_scales};
  p.b = {(const uint8_t*)b_codes, (const uint8_t*)b_scales};
  p.y = y, p.rows = rows, p.cols = (uint32_t)cols, p.depth = (uint32_t)depth;
  p.offsets = offsets, p.experts = experts, p.tokens = tokens;
  return tiles<kTokens>(p, type, (hipStream_t)stream);
}

uint32_t ec_mx_product_tile(uint64_t rows, uint64_t cols, uint64_t depth, int type,
                            uint32_t experts, uint64_t tokens) {
  if (!type_known(type) || rows == 0 || cols == 0 || (tokens && !experts)) return 0;
  const int mode = tokens ? kTokens : experts ? kExperts : kDense;
  if (mode == kDense && rows <= kFewRows) return kFewRows;
  return side_of(tiles_for(mode, rows, cols, mean_depth(mode, depth, tokens, experts), experts,
                           type_bytes(type)));
}

uint64_t ec_mx_product_rows_first(uint64_t rows, uint64_t cols, uint64_t depth, int type) {
  return type_known(type) ? rows_first(rows, cols, depth, type_bytes(type)) : 0;
}

size_t ec_mx_linear_workspace_bytes(uint64_t rows, uint64_t depth, uint64_t cols,
                                    uint32_t experts) {
  (void)cols;
  const uint64_t padded = ec_mx_padded(depth);
  if (rows == 0 || way_of(rows, padded, experts) == kFewQuantizing) return 0;
  return (rows * (padded / 2) + 15) / 16 * 16 + rows * (padded / 32);
}

ec_status ec_mx_linear(const void* x, int type, uint64_t rows, uint64_t depth, uint64_t stride,
                       const void* w_codes, const void* w_scales, uint64_t cols,
                       const int32_t* offsets, uint32_t experts, void* y, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!type_known(type) || depth == 0 || cols == 0 || stride < depth || (!offsets) != (!experts))
    return EC_ERR_INVALID;
  if (experts > EC_MX_MAX_GROUPS || rows > EC_MX_MAX_ROWS || cols > EC_MX_MAX_ROWS ||
      depth > EC_MX_MAX_DEPTH)
    return EC_ERR_UNSUPPORTED;
  if (rows == 0) return EC_OK;
  if (!x || !aligned(x, type_bytes(type)) || !y || !aligned(y, type_bytes(type)) ||
      !read_ok(w_codes, w_scales) || !aligned(offsets, 4) || !aligned(workspace, 16))
    return EC_ERR_INVALID;
  const size_t need = ec_mx_linear_workspace_bytes(rows, depth, cols, experts);
  if (need && !workspace) return EC_ERR_INVALID;
  if (workspace_bytes < need) return EC_ERR_CAPACITY;
  const uint64_t padded = ec_mx_padded(depth);
  const Way way = way_of(rows, padded, experts);
  if (way == kFewQuantizing) {
    Few f{};
    f.x = x, f.stride = stride, f.raw_depth = (uint32_t)depth;
    f.b = {(const uint8_t*)w_codes, (const uint8_t*)w_scales};
    f.y = y, f.rows = rows, f.cols = (uint32_t)cols, f.depth = (uint32_t)padded;
    f.offsets = offsets, f.experts = experts;
    f.held = held_rows(padded);
    return few(f, type, true, (hipStream_t)stream);
  }
  uint8_t* codes = (uint8_t*)workspace;
  uint8_t* scales = codes + (rows * (padded / 2) + 15) / 16 * 16;
  const ec_status st = ec_mx_quantize(x, type, rows, depth, stride, codes, scales, stream);
  if (st != EC_OK) return st;
  if (experts)
    return ec_mx_product_experts(codes, scales, rows, w_codes, w_scales, cols, padded, offsets,
                                 experts, y, type, stream);
  return ec_mx_product(codes, scales, rows, w_codes, w_scales, cols, padded, y, type, stream);
}

}  // extern "C"
