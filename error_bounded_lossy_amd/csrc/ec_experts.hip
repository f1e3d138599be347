// Tokens sorted by expert and back (include/ec_experts.h): a stable counting
// sort of the choices, and the moves of rows between the tokens' order and
// the experts', with weights and gradients.  The moves are bound by memory:
// each one reads and writes every row it has to once.
#include "ec_experts.h"
#include "ec_mx_device.h"

using namespace ecmx;

namespace {

// ---------------------------------------------------------------- sort

constexpr uint32_t kSortThreads = 1024, kSortWaves = kSortThreads / 64;
// ids of one workgroup's part; several parts count first and place after
constexpr uint32_t kPart = 1024;

__device__ __forceinline__ uint32_t expert_of(const void* ids, uint32_t wide, uint64_t i,
                                              uint32_t experts) {
  const int64_t id = wide ? ((const int64_t*)ids)[i] : ((const int32_t*)ids)[i];
  return id >= 0 && id < (int64_t)experts ? (uint32_t)id : experts;
}

// Lanes of this wave that hold the same expert: one ballot a bit of its number.
__device__ __forceinline__ uint64_t same_lanes(uint32_t e, uint32_t bits, uint64_t active) {
  uint64_t same = active;
  for (uint32_t b = 0; b < bits; b++) {
    const uint64_t m = __ballot((e >> b) & 1);
    same &= (e >> b) & 1 ? m : ~m;
  }
  return same;
}

// counts[part][experts + 1] (the last column: dropped choices).
__global__ __launch_bounds__(kSortThreads) void expert_count(const void* ids, uint32_t wide,
                                                             uint64_t n, uint32_t experts,
                                                             uint32_t per, uint32_t* counts) {
  __shared__ uint32_t count[EC_EXPERTS_MAX + 1];
  for (uint32_t e = threadIdx.x; e <= experts; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const uint64_t first = (uint64_t)blockIdx.x * per, last = min(first + per, n);
  for (uint64_t i = first + threadIdx.x; i < last; i += kSortThreads)
    atomicAdd(&count[expert_of(ids, wide, i, experts)], 1u);  // whole numbers: any order
  __syncthreads();
  for (uint32_t e = threadIdx.x; e <= experts; e += kSortThreads)
    counts[(uint64_t)blockIdx.x * (experts + 1) + e] = count[e];
}

// Each workgroup places its part: it adds up the counts of the parts before
// it (and of all, for the offsets), then ranks its choices 1024 at a time: a
// rank is the number of equal choices before it in its wave, in the waves
// before it and in the rounds before.  A single part counts for itself.
// Bound by its chain of loads, barriers and LDS sums: 6.3 us for 65536 choices
// in 64 parts (after 4.6 us of counting), 3.6 us for 256 in one.
__global__ __launch_bounds__(kSortThreads) void expert_place(
    const void* ids, uint32_t wide, uint64_t n, uint32_t experts, uint32_t per, uint32_t parts,
    const uint32_t* counts, int32_t* order, int32_t* place, int32_t* offsets) {
  __shared__ uint32_t next[EC_EXPERTS_MAX + 1];   // where the next choice of an expert goes
  extern __shared__ uint16_t ahead[];             // [waves][experts]: of this round
  __shared__ uint32_t sums[kSortWaves];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, cols = experts + 1;
  const uint64_t first = (uint64_t)blockIdx.x * per, last = min(first + per, n);

  // thread e: this expert's choices in all parts, and in the parts before
  uint32_t all = 0, before = 0;
  if (counts) {
    // 16 loads at a time: a latency each would be most of this kernel's time
    if (tid < cols) {
      for (uint32_t p = 0; p < parts; p += 16) {
        uint32_t c[16];
#pragma unroll
        for (int i = 0; i < 16; i++)
          c[i] = p + i < parts ? counts[(uint64_t)(p + i) * cols + tid] : 0;
#pragma unroll
        for (int i = 0; i < 16; i++) {
          before += p + i < blockIdx.x ? c[i] : 0;
          all += c[i];
        }
      }
    }
  } else {
    for (uint32_t e = tid; e < cols; e += kSortThreads) next[e] = 0;
    __syncthreads();
    for (uint64_t i = first + tid; i < last; i += kSortThreads)
      atomicAdd(&next[expert_of(ids, wide, i, experts)], 1u);
    __syncthreads();
    if (tid < cols) all = next[tid];
    __syncthreads();
  }
  // exclusive sum over the experts (at most 1024: thread 1024 would be the
  // dropped ones with 1024 experts, which need no place)
  const uint32_t mine = tid < experts ? all : 0;
  uint32_t upto = mine;
  for (uint32_t d = 1; d < 64; d <<= 1) {
    const uint32_t t = __shfl_up(upto, d);
    upto += lane >= d ? t : 0;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  uint32_t base = 0, total = 0;
  for (uint32_t w = 0; w < kSortWaves; w++) {
    base += w < wave ? sums[w] : 0;
    total += sums[w];
  }
  const uint32_t start = base + upto - mine;
  if (tid < experts) {
    next[tid] = start + before;
    if (blockIdx.x == 0) offsets[tid] = (int32_t)start;
  }
  if (blockIdx.x == 0 && tid == 0) offsets[experts] = (int32_t)total;
  for (uint64_t i = (uint64_t)total + blockIdx.x * kSortThreads + tid; i < n;
       i += (uint64_t)gridDim.x * kSortThreads)
    order[i] = -1;

  const uint32_t bits = 32 - __builtin_clz(experts);  // numbers 0 .. experts
  for (uint64_t r = first; r < last; r += kSortThreads) {
    for (uint32_t k = tid; k < kSortWaves * experts; k += kSortThreads) ahead[k] = 0;
    __syncthreads();
    const uint64_t i = r + tid;
    const uint32_t e = i < last ? expert_of(ids, wide, i, experts) : experts;
    const uint64_t same = same_lanes(e, bits, ~0ull);
    const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
    if (e < experts && rank == 0) ahead[wave * experts + e] = (uint16_t)__popcll(same);
    __syncthreads();
    uint32_t to = 0;
    if (e < experts) {
      to = next[e] + rank;
#pragma unroll
      for (uint32_t w = 0; w < kSortWaves; w++) to += w < wave ? ahead[w * experts + e] : 0u;
    }
    if (i < last) {
      place[i] = e < experts ? (int32_t)to : -1;
      if (e < experts) order[to] = (int32_t)i;
    }
    if (r + kSortThreads >= last) break;
    __syncthreads();
    for (uint32_t x = tid; x < experts; x += kSortThreads) {
      uint32_t c = 0;
      for (uint32_t w = 0; w < kSortWaves; w++) c += ahead[w * experts + x];
      next[x] += c;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- rows

constexpr uint32_t kThreads = 256;

__device__ __forceinline__ float weight_at(const void* w, int type, uint64_t i) {
  if (type == EC_TYPE_F32) return ((const float*)w)[i];
  if (type == EC_TYPE_F16) return (float)((const f16_t*)w)[i];
  return (float)((const bf16_t*)w)[i];
}
__device__ __forceinline__ void set_weight(void* w, int type, uint64_t i, float v) {
  if (type == EC_TYPE_F32) ((float*)w)[i] = v;
  else if (type == EC_TYPE_F16) ((f16_t*)w)[i] = (f16_t)v;
  else ((bf16_t*)w)[i] = (bf16_t)v;
}

// Threads of a workgroup: 2^shift lanes along a row of `chunks` pieces of 8
// elements, 256 >> shift tokens.  Wide enough that a lane seldom has more
// than two pieces, and never wider than the row.
struct Shape {
  uint64_t tokens;
  uint32_t cols, chunks, shift, choices;
  uint64_t rows;  // tokens * choices
  bool past;      // stores of 16-bit types go past the caches
};

struct At {
  uint64_t token;
  uint32_t lane, lanes;
};
__device__ __forceinline__ At at(const Shape& s) {
  return {(uint64_t)block_number() * (kThreads >> s.shift) + (threadIdx.x >> s.shift),
          threadIdx.x & ((1u << s.shift) - 1), 1u << s.shift};
}

__device__ __forceinline__ int64_t row_of(const int32_t* place, const Shape& s, uint64_t token,
                                          uint32_t j) {
  const int64_t r = place[token * s.choices + j];
  return r < (int64_t)s.rows ? r : -1;
}

// The first row of no expert.
__device__ __forceinline__ uint64_t no_rows(const int32_t* offsets, uint32_t experts,
                                            uint64_t rows) {
  const int64_t t = offsets[experts];
  return t < 0 ? 0 : (uint64_t)t > rows ? rows : (uint64_t)t;
}

// As many rows belong to no expert as choices were dropped: at most `choices`
// a token, which clears them on the way.
template <typename T>
__device__ __forceinline__ void clear_rows(T* xs, const Shape& s, const At& a, uint64_t none) {
  for (uint64_t r = none + a.token; r < s.rows; r += s.tokens)
    for (uint32_t c = a.lane; c < s.chunks; c += a.lanes)
      store_eight(xs + r * s.cols + c * 8, (int64_t)s.cols - c * 8, Eight<T>{}, s.past);
}

// 16384 tokens, 4 choices, 4096 bf16: 110 us in a loop of its own (6.1 TB/s), 133
// among the other moves, whose lines the caches still write back.
template <typename T>
__global__ __launch_bounds__(kThreads) void expert_dispatch(const T* __restrict__ x, Shape s,
                                                            const int32_t* __restrict__ place,
                                                            const int32_t* __restrict__ offsets,
                                                            uint32_t experts, T* xs) {
  const At a = at(s);
  if (a.token >= s.tokens) return;
  for (uint32_t c = a.lane; c < s.chunks; c += a.lanes) {
    const int64_t n = (int64_t)s.cols - c * 8;
    const Eight<T> v = load_eight(x + a.token * s.cols + c * 8, n);
    for (uint32_t j = 0; j < s.choices; j++) {
      const int64_t r = row_of(place, s, a.token, j);
      if (r >= 0) store_eight(xs + r * s.cols + c * 8, n, v, s.past);
    }
  }
  clear_rows(xs, s, a, no_rows(offsets, experts, s.rows));
}

// chunks covers the padded row here, so that whole quads of lanes work.
template <typename T>
__global__ __launch_bounds__(kThreads) void expert_dispatch_mx(
    const T* __restrict__ x, Shape s, const int32_t* __restrict__ place,
    const int32_t* __restrict__ offsets, uint32_t experts, uint8_t* codes, uint8_t* scales) {
  const At a = at(s);
  if (a.token >= s.tokens) return;
  const uint64_t pitch = s.chunks * 4, spitch = s.chunks / 4;
  for (uint32_t c = a.lane; c < s.chunks; c += a.lanes) {
    const Eight<T> v = load_eight(x + a.token * s.cols + c * 8, (int64_t)s.cols - c * 8);
    const Scale b = scale_of(exponent_of<T>(max_of_4_lanes(magnitude_of_eight(v))));
    const uint32_t code = code_eight(v, b.size);
    for (uint32_t j = 0; j < s.choices; j++) {
      const int64_t r = row_of(place, s, a.token, j);
      if (r < 0) continue;
      *reinterpret_cast<uint32_t*>(codes + r * pitch + c * 4) = code;
      if ((c & 3) == 0) scales[r * spitch + c / 4] = (uint8_t)b.byte;
    }
  }
  for (uint64_t r = no_rows(offsets, experts, s.rows) + a.token; r < s.rows; r += s.tokens)
    for (uint32_t c = a.lane; c < s.chunks; c += a.lanes) {
      *reinterpret_cast<uint32_t*>(codes + r * pitch + c * 4) = 0;
      if ((c & 3) == 0) scales[r * spitch + c / 4] = 0;
    }
}

// y[t] = sum over the choices of w (or 1) times the choice's row, in fp32 and
// in the choices' order.  A lane has PIECES pieces of J rows in flight, and
// places and weights are looked up once for all of them.  16384 tokens, 4
// choices, 4096 bf16: 108 us with weights after a dispatch, 125 without after a
// combine's gradient (6.2 and 5.4 TB/s), 119 and 126 in loops of their own.  With
// one piece instead, both took 6% longer.
template <typename T, bool WEIGHTED, int PIECES>
__global__ __launch_bounds__(kThreads) void expert_gather(const T* __restrict__ ys, Shape s,
                                                          const int32_t* __restrict__ place,
                                                          const void* __restrict__ weights,
                                                          int wtype, T* y) {
  constexpr int J = 4;
  const At a = at(s);
  if (a.token >= s.tokens) return;
  for (uint32_t c0 = a.lane; c0 < s.chunks; c0 += a.lanes * PIECES) {
    float sum[PIECES][8] = {};
    for (uint32_t j0 = 0; j0 < s.choices; j0 += J) {
      int64_t r[J];
      float w[J];
#pragma unroll
      for (int j = 0; j < J; j++)
        r[j] = j0 + j < s.choices ? row_of(place, s, a.token, j0 + j) : -1;
      if (WEIGHTED) {
        const uint64_t at = a.token * s.choices + j0;
#pragma unroll
        for (int j = 0; j < J; j++) {  // a dropped choice's weight may hold anything
          w[j] = weight_at(weights, wtype, at + (j0 + j < s.choices ? j : 0));
          w[j] = r[j] < 0 ? 0.0f : w[j];
        }
      }
      Eight<T> v[PIECES][J];
#pragma unroll
      for (int j = 0; j < J; j++)
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
          const uint32_t c = c0 + i * a.lanes;
          v[i][j] = load_eight(ys + r[j] * s.cols + (uint64_t)c * 8,
                               r[j] >= 0 && c < s.chunks ? (int64_t)s.cols - (int64_t)c * 8 : 0);
        }
#pragma unroll
      for (int i = 0; i < PIECES; i++)
#pragma unroll
        for (int j = 0; j < J; j++) {
          float f[8];
          widen(v[i][j], f);
#pragma unroll
          for (int q = 0; q < 8; q++) sum[i][q] += WEIGHTED ? w[j] * f[q] : f[q];
        }
    }
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      const uint32_t c = c0 + i * a.lanes;
      if (c < s.chunks)
        store_eight(y + a.token * s.cols + (uint64_t)c * 8, (int64_t)s.cols - (int64_t)c * 8,
                    narrow<T>(sum[i]), s.past);
    }
  }
}

// One pass over dy and ys: dys' rows and the products for dweights.  PIECES
// of dy stay in registers while the choices' rows go by, so a row of dy is
// read once where 2^shift lanes hold it (up to 8 PIECES 2^shift elements).
// 16384 tokens, 4 choices, 4096 bf16: 210 us (5.8 TB/s).
template <typename T, int PIECES>
__global__ __launch_bounds__(kThreads) void expert_combine_back(
    const T* __restrict__ dy, const T* __restrict__ ys, Shape s, const int32_t* __restrict__ place,
    const void* __restrict__ weights, int wtype, const int32_t* __restrict__ offsets,
    uint32_t experts, T* dys, void* dweights) {
  __shared__ float part[kThreads / 64];
  const At a = at(s);
  const bool here = a.token < s.tokens;  // a workgroup's last tokens may be past the end
  const uint64_t token = here ? a.token : s.tokens - 1;
  const uint32_t rounds = (s.chunks + a.lanes * PIECES - 1) / (a.lanes * PIECES);
  Eight<T> d[PIECES];
  auto load_dy = [&](uint32_t round) {
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
      const uint32_t c = (round * PIECES + i) * a.lanes + a.lane;
      d[i] = load_eight(dy + token * s.cols + (uint64_t)c * 8,
                        c < s.chunks ? (int64_t)s.cols - (int64_t)c * 8 : 0);
    }
  };
  if (rounds == 1) load_dy(0);
  for (uint32_t j = 0; j < s.choices; j++) {
    const int64_t r = row_of(place, s, token, j);
    const float w = r >= 0 ? weight_at(weights, wtype, token * s.choices + j) : 0.0f;
    float dot = 0;
    if (r >= 0)
      for (uint32_t round = 0; round < rounds; round++) {
        if (rounds > 1) load_dy(round);
        Eight<T> v[PIECES];
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
          const uint32_t c = (round * PIECES + i) * a.lanes + a.lane;
          v[i] = load_eight(ys + r * s.cols + (uint64_t)c * 8,
                            c < s.chunks ? (int64_t)s.cols - (int64_t)c * 8 : 0);
        }
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
          const uint32_t c = (round * PIECES + i) * a.lanes + a.lane;
          float f[8], g[8];
          widen(v[i], f);
          widen(d[i], g);
          float p = 0;
#pragma unroll
          for (int q = 0; q < 8; q++) {
            p += f[q] * g[q];
            g[q] *= w;
          }
          dot += p;
          if (here && c < s.chunks)
            store_eight(dys + r * s.cols + (uint64_t)c * 8, (int64_t)s.cols - (int64_t)c * 8,
                        narrow<T>(g));
        }
      }
    // the token's lanes together: within a wave by exchange, else over LDS
    const uint32_t within = a.lanes < 64 ? a.lanes : 64;
    for (uint32_t m = within / 2; m > 0; m >>= 1) dot += __shfl_xor(dot, m);
    if (a.lanes > 64) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
      __syncthreads();
      const uint32_t waves = a.lanes / 64, w0 = (threadIdx.x >> s.shift) * waves;
      dot = 0;
      for (uint32_t i = 0; i < waves; i++) dot += part[w0 + i];
    }
    if (here && a.lane == 0) set_weight(dweights, wtype, token * s.choices + j, dot);
  }
  if (here) clear_rows(dys, s, a, no_rows(offsets, experts, s.rows));
}

// ---------------------------------------------------------------- host

ec_status launched() { return hipGetLastError() == hipSuccess ? EC_OK : EC_ERR_DEVICE; }

// `pieces`: how many a lane should have before the row takes more lanes
Shape shape_of(uint64_t tokens, uint64_t cols, uint32_t choices, uint32_t chunks,
               uint32_t pieces, bool past) {
  Shape s{};
  s.tokens = tokens, s.cols = (uint32_t)cols, s.choices = choices, s.rows = tokens * choices;
  s.chunks = chunks, s.past = past;
  s.shift = 4;
  while (s.shift < 8 && (pieces << s.shift) < chunks) s.shift++;
  return s;
}
uint64_t blocks_of(const Shape& s) { return ceil_div(s.tokens, kThreads >> s.shift); }

ec_status check(int type, uint64_t tokens, uint64_t cols, uint32_t choices) {
  if (!type_known(type) || cols == 0 || choices == 0) return EC_ERR_INVALID;
  if (choices > EC_EXPERTS_MAX_CHOICES || cols > EC_MX_MAX_DEPTH || tokens > EC_MX_MAX_ROWS ||
      tokens * choices > EC_MX_MAX_ROWS)
    return EC_ERR_UNSUPPORTED;
  return EC_OK;
}
ec_status check_experts(uint32_t experts) {
  return experts == 0 ? EC_ERR_INVALID : experts > EC_EXPERTS_MAX ? EC_ERR_UNSUPPORTED : EC_OK;
}
bool fine(const void* p, size_t to) { return p && aligned(p, to); }

#define BY_TYPE(type, call)                        \
  switch (type) {                                  \
    case EC_TYPE_F32: { using T = float; call; } break;  \
    case EC_TYPE_F16: { using T = f16_t; call; } break;  \
    default: { using T = bf16_t; call; } break;    \
  }

// Parts of the sort: one where a workgroup does it all in two rounds (2048
// choices: 5.9 us, in parts 6.1; 4096: 9.1 and 6.7), else up to 256, so that
// adding up the parts before stays short.
uint32_t sort_parts(uint64_t n) {
  if (n <= 2 * kPart) return 1;
  const uint64_t p = ceil_div(n, kPart);
  return p > 256 ? 256 : (uint32_t)p;
}

}  // namespace

extern "C" {

size_t ec_expert_sort_workspace_bytes(uint64_t n, uint32_t experts) {
  const uint32_t parts = sort_parts(n);
  return parts > 1 ? (size_t)parts * (experts + 1) * 4 : 0;
}

ec_status ec_expert_sort(const void* ids, uint32_t id_bytes, uint64_t n, uint32_t experts,
                         int32_t* order, int32_t* place, int32_t* offsets, void* workspace,
                         size_t workspace_bytes, void* stream) {
  const ec_status st = check_experts(experts);
  if (st != EC_OK) return st;
  if ((id_bytes != 4 && id_bytes != 8) || !fine(offsets, 4)) return EC_ERR_INVALID;
  if (n > EC_MX_MAX_ROWS) return EC_ERR_UNSUPPORTED;
  if (n && (!fine(ids, id_bytes) || !fine(order, 4) || !fine(place, 4))) return EC_ERR_INVALID;
  const size_t need = ec_expert_sort_workspace_bytes(n, experts);
  if (need && !fine(workspace, 4)) return EC_ERR_INVALID;
  if (workspace_bytes < need) return EC_ERR_CAPACITY;
  const uint32_t parts = sort_parts(n);
  const uint32_t per =
      (uint32_t)(ceil_div(ceil_div(n, parts), kSortThreads) * kSortThreads);
  hipStream_t s = (hipStream_t)stream;
  uint32_t* counts = need ? (uint32_t*)workspace : nullptr;
  if (counts)
    hipLaunchKernelGGL(expert_count, dim3(parts), dim3(kSortThreads), 0, s, ids, id_bytes == 8, n,
                       experts, per, counts);
  hipLaunchKernelGGL(expert_place, dim3(parts), dim3(kSortThreads),
                     kSortWaves * experts * sizeof(uint16_t), s, ids, id_bytes == 8, n, experts,
                     per, parts, counts, order, place, offsets);
  return launched();
}

ec_status ec_expert_dispatch(const void* x, int type, uint64_t tokens, uint64_t cols,
                             const int32_t* place, uint32_t choices, const int32_t* offsets,
                             uint32_t experts, void* xs, void* stream) {
  ec_status st = check(type, tokens, cols, choices);
  if (st == EC_OK) st = check_experts(experts);
  if (st != EC_OK || tokens == 0) return st;
  if (!fine(x, type_bytes(type)) || !fine(xs, type_bytes(type)) || !fine(place, 4) ||
      !fine(offsets, 4))
    return EC_ERR_INVALID;
  const uint64_t row = cols * type_bytes(type);
  const Shape s = shape_of(tokens, cols, choices, (uint32_t)ceil_div(cols, 8), 2,
                           past_caches(tokens * choices * row, row));
  BY_TYPE(type, hipLaunchKernelGGL((expert_dispatch<T>), grid_of(blocks_of(s)),
                                   dim3(kThreads), 0, (hipStream_t)stream, (const T*)x, s, place,
                                   offsets, experts, (T*)xs));
  return launched();
}

ec_status ec_expert_dispatch_mx(const void* x, int type, uint64_t tokens, uint64_t cols,
                                const int32_t* place, uint32_t choices, const int32_t* offsets,
                                uint32_t experts, void* codes, void* scales, void* stream) {
  ec_status st = check(type, tokens, cols, choices);
  if (st == EC_OK) st = check_experts(experts);
  if (st != EC_OK || tokens == 0) return st;
  if (!fine(x, type_bytes(type)) || !written_ok(codes, scales) || !fine(place, 4) ||
      !fine(offsets, 4))
    return EC_ERR_INVALID;
  const Shape s = shape_of(tokens, cols, choices, (uint32_t)(ec_mx_padded(cols) / 8), 2,
                           false);
  BY_TYPE(type, hipLaunchKernelGGL((expert_dispatch_mx<T>), grid_of(blocks_of(s)),
                                   dim3(kThreads), 0, (hipStream_t)stream, (const T*)x, s, place,
                                   offsets, experts, (uint8_t*)codes, (uint8_t*)scales));
  return launched();
}

ec_status ec_expert_dispatch_backward(const void* dxs, int type, uint64_t tokens, uint64_t cols,
                                      const int32_t* place, uint32_t choices, void* dx,
                                      void* stream) {
  const ec_status st = check(type, tokens, cols, choices);
  if (st != EC_OK || tokens == 0) return st;
  if (!fine(dxs, type_bytes(type)) || !fine(dx, type_bytes(type)) || !fine(place, 4))
    return EC_ERR_INVALID;
  const uint64_t row = cols * type_bytes(type);
  const Shape s = shape_of(tokens, cols, choices, (uint32_t)ceil_div(cols, 8), 2,
                           past_caches(tokens * row, row));
  BY_TYPE(type, hipLaunchKernelGGL((expert_gather<T, false, 2>), grid_of(blocks_of(s)),
                                   dim3(kThreads), 0, (hipStream_t)stream, (const T*)dxs, s, place,
                                   (const void*)nullptr, 0, (T*)dx));
  return launched();
}

ec_status ec_expert_combine(const void* ys, int type, uint64_t tokens, uint64_t cols,
                            const int32_t* place, uint32_t choices, const void* weights,
                            int wtype, void* y, void* stream) {
  const ec_status st = check(type, tokens, cols, choices);
  if (st != EC_OK) return st;
  if (!type_known(wtype)) return EC_ERR_INVALID;
  if (tokens == 0) return EC_OK;
  if (!fine(ys, type_bytes(type)) || !fine(y, type_bytes(type)) || !fine(place, 4) ||
      !fine(weights, type_bytes(wtype)))
    return EC_ERR_INVALID;
  const uint64_t row = cols * type_bytes(type);
  const Shape s = shape_of(tokens, cols, choices, (uint32_t)ceil_div(cols, 8), 2,
                           past_caches(tokens * row, row));
  BY_TYPE(type, hipLaunchKernelGGL((expert_gather<T, true, 2>), grid_of(blocks_of(s)),
                                   dim3(kThreads), 0, (hipStream_t)stream, (const T*)ys, s, place,
                                   weights, wtype, (T*)y));
  return launched();
}

ec_status ec_expert_combine_backward(const void* dy, const void* ys, int type, uint64_t tokens,
                                     uint64_t cols, const int32_t* place, uint32_t choices,
                                     const void* weights, int wtype, const int32_t* offsets,
                                     uint32_t experts, void* dys, void* dweights, void* stream) {
  ec_status st = check(type, tokens, cols, choices);
  if (st == EC_OK) st = check_experts(experts);
  if (st != EC_OK) return st;
  if (!type_known(wtype)) return EC_ERR_INVALID;
  if (tokens == 0) return EC_OK;
  const size_t b = type_bytes(type), wb = type_bytes(wtype);
  if (!fine(dy, b) || !fine(ys, b) || !fine(dys, b) || !fine(place, 4) || !fine(offsets, 4) ||
      !fine(weights, wb) || !fine(dweights, wb))
    return EC_ERR_INVALID;
  // (stored past the caches dys of 256 MiB to 2 GiB took 2 to 4% longer)
  const Shape s = shape_of(tokens, cols, choices, (uint32_t)ceil_div(cols, 8), 2, false);
  BY_TYPE(type, hipLaunchKernelGGL((expert_combine_back<T, 2>), grid_of(blocks_of(s)),
                                   dim3(kThreads), 0, (hipStream_t)stream, (const T*)dy,
                                   (const T*)ys, s, place, weights, wtype, offsets, experts,
                                   (T*)dys, dweights));
  return launched();
}

}  // extern "C"
