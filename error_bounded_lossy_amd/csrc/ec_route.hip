// Routing of tokens to experts (include/ec_experts.h): which experts a token
// takes, their weights, and the gradient of the logits.
#include <cmath>

#include "ec_experts.h"
#include "ec_mx_device.h"

using namespace ecmx;

namespace {

constexpr uint32_t kThreads = 256;

// A token has 2^shift lanes, a lane KEYS experts.  The lanes are divided among
// the groups, 2^lane_shift each: lane l's expert i is number (l within its
// group) * KEYS + i of group l >> lane_shift, so experts rise with lanes, and a
// group's experts lie in a run of lanes.
struct Layout {
  uint64_t tokens, stride;
  uint32_t experts, groups, size;  // size: experts of a group
  uint32_t shift, lane_shift;
  uint32_t choices, top_groups;
  float scale;
  bool sigmoid, renormalize;
};

struct Here {
  uint64_t token;
  uint32_t lane, lanes, group, first;  // first: number of the lane's expert 0 in its group
  bool valid;                          // the token exists
};
template <int KEYS>
__device__ __forceinline__ Here here_of(const Layout& s) {
  Here a;
  a.lanes = 1u << s.shift;
  a.lane = threadIdx.x & (a.lanes - 1);
  a.token = (uint64_t)block_number() * (kThreads >> s.shift) + (threadIdx.x >> s.shift);
  a.valid = a.token < s.tokens;
  a.group = a.lane >> s.lane_shift;
  a.first = (a.lane & ((1u << s.lane_shift) - 1)) * KEYS;
  return a;
}

// Whether expert i of the lane exists, and its number.
__device__ __forceinline__ bool exists(const Layout& s, const Here& a, int i) {
  return a.group < s.groups && a.first + i < s.size;
}
__device__ __forceinline__ uint32_t expert_at(const Layout& s, const Here& a, int i) {
  return a.group * s.size + a.first + i;
}

template <typename V>
__device__ __forceinline__ V sum_of(V v, uint32_t lanes) {
  for (uint32_t m = lanes / 2; m > 0; m >>= 1) v += (V)__shfl_xor(v, m);
  return v;
}
template <typename V>
__device__ __forceinline__ V max_of(V v, uint32_t lanes) {
  for (uint32_t m = lanes / 2; m > 0; m >>= 1) {
    const V t = __shfl_xor(v, m);
    v = t > v ? t : v;
  }
  return v;
}

// Patterns that order as the numbers do, above 0; NaN above all, both zeros alike.
__device__ __forceinline__ uint32_t ordered(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = bits_as<uint32_t>(v + 0.0f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double v) {
  if (v != v) return ~0ull;
  const uint64_t b = bits_as<uint64_t>(v + 0.0);
  return b >> 63 ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ double sigmoid_of(double l) { return 1.0 / (1.0 + exp(-l)); }

// The lanes of this token among the wave's.
__device__ __forceinline__ uint64_t token_lanes(uint32_t lanes) {
  const uint64_t all = lanes == 64 ? ~0ull : (1ull << lanes) - 1;
  return all << (threadIdx.x & 63 & ~(lanes - 1));
}

// The largest logit of a row (0 where none is open) and the sum of e^(l - top); a
// row with nothing open has sum 1, so that 0 / sum is 0.
template <int KEYS>
__device__ __forceinline__ void softmax_of(const float (&l)[KEYS], uint32_t lanes, double& top,
                                           double& total) {
  float m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < KEYS; i++) {
    m = l[i] > m ? l[i] : m;
    nan |= l[i] != l[i];
  }
  m = max_of(m, lanes);
  top = m > -INFINITY ? (double)m : 0.0;
  total = nan ? NAN : 0.0;
#pragma unroll
  for (int i = 0; i < KEYS; i++) total += exp((double)l[i] - top);
  total = sum_of(total, lanes);
  total = total == 0 ? 1.0 : total;
}

// The weights of a token's choices, choice j in lane j, from their logits (`here`:
// the choice has an expert).  Softmax of the chosen ones alone where weights are
// renormalised; sigmoids so small that their sum has no digits go by e^l.
struct Chosen {
  double weight, opposite;  // without the factor; 1 - sigmoid of the logit
};
__device__ __forceinline__ Chosen chosen_of(const Layout& s, uint32_t lanes, bool here, double l,
                                            double top, double total) {
  const double opposite = s.sigmoid ? sigmoid_of(-l) : 1.0;
  if (!s.renormalize) {
    if (!here) return {0, 0};
    return {s.sigmoid ? sigmoid_of(l) : exp(l - top) / total, opposite};
  }
  const double best = max_of(here ? l : -(double)INFINITY, lanes);
  const bool digits = s.sigmoid && best > -600.0;
  const double e = here ? (digits ? sigmoid_of(l) : exp(l - best)) : 0.0;
  const double sum = sum_of(e, lanes);
  return here ? Chosen{e / sum, opposite} : Chosen{0, 0};
}

// KEY: uint32_t where experts go by their logits, uint64_t by score and bias.
template <typename T, int KEYS, typename KEY>
__global__ __launch_bounds__(kThreads) void expert_route(const T* __restrict__ logits, Layout s,
                                                         const float* __restrict__ bias,
                                                         int32_t* ids, float* weights) {
  const Here a = here_of<KEYS>(s);
  const T* row = logits + (a.valid ? a.token : s.tokens - 1) * s.stride;
  float l[KEYS];
#pragma unroll
  for (int i = 0; i < KEYS; i++)
    l[i] = exists(s, a, i) ? (float)row[expert_at(s, a, i)] : -INFINITY;

  // what the softmax needs of the whole row
  double top = 0, total = 1;
  if (!s.sigmoid && (sizeof(KEY) == 8 || s.groups > 1 || !s.renormalize))
    softmax_of(l, a.lanes, top, total);
  KEY key[KEYS];
  double one = -INFINITY, two = -INFINITY;  // the lane's two best, for the group
#pragma unroll
  for (int i = 0; i < KEYS; i++) {
    const bool open = l[i] != -INFINITY;
    key[i] = open ? (KEY)ordered(l[i]) : 0;
    if (sizeof(KEY) == 8 || s.groups > 1) {
      double v = s.sigmoid ? sigmoid_of(l[i]) : exp((double)l[i] - top) / total;
      if (bias) v += (double)(exists(s, a, i) ? bias[expert_at(s, a, i)] : 0.0f);
      if (sizeof(KEY) == 8) key[i] = open && v != -INFINITY ? (KEY)ordered(v) : 0;
      v = key[i] == 0 ? -INFINITY : v != v ? INFINITY : v;
      two = v > one ? one : v > two ? v : two;
      one = v > one ? v : one;
    }
  }
  if (s.groups > 1) {
    for (uint32_t m = (1u << s.lane_shift) / 2; m > 0; m >>= 1) {
      const double p = __shfl_xor(one, m), q = __shfl_xor(two, m);
      const double least = p < one ? p : one;
      one = p > one ? p : one;
      two = q > two ? q : two;
      two = least > two ? least : two;
    }
    const double score = one + (two > -INFINITY ? two : 0.0);
    // how many groups come before this one
    uint32_t before = 0;
    for (uint32_t g = 0; g < s.groups; g++) {
      const double other = __shfl(score, (int)(g << s.lane_shift), (int)a.lanes);
      before += other > score || (other == score && g < a.group);
    }
    if (before >= s.top_groups)
#pragma unroll
      for (int i = 0; i < KEYS; i++) key[i] = 0;
  }

  // The largest of each lane, then of the token's lanes, `choices` times over.
  const uint64_t mine = token_lanes(a.lanes);
  int32_t id = -1;  // choice j in lane j
  float chosen = 0;
  for (uint32_t j = 0; j < s.choices; j++) {
    KEY best = key[0];
    uint32_t at = 0;
    float value = l[0];
#pragma unroll
    for (int i = 1; i < KEYS; i++)
      if (key[i] > best) best = key[i], at = i, value = l[i];
    const KEY most = max_of(best, a.lanes);
    const uint64_t who = __ballot(best == most) & mine;
    const int from = __builtin_ctzll(who);
    const uint32_t found = __shfl(expert_at(s, a, (int)at), from);
    const float logit = __shfl(value, from);
    if (a.lane == j && most != 0) id = (int32_t)found, chosen = logit;
    if ((threadIdx.x & 63) == (uint32_t)from)
#pragma unroll
      for (int i = 0; i < KEYS; i++) key[i] = at == (uint32_t)i ? 0 : key[i];
  }
  const Chosen c = chosen_of(s, a.lanes, id >= 0, (double)chosen, top, total);
  if (a.valid && a.lane < s.choices) {
    const uint64_t to = a.token * s.choices + a.lane;
    ids[to] = id;
    weights[to] = id >= 0 ? (float)((double)s.scale * c.weight) : 0.0f;
  }
}

// Choice j is in lane j; a token's lanes are at least as many as its choices.
template <typename T, int KEYS>
__global__ __launch_bounds__(kThreads) void expert_route_back(const float* __restrict__ dweights,
                                                              const T* __restrict__ logits,
                                                              Layout s,
                                                              const int32_t* __restrict__ ids,
                                                              T* dlogits) {
  const Here a = here_of<KEYS>(s);
  const uint64_t token = a.valid ? a.token : s.tokens - 1;
  const T* row = logits + token * s.stride;
  const bool whole = !s.sigmoid && !s.renormalize;  // the gradient reaches every logit
  double top = 0, total = 1;
  float l[KEYS] = {};
  if (whole) {
#pragma unroll
    for (int i = 0; i < KEYS; i++)
      l[i] = exists(s, a, i) ? (float)row[expert_at(s, a, i)] : -INFINITY;
    softmax_of(l, a.lanes, top, total);
  }
  int32_t id = -1;
  float chosen = 0, dw = 0;
  if (a.lane < s.choices) {
    const uint64_t at = token * s.choices + a.lane;
    id = ids[at];
    if (id < 0 || (uint32_t)id >= s.experts) id = -1;
    if (id >= 0) {
      chosen = (float)row[id];
      dw = dweights[at];
      if (chosen == -INFINITY) id = -1;
    }
  }
  const bool here = id >= 0;
  const Chosen c = chosen_of(s, a.lanes, here, (double)chosen, top, total);
  const double d = here ? (double)s.scale * (double)dw : 0.0;
  const double mean = sum_of(here ? d * c.weight : 0.0, a.lanes);
  // what this choice's own logit gets; of the whole row the softmax's mean part
  // is taken off below
  double g = 0;
  if (here) g = c.weight * (s.renormalize ? d - mean : d) * c.opposite;
  float out[KEYS];
#pragma unroll
  for (int i = 0; i < KEYS; i++)
    out[i] = whole && exists(s, a, i) ? (float)(-exp((double)l[i] - top) / total * mean) : 0.0f;
  // an expert chosen twice gets both parts, in the choices' order
  for (uint32_t j = 0; j < s.choices; j++) {
    const int32_t e = __shfl(id, (int)j, (int)a.lanes);
    const float v = __shfl((float)g, (int)j, (int)a.lanes);
#pragma unroll
    for (int i = 0; i < KEYS; i++)
      if (e >= 0 && exists(s, a, i) && expert_at(s, a, i) == (uint32_t)e) out[i] += v;
  }
  if (a.valid)
#pragma unroll
    for (int i = 0; i < KEYS; i++)
      if (exists(s, a, i)) dlogits[token * s.experts + expert_at(s, a, i)] = (T)out[i];
}

// ---------------------------------------------------------------- host

ec_status launched() { return hipGetLastError() == hipSuccess ? EC_OK : EC_ERR_DEVICE; }
bool fine(const void* p, size_t to) { return p && aligned(p, to); }

// At least as many lanes as choices; returns the keys of a lane.
uint32_t lay_out(Layout& s) {
  uint32_t most = 0;  // lanes of a group: a power of two, all groups within 64
  while ((s.groups << (most + 1)) <= 64 && (1u << most) < s.size) most++;
  s.lane_shift = most;
  uint32_t need = s.groups << most;
  if (need < s.choices) need = s.choices;
  s.shift = 2;
  while ((1u << s.shift) < need) s.shift++;
  const uint32_t keys = (uint32_t)ceil_div(s.size, 1u << most);
  uint32_t k = 1;
  while (k < keys) k *= 2;
  return k;
}
uint64_t blocks_of(const Layout& s) { return ceil_div(s.tokens, kThreads >> s.shift); }

ec_status check(int type, uint64_t tokens, uint64_t stride, uint32_t experts, uint32_t choices,
                int score, float scale) {
  if (!type_known(type) || experts == 0 || choices == 0 || stride < experts ||
      (score != EC_SCORE_SOFTMAX && score != EC_SCORE_SIGMOID) || !std::isfinite(scale))
    return EC_ERR_INVALID;
  if (experts > EC_EXPERTS_MAX || choices > EC_EXPERTS_MAX_CHOICES || tokens > EC_MX_MAX_ROWS ||
      tokens * choices > EC_MX_MAX_ROWS)
    return EC_ERR_UNSUPPORTED;
  return EC_OK;
}

template <typename T, int KEYS>
ec_status route_as(const void* logits, const Layout& s, const float* bias, int32_t* ids,
                   float* weights, hipStream_t stream) {
  if (bias)
    hipLaunchKernelGGL((expert_route<T, KEYS, uint64_t>), grid_of(blocks_of(s)), dim3(kThreads), 0,
                       stream, (const T*)logits, s, bias, ids, weights);
  else
    hipLaunchKernelGGL((expert_route<T, KEYS, uint32_t>), grid_of(blocks_of(s)), dim3(kThreads), 0,
                       stream, (const T*)logits, s, bias, ids, weights);
  return launched();
}
template <typename T>
ec_status route_of(const void* logits, Layout s, const float* bias, int32_t* ids, float* weights,
                   hipStream_t stream) {
  switch (lay_out(s)) {
    case 1: return route_as<T, 1>(logits, s, bias, ids, weights, stream);
    case 2: return route_as<T, 2>(logits, s, bias, ids, weights, stream);
    case 4: return route_as<T, 4>(logits, s, bias, ids, weights, stream);
    case 8: return route_as<T, 8>(logits, s, bias, ids, weights, stream);
    case 16: return route_as<T, 16>(logits, s, bias, ids, weights, stream);
    default: return route_as<T, 32>(logits, s, bias, ids, weights, stream);
  }
}

template <typename T>
ec_status back_of(const float* dweights, const void* logits, Layout s, const int32_t* ids,
                  void* dlogits, hipStream_t stream) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid_of(blocks_of(s)), dim3(kThreads), 0, stream, dweights,
                       (const T*)logits, s, ids, (T*)dlogits);
  };
  switch (lay_out(s)) {  // one group: 16 keys at most
    case 1: go(expert_route_back<T, 1>); break;
    case 2: go(expert_route_back<T, 2>); break;
    case 4: go(expert_route_back<T, 4>); break;
    case 8: go(expert_route_back<T, 8>); break;
    default: go(expert_route_back<T, 16>);
  }
  return launched();
}

}  // namespace

extern "C" {

ec_status ec_expert_route(const void* logits, int type, uint64_t tokens, uint64_t stride,
                          uint32_t experts, const float* bias, uint32_t choices, int score,
                          uint32_t groups, uint32_t top_groups, int renormalize, float scale,
                          int32_t* ids, float* weights, void* stream) {
  const ec_status st = check(type, tokens, stride, experts, choices, score, scale);
  if (st == EC_ERR_INVALID) return st;
  if (groups == 0 || experts % groups || top_groups == 0 || top_groups > groups ||
      choices > (uint64_t)(experts / groups) * top_groups)
    return EC_ERR_INVALID;
  if (st != EC_OK || groups > EC_EXPERTS_MAX_GROUPS) return EC_ERR_UNSUPPORTED;
  if (tokens == 0) return EC_OK;
  if (!fine(logits, type_bytes(type)) || !aligned(bias, 4) || !fine(ids, 4) || !fine(weights, 4))
    return EC_ERR_INVALID;
  Layout s{};
  s.tokens = tokens, s.stride = stride, s.experts = experts, s.groups = groups;
  s.size = experts / groups, s.choices = choices, s.top_groups = top_groups;
  if (top_groups == groups) s.groups = 1, s.size = experts;  // all of them: no groups
  s.scale = scale, s.sigmoid = score == EC_SCORE_SIGMOID, s.renormalize = renormalize != 0;
  hipStream_t q = (hipStream_t)stream;
  switch (type) {
    case EC_TYPE_F32: return route_of<float>(logits, s, bias, ids, weights, q);
    case EC_TYPE_F16: return route_of<f16_t>(logits, s, bias, ids, weights, q);
    default: return route_of<bf16_t>(logits, s, bias, ids, weights, q);
  }
}

ec_status ec_expert_route_backward(const float* dweights, const void* logits, int type,
                                   uint64_t tokens, uint64_t stride, uint32_t experts,
                                   const int32_t* ids, uint32_t choices, int score,
                                   int renormalize, float scale, void* dlogits, void* stream) {
  const ec_status st = check(type, tokens, stride, experts, choices, score, scale);
  if (st != EC_OK || tokens == 0) return st;
  const size_t b = type_bytes(type);
  if (!fine(dweights, 4) || !fine(logits, b) || !fine(ids, 4) || !fine(dlogits, b))
    return EC_ERR_INVALID;
  Layout s{};
  s.tokens = tokens, s.stride = stride, s.experts = experts, s.groups = 1, s.size = experts;
  s.choices = choices, s.top_groups = 1;
  s.scale = scale, s.sigmoid = score == EC_SCORE_SIGMOID, s.renormalize = renormalize != 0;
  hipStream_t q = (hipStream_t)stream;
  switch (type) {
    case EC_TYPE_F32: return back_of<float>(dweights, logits, s, ids, dlogits, q);
    case EC_TYPE_F16: return back_of<f16_t>(dweights, logits, s, ids, dlogits, q);
    default: return back_of<bf16_t>(dweights, logits, s, ids, dlogits, q);
  }
}

}  // extern "C"
