// Routing of tokens to experts (include/ec_experts.h): which experts a token
// takes, their weights, and the gradient of the logits.
#include <cmath>

#include "ec_experts.h"
#include "ec_lanes_device.h"

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

// Patterns that order as the numbers do, above 0; NaN above all, both zeros alike.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = bits_as<uint32_t>(v + 0.0f);
  return v != v ? 0xffffffffu : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v) {
  if (v != v) return ~0ull;
  const uint64_t b = bits_as<uint64_t>(v + 0.0);
  return b >> 63 ? ~b : b | 1ull << 63;
}
// -infinity and everything below are no numbers to choose.
__device__ __forceinline__ bool is_open(uint32_t key) { return key > 0x007fffffu; }
__device__ __forceinline__ bool is_open(uint64_t key) { return key > 0x000fffffffffffffull; }
__device__ __forceinline__ double number_of(uint64_t o) {
  return bits_as<double>(o >> 63 ? o & ~(1ull << 63) : ~o);
}
__device__ __forceinline__ float number_of(uint32_t o) {
  return bits_as<float>(o >> 31 ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ double sigmoid_of(double l) { return 1.0 / (1.0 + exp(-l)); }

// 64-bit pieces for numbers that are rounded to 32 bits in the end: good to some
// 2^-46 (a reciprocal is the instruction's with two Newton steps, an exponential
// e^r 2^n with |r| <= ln 2 / 2 and r's powers to the eleventh: 6e-15).
__device__ __forceinline__ double quotient_of(double a, double b) {
  double r = __builtin_amdgcn_rcp(b);
  r = __builtin_fma(__builtin_fma(-b, r, 1.0), r, r);
  r = __builtin_fma(__builtin_fma(-b, r, 1.0), r, r);
  return a * r;
}
__device__ __forceinline__ double power_of(double x) {  // e^x, x finite and not over 700
  x = x < -1000.0 ? -1000.0 : x;
  const double n = __builtin_rint(x * 1.4426950408889634);
  // ln 2 in two parts (Cody and Waite): its nearest multiple of 2^-40, whose product
  // with n is exact, and what is left of it
  double r = __builtin_fma(n, -0x1.62e42fefa4p-1, x);
  r = __builtin_fma(n, 0x1.8432a1b0e2634p-43, r);
  double p = 1.0 / 39916800;
  p = __builtin_fma(p, r, 1.0 / 3628800);
  p = __builtin_fma(p, r, 1.0 / 362880);
  p = __builtin_fma(p, r, 1.0 / 40320);
  p = __builtin_fma(p, r, 1.0 / 5040);
  p = __builtin_fma(p, r, 1.0 / 720);
  p = __builtin_fma(p, r, 1.0 / 120);
  p = __builtin_fma(p, r, 1.0 / 24);
  p = __builtin_fma(p, r, 1.0 / 6);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// The lanes of this token among the wave's.
__device__ __forceinline__ uint64_t token_lanes(uint32_t lanes) {
  const uint64_t all = lanes == 64 ? ~0ull : (1ull << lanes) - 1;
  return all << (threadIdx.x & 63 & ~(lanes - 1));
}

// The largest logit of a row (0 where none is open) and the sum of e^(l - top),
// whose terms are left in `e`; a row with nothing open has sum 1, so that 0 / sum
// is 0.
template <int KEYS>
__device__ __forceinline__ void softmax_of(const float (&l)[KEYS], uint32_t shift, double& top,
                                           double& total, double (&e)[KEYS]) {
  float m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < KEYS; i++) {
    m = l[i] > m ? l[i] : m;
    nan |= l[i] != l[i];
  }
  m = max_of(m, shift);
  top = m > -INFINITY ? (double)m : 0.0;
  total = nan ? NAN : 0.0;
#pragma unroll
  for (int i = 0; i < KEYS; i++) total += e[i] = exp((double)l[i] - top);
  total = sum_of(total, shift);
  total = total == 0 ? 1.0 : total;
}

// The weights of a token's choices, choice j in lane j, from their logits (`here`:
// the choice has an expert).  Softmax of the chosen ones alone where weights are
// renormalised; sigmoids so small that their sum has no digits go by e^l.
struct Chosen {
  double weight, opposite;  // without the factor; 1 - sigmoid of the logit
};
__device__ __forceinline__ Chosen chosen_of(const Layout& s, uint32_t shift, bool here, float l,
                                            double top, double total) {
  // e^-|l|, 1 / (1 + e^-|l|) and e^-|l| / (1 + e^-|l|): a sigmoid and its opposite
  double score = 0, opposite = 1;
  if (s.sigmoid) {
    const double e = power_of(-__builtin_fabs((double)l)), r = quotient_of(1.0, 1.0 + e);
    score = l >= 0 ? r : e * r;
    opposite = l >= 0 ? e * r : r;
    if (l != l) score = opposite = (double)l;
  }
  if (!s.renormalize) {
    if (!here) return {0, 0};
    if (!s.sigmoid) score = l != l ? (double)l : quotient_of(power_of((double)l - top), total);
    return {score, opposite};
  }
  const float best = max_of(here ? l : -INFINITY, shift);
  if (!s.sigmoid || !(best > -600.0f)) {
    const double x = (double)l - (double)best;
    score = x != x ? x : power_of(x);
  }
  if (!here) score = 0;
  const double sum = sum_of(score, shift);
  return here ? Chosen{quotient_of(score, sum), opposite} : Chosen{0, 0};
}

// The lane's part of a row of logits, or of biases.
template <typename T, int KEYS>
__device__ __forceinline__ void load_part(const T* row, const Layout& s, const Here& a,
                                          float none, float (&l)[KEYS]) {
  const T* from = row + expert_at(s, a, 0);
  if (a.group < s.groups && a.first + KEYS <= s.size) {
    T v[KEYS];
    __builtin_memcpy(v, from, sizeof(v));
#pragma unroll
    for (int i = 0; i < KEYS; i++) l[i] = (float)v[i];
  } else {
#pragma unroll
    for (int i = 0; i < KEYS; i++) l[i] = exists(s, a, i) ? (float)from[i] : none;
  }
}

// ---------------------------------------------------------------- forward

// Scores in 32 bits are off by less than these: a sigmoid, 1 / (1 + 2^(-l log2 e)),
// by 2.3e-7 (the exponent by |l| 1.3e-7, which |l| s (1 - s) <= 0.224 bounds, the
// instructions by one unit each), a softmax by 3.2e-6 of its largest score (the
// sum's terms the most).  Numbers that are less apart than what both are off by
// are put in order in 64 bits.
constexpr float kSigmoidOff = 1e-6f, kSoftmaxOff = 1.3e-5f;

// Whether b, which comes after a, may belong before it: the bias' addition and the
// places in the lowest bits (`keys` units of each) are relative.  NaN and
// infinities may.
constexpr float kBiasOff = 1e-6f;
__device__ __forceinline__ bool near(float a, float b, float off, int keys) {
  const float size = __builtin_fmaxf(__builtin_fabsf(a), __builtin_fabsf(b));
  return !(a - b > off + (kBiasOff + (float)keys * 0x1p-22f) * size);
}

// Two best keys of a run of 2^shift lanes, from each lane's.
template <typename K>
__device__ __forceinline__ void best_two(K& one, K& two, uint32_t shift) {
  auto join = [&](K p, K q) {
    const K least = p < one ? p : one;
    one = p > one ? p : one;
    two = q > two ? q : two;
    two = least > two ? least : two;
  };
  using std::integral_constant;
  if (shift > 0) join(moved(one, integral_constant<int, 0xb1>{}), moved(two, integral_constant<int, 0xb1>{}));
  if (shift > 1) join(moved(one, integral_constant<int, 0x4e>{}), moved(two, integral_constant<int, 0x4e>{}));
  if (shift > 2) join(moved(one, integral_constant<int, 0x141>{}), moved(two, integral_constant<int, 0x141>{}));
  if (shift > 3) join(moved(one, integral_constant<int, 0x140>{}), moved(two, integral_constant<int, 0x140>{}));
  if (shift > 4) join((K)__shfl_xor(one, 16), (K)__shfl_xor(two, 16));
}

// Whether the lane's group is one that is chosen, by each group's two best, whose
// scores are value(key) (a NaN counts as infinity).  `unsure`: one that is and one
// that is not are nearer than what their sums are off by, which goes by the two
// best's sizes: with biases of both signs the sum may be far smaller.
template <bool WAVE, typename V, typename KEY, int KEYS, typename F>
__device__ __forceinline__ bool in_chosen_group(const Layout& s, const Here& a, uint32_t shift,
                                                const KEY (&key)[KEYS], float off, F&& value,
                                                bool& unsure) {
  KEY one = 0, two = 0;
#pragma unroll
  for (int i = 0; i < KEYS; i++) {
    const KEY least = key[i] < one ? key[i] : one;
    one = key[i] > one ? key[i] : one;
    two = least > two ? least : two;
  }
  best_two(one, two, s.lane_shift);
  auto score_of = [&](KEY k) {
    const V v = value(k);
    return v != v ? (V)INFINITY : v;
  };
  const V first = is_open(one) ? score_of(one) : (V)-INFINITY;
  const V second = is_open(two) ? score_of(two) : (V)0, score = first + second;
  uint32_t before = 0;  // groups that come before this one
  for (uint32_t g = 0; g < s.groups; g++) {
    V other;
    if constexpr (WAVE && sizeof(V) == 4)
      other = bits_as<float>(lane_value(bits_as<uint32_t>(score), (int)(g << s.lane_shift)));
    else
      other = __shfl(score, (int)(g << s.lane_shift), (int)a.lanes);
    before += other > score || (other == score && g < a.group);
  }
  const bool kept = before < s.top_groups;
  if constexpr (sizeof(V) == 4) {
    // (where a sum is infinite, also one too large for 32 bits, there is nothing to compare)
    const float by = off + 0.5f * kBiasOff * (__builtin_fabsf(first) + __builtin_fabsf(second));
    const bool any = is_open(one);
    const float least = -max_of(any && kept ? by - score : -INFINITY, shift);
    const float most = max_of(any && !kept ? score + by : -INFINITY, shift);
    unsure |= any && !(by < INFINITY);
    unsure |= most > -INFINITY && !(least > most);
  }
  return kept;
}

// A lane's keys in descending order (Batcher's odd-even merge).
template <int N>
__device__ __forceinline__ void sorted(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; i++)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t x = v[i + j], y = v[i + j + k];
            v[i + j] = x > y ? x : y;
            v[i + j + k] = x > y ? y : x;
          }
}

// How sure the order of 32-bit keys is.
enum Sure {
  kSure,    // it is: the keys are exact
  kPlaced,  // but where they agree in all bits that a place does not take
  kRounded  // but where they are nearer than what they are off by
};

// The largest of 32-bit keys, `choices` times over: every lane sorts its own, with
// their places in the lowest bits (comparisons of one word cost two instructions,
// of a word and a place six), then the lanes' first ones are compared and the
// winner's next moves up.  Ties: the lowest lane and in it the lowest place, which
// is the lowest expert.
//
// Where neighbours, or the first one left out, may be in another order, those
// that follow are taken too while they are as near, and all of them are put in
// order by exact(expert), their keys in 64 bits.  (All experts again in 64 bits
// made such waves, a few in a hundred, twice as long, and the kernel with them.)
// `failed`: there are more such ones than lanes.
template <Sure SURE, bool WAVE, int KEYS, typename F>
__device__ __forceinline__ int32_t select(const Layout& s, const Here& a, uint32_t shift,
                                          const uint32_t (&key)[KEYS], bool kept, float off,
                                          F&& exact, bool& failed) {
  constexpr uint32_t kPlace = KEYS - 1;
  const uint32_t mask = kept ? ~kPlace : 0;
  uint32_t list[KEYS];
#pragma unroll
  for (int i = 0; i < KEYS; i++) list[i] = (key[i] & mask) | (kPlace - i);
  sorted(list);
  uint32_t chosen = 0, taken = 0;  // choice j in lane j: its number among the keys, its key
  auto most_now = [&] {
    const uint32_t most = max_of(list[0], shift) | kPlace;
    return WAVE ? __builtin_amdgcn_readfirstlane(most) : most;
  };
  auto take = [&](uint32_t j, uint32_t most, bool really) {
    uint32_t number;
    if constexpr (WAVE) {  // the same for all lanes
      const uint32_t lane = (uint32_t)__builtin_ctzll(__ballot((list[0] | kPlace) == most));
      number = lane * KEYS + (kPlace - (lane_value(list[0], (int)lane) & kPlace));
    } else {
      number = (list[0] | kPlace) == most ? a.lane * KEYS + (kPlace - (list[0] & kPlace)) : ~0u;
      number = over_lanes(number, shift, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
    }
    const bool set = a.lane == j && really;
    chosen = set ? number : chosen;
    taken = set ? most : taken;
    // (bits, not a choice of two elements, which the compiler makes an index of)
    const uint32_t win = a.lane == number / KEYS && really ? ~0u : 0u;
#pragma unroll
    for (int i = 0; i < KEYS; i++)
      list[i] = (i + 1 < KEYS ? list[i + 1] & win : 0) | (list[i] & ~win);
  };
  auto expert = [&] {
    const uint32_t lane = chosen / KEYS, in_group = lane & ((1u << s.lane_shift) - 1);
    return (lane >> s.lane_shift) * s.size + in_group * KEYS + chosen % KEYS;
  };
  for (uint32_t j = 0; j < s.choices; j++) take(j, most_now(), true);
  if constexpr (SURE != kSure) {
    auto close = [&](uint32_t x, uint32_t y) {
      if (SURE == kPlaced) return x == y;
      return near(number_of(x), number_of(y), off, KEYS);
    };
    uint32_t next = most_now();
    const uint32_t after = __shfl_down(taken, 1);
    bool unsure = false;
    {
      const uint32_t other = a.lane + 1 < s.choices ? after : next;
      unsure = a.lane < s.choices && is_open(other) && close(taken, other);
    }
    if (__any(unsure)) {
      uint32_t count = s.choices;  // of this token
      uint32_t last = __shfl(taken, (int)count - 1, (int)a.lanes);
      for (;;) {
        const bool more = is_open(next) && close(last, next);
        if (!__any(more)) break;
        failed |= more && count == a.lanes;
        if (__any(failed)) return -1;
        take(count, next, more);
        count += more;
        last = more ? next : last;
        next = most_now();
      }
      const int32_t mine = (int32_t)expert();
      const bool candidate = a.lane < count && is_open(taken);
      const uint64_t found = ordered(exact(candidate ? (uint32_t)mine : 0));  // by all lanes
      const uint64_t value = candidate ? found : 0;
      const uint32_t most = max_of(count, 6);
      uint32_t rank = 0;
      for (uint32_t i = 0; i < most; i++) {
        const uint64_t v = __shfl(value, (int)i, (int)a.lanes);
        const int32_t e = __shfl(mine, (int)i, (int)a.lanes);
        rank += i < count && (v > value || (v == value && e < mine && v != 0));
      }
      rank = candidate ? rank : 64 + a.lane;
      int32_t id = -1;
      for (uint32_t i = 0; i < most; i++) {
        const uint32_t r = __shfl(rank, (int)i, (int)a.lanes);
        const int32_t e = __shfl(mine, (int)i, (int)a.lanes);
        id = r == a.lane ? e : id;
      }
      return a.lane < s.choices ? id : -1;
    }
  }
  return is_open(taken) ? (int32_t)expert() : -1;
}

// The same of 64-bit keys.
template <int KEYS>
__device__ __forceinline__ int32_t select_exact(const Layout& s, const Here& a, uint32_t shift,
                                                uint64_t (&key)[KEYS]) {
  const uint64_t mine = token_lanes(a.lanes);
  int32_t id = -1;
  for (uint32_t j = 0; j < s.choices; j++) {
    uint64_t best = key[0];
    uint32_t at = 0;
#pragma unroll
    for (int i = 1; i < KEYS; i++)
      if (key[i] > best) best = key[i], at = i;
    const uint64_t most = max_of(best, shift);
    const uint64_t who = __ballot(best == most) & mine;
    const int from = __builtin_ctzll(who);
    const uint32_t e = __shfl(expert_at(s, a, (int)at), from);
    if (a.lane == j && is_open(most)) id = (int32_t)e;
    if ((threadIdx.x & 63) == (uint32_t)from)
#pragma unroll
      for (int i = 0; i < KEYS; i++) key[i] = at == (uint32_t)i ? 0 : key[i];
  }
  return id;
}

// Everything in 64 bits.
template <int KEYS>
__device__ int32_t route_exact(const Layout& s, const Here& a, uint32_t shift,
                               const float (&l)[KEYS], const float (&b)[KEYS], bool biased) {
  double top = 0, total = 1, v[KEYS];
  if (!s.sigmoid) softmax_of(l, shift, top, total, v);
  uint64_t key[KEYS];
#pragma unroll
  for (int i = 0; i < KEYS; i++) {
    v[i] = (s.sigmoid ? sigmoid_of(l[i]) : v[i] / total) + (double)b[i];
    key[i] = l[i] == -INFINITY ? 0 : ordered(v[i]);
  }
  bool kept = true, sure;
  if (s.groups > 1)
    kept = in_chosen_group<false, double>(s, a, shift, key, 0, [](uint64_t k) { return number_of(k); },
                                          sure);
#pragma unroll
  for (int i = 0; i < KEYS; i++)
    if (!kept) key[i] = 0;
    else if (!biased) key[i] = ordered((double)l[i]);
  return select_exact(s, a, shift, key);
}

// What bounds it is vector instructions, and where tokens are few their latency:
// 16384 x 256, 8 choices, bias and groups, has 880 a wave of two tokens and takes 19 to
// 21 us (13 of issue); 32 tokens take 5.5 us.  So a lane's keys are 32 bits.  Where experts go
// by score and bias, that is decided in 32 bits, and in 64 where two numbers are too
// near.  (64-bit keys throughout: 1127 instructions a token, 44 us.)
template <typename T, int KEYS, bool BIAS, bool WAVE>
__global__ __launch_bounds__(kThreads) void expert_route(const T* __restrict__ logits, Layout s,
                                                         const float* __restrict__ bias,
                                                         int32_t* ids, float* weights) {
  const Here a = here_of<KEYS>(s);
  const uint32_t shift = WAVE ? 6 : s.shift;
  const T* row = logits + (a.valid ? a.token : s.tokens - 1) * s.stride;
  float l[KEYS], b[KEYS] = {};
  load_part(row, s, a, -INFINITY, l);
  if (BIAS) load_part(bias, s, a, 0.0f, b);

  constexpr float kLog2e = 1.44269504f;
  float off = kSigmoidOff, top32 = 0, by = 1;
  if ((BIAS || s.groups > 1) && !s.sigmoid) {
    float m = -INFINITY, sum = 0;
#pragma unroll
    for (int i = 0; i < KEYS; i++) m = l[i] > m ? l[i] : m;
    m = max_of(m, shift);
    top32 = m > -INFINITY ? m : 0;
#pragma unroll
    for (int i = 0; i < KEYS; i++) sum += __builtin_amdgcn_exp2f((l[i] - top32) * kLog2e);
    by = __builtin_amdgcn_rcpf(sum_of(sum, shift));
    off = kSoftmaxOff * by;
  }
  auto score = [&](float v) {
    return s.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e))
                     : __builtin_amdgcn_exp2f((v - top32) * kLog2e) * by;
  };
  uint32_t key[KEYS];
#pragma unroll
  for (int i = 0; i < KEYS; i++)
    key[i] = ordered(!BIAS ? l[i] : l[i] == -INFINITY ? -INFINITY : score(l[i]) + b[i]);
  bool kept = true, unsure = false;
  if (s.groups > 1)
    kept = in_chosen_group<WAVE, float>(
        s, a, shift, key, off,
        [&](uint32_t k) { return BIAS ? number_of(k) : score(number_of(k)); }, unsure);
  // (a 16-bit logit leaves the lowest bits of its pattern to the place)
  constexpr Sure kHow = BIAS ? kRounded : sizeof(T) == 4 && KEYS > 1 ? kPlaced : kSure;
  int32_t id = select<kHow, WAVE>(
      s, a, shift, key, kept, off,
      [&](uint32_t e) {
        const double logit = (double)(float)row[e];
        if (!BIAS) return logit;
        double top = 0, total = 1;
        if (!s.sigmoid) {
          double terms[KEYS];
          softmax_of(l, shift, top, total, terms);
        }
        return (s.sigmoid ? sigmoid_of(logit) : exp(logit - top) / total) + (double)bias[e];
      },
      unsure);
  if (__any(unsure)) id = route_exact(s, a, shift, l, b, BIAS);

  double top = 0, total = 1;
  if (!s.sigmoid && !s.renormalize) {
    double e[KEYS];
    softmax_of(l, shift, top, total, e);
  }
  const float mine = id >= 0 ? (float)row[id] : 0.0f;
  const Chosen c = chosen_of(s, shift, id >= 0, mine, top, total);
  if (a.valid && a.lane < s.choices) {
    const uint64_t to = a.token * s.choices + a.lane;
    ids[to] = id;
    weights[to] = id >= 0 ? (float)((double)s.scale * c.weight) : 0.0f;
  }
}

// ---------------------------------------------------------------- backward

// A choice as the forward pass left it: choice j is in lane j.
struct Choice {
  int32_t id;  // -1: takes no part
  float logit, dw;
};
template <typename T>
__device__ __forceinline__ Choice choice_at(const Layout& s, const T* row, const int32_t* ids,
                                            const float* dweights, uint64_t token, uint32_t lane) {
  Choice c{-1, 0, 0};
  if (lane < s.choices) {
    const uint64_t at = token * s.choices + lane;
    c.id = ids[at];
    if (c.id < 0 || (uint32_t)c.id >= s.experts) c.id = -1;
    if (c.id >= 0) {
      c.logit = (float)row[c.id];
      c.dw = dweights[at];
      if (c.logit == -INFINITY) c.id = -1;
    }
  }
  return c;
}

template <typename T, int N>
__device__ __forceinline__ void store_logits(T* to, int64_t n, const float (&f)[N]) {
  T v[N];
#pragma unroll
  for (int i = 0; i < N; i++) v[i] = (T)f[i];
  if (n >= N) {
    __builtin_memcpy(to, v, sizeof(v));
  } else {
#pragma unroll
    for (int i = 0; i < N; i++)
      if (i < n) to[i] = v[i];
  }
}

// Where only the chosen logits have a gradient: 2^shift lanes a token (as many as
// it has choices) compute theirs, then the wave writes its tokens' rows by way of
// a row of LDS that is zero but for the chosen ones.  (Comparing every expert's
// number with every choice instead took 11 us for 16384 x 256 fp32, 8 choices; this
// takes 8.1 to 8.9, 3.3 of them for the stores: a wave's tokens leave one by one.)
template <typename T>
__global__ __launch_bounds__(kThreads) void expert_route_back(const float* __restrict__ dweights,
                                                              const T* __restrict__ logits,
                                                              Layout s,
                                                              const int32_t* __restrict__ ids,
                                                              T* dlogits) {
  extern __shared__ __attribute__((aligned(16))) float rows[];
  constexpr uint32_t E = 16 / sizeof(T);  // elements of a piece
  const uint32_t lane = threadIdx.x & 63, padded = (s.experts + E - 1) / E * E;
  float* mine = rows + (threadIdx.x >> 6) * padded;
  for (uint32_t e = lane; e < padded; e += 64) mine[e] = 0;
  const Here a = here_of<1>(s);
  const uint64_t token = a.valid ? a.token : s.tokens - 1;
  const Choice m = choice_at(s, logits + token * s.stride, ids, dweights, token, a.lane);
  const bool here = m.id >= 0;
  const Chosen c = chosen_of(s, s.shift, here, m.logit, 0, 1);
  const double d = here ? (double)s.scale * (double)m.dw : 0.0;
  // Of renormalised weights w, whose sum is 1, d - sum of w d is the sum of w_j (d - d_j):
  // so it keeps its digits where a weight is nearly 1.
  double from = d;
  if (s.renormalize) {
    from = 0;
    for (uint32_t j = 0; j < s.choices; j++)
      from += __shfl(c.weight, (int)j, (int)a.lanes) * (d - __shfl(d, (int)j, (int)a.lanes));
  }
  const double g = here ? c.weight * from * c.opposite : 0.0;
  // an expert chosen twice gets both parts, in the choices' order, from each
  double all = 0;
  for (uint32_t j = 0; j < s.choices; j++) {
    const int32_t id = __shfl(m.id, (int)j, (int)a.lanes);
    const double v = __shfl(g, (int)j, (int)a.lanes);
    all += id == m.id ? v : 0.0;
  }
  const uint64_t first = a.token - (lane >> s.shift);
  auto together = [] {
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  for (uint32_t t = 0; t < 64u >> s.shift; t++) {
    if (first + t >= s.tokens) return;
    const bool now = here && lane >> s.shift == t;
    if (now) mine[m.id] = (float)all;
    together();
    T* to = dlogits + (first + t) * s.experts;
    for (uint32_t e0 = lane * E; e0 < s.experts; e0 += 64 * E) {
      float out[E];
      __builtin_memcpy(out, __builtin_assume_aligned(mine + e0, 16), sizeof(out));
      store_logits(to + e0, (int64_t)s.experts - e0, out);
    }
    together();
    if (now) mine[m.id] = 0;
  }
}

// A softmax over all whose weights stay as they are: the gradient reaches every
// logit.  8190 x 60 bf16, 4 choices: 7.8 us, of vector instructions (350 a token,
// which has a wave; most for the exponentials in 64 bits).
template <typename T, int KEYS, bool WAVE>
__global__ __launch_bounds__(kThreads) void expert_softmax_back(
    const float* __restrict__ dweights, const T* __restrict__ logits, Layout s,
    const int32_t* __restrict__ ids, T* dlogits) {
  const Here a = here_of<KEYS>(s);
  const uint32_t shift = WAVE ? 6 : s.shift;
  const uint64_t token = a.valid ? a.token : s.tokens - 1;
  const T* row = logits + token * s.stride;
  float l[KEYS];
  double top, total, e[KEYS];
  load_part(row, s, a, -INFINITY, l);
  softmax_of(l, shift, top, total, e);
  const Choice m = choice_at(s, row, ids, dweights, token, a.lane);
  const Chosen c = chosen_of(s, shift, m.id >= 0, m.logit, top, total);
  // choice j's value (where it has the whole wave, without the way through LDS)
  auto of = [&](auto v, uint32_t j) {
    if constexpr (!WAVE) return __shfl(v, (int)j, (int)a.lanes);
    else if constexpr (sizeof(v) == 4) return bits_as<decltype(v)>(lane_value(bits_as<uint32_t>(v), (int)j));
    else {
      const uint64_t w = bits_as<uint64_t>(v);
      return bits_as<decltype(v)>((uint64_t)lane_value((uint32_t)(w >> 32), (int)j) << 32 |
                                  lane_value((uint32_t)w, (int)j));
    }
  };
  // p (ds - sum of p ds), with the scores p and their gradients ds, is the sum of
  // p p_k (ds - ds_k) over all experts: so it keeps its digits where a score is nearly
  // 1.  What an expert gets that is chosen more than once is added up, in each of its
  // choices, and its score counts in the first.
  double d = 0;
  bool again = false;
  uint32_t taken = 0;  // of the lane's experts, as bits
  for (uint32_t j = 0; j < s.choices; j++) {
    const int32_t id = of(m.id, j);
    const double v = (double)of(m.dw, j);
    if (id >= 0 && id == m.id) d += v, again |= j < a.lane;
    const uint32_t at = (uint32_t)id - expert_at(s, a, 0);
    if (id >= 0 && at < KEYS) taken |= 1u << at;
  }
  d *= (double)s.scale;
  const bool counts = m.id >= 0 && !again;
  const double p = counts ? c.weight : 0.0, mine = counts ? d : 0.0;
  const double part = quotient_of(1.0, total), mean = sum_of(p * mine, shift) * part;
  double others = 0;  // the scores' sum without the chosen ones
#pragma unroll
  for (int i = 0; i < KEYS; i++) others += taken >> i & 1 ? 0.0 : e[i];
  double g = d * (sum_of(others, shift) * part);
  for (uint32_t j = 0; j < s.choices; j++)
    g += of(p, j) * (d - of(mine, j));
  g *= c.weight;
  float out[KEYS];
#pragma unroll
  for (int i = 0; i < KEYS; i++) out[i] = (float)(-e[i] * mean);
  for (uint32_t j = 0; j < s.choices; j++) {
    const int32_t id = of(m.id, j);
    const float v = of((float)g, j);
    const uint32_t at = (uint32_t)id - expert_at(s, a, 0);
#pragma unroll
    for (int i = 0; i < KEYS; i++) out[i] = id >= 0 && at == (uint32_t)i ? v : out[i];
  }
  if (a.valid)
    store_logits(dlogits + token * s.experts + expert_at(s, a, 0),
                 (int64_t)s.experts - expert_at(s, a, 0), out);
}

// ---------------------------------------------------------------- host

ec_status launched() { return hipGetLastError() == hipSuccess ? EC_OK : EC_ERR_DEVICE; }
bool fine(const void* p, size_t to) { return p && aligned(p, to); }

// Divides `width` lanes, or as few as do, among the groups; returns the keys of a
// lane (0: there are more groups or choices than lanes).
uint32_t lay_out(Layout& s, uint32_t width) {
  if (s.groups > width || s.choices > width) return 0;
  uint32_t most = 0;  // lanes of a group: a power of two
  while ((s.groups << (most + 1)) <= width && (1u << most) < s.size) most++;
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

template <typename T, int KEYS, bool WAVE>
ec_status route_as(const void* logits, const Layout& s, const float* bias, int32_t* ids,
                   float* weights, hipStream_t stream) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid_of(blocks_of(s)), dim3(kThreads), 0, stream, (const T*)logits,
                       s, bias, ids, weights);
  };
  if (bias) go(expert_route<T, KEYS, true, WAVE>);
  else go(expert_route<T, KEYS, false, WAVE>);
  return launched();
}

// A token's lanes: a whole wave, which is done soonest, or where the waves would
// be more than kEnoughWaves, as few as keep that many, 16 at least, with up to 16
// keys each: a round of the selection then serves up to four tokens.  16384 x 256
// with bias and groups, forward and backward: 16 lanes 29.2 us, 32 lanes 25.1, 64
// lanes 27.4; 65536 tokens, forward, 43, 37 and 43.
constexpr uint64_t kEnoughWaves = 8192;
template <typename T>
ec_status route_of(const void* logits, Layout s, const float* bias, int32_t* ids, float* weights,
                   hipStream_t stream) {
  uint32_t width = 64;
  while (width > 16 && s.tokens * (width / 2) >= kEnoughWaves * 64) width /= 2;
  uint32_t keys = 0;
  for (; width < 64; width *= 2) {
    Layout t = s;
    keys = lay_out(t, width);
    if (keys == 0 || keys > 16) continue;
    switch (keys) {
      case 1: return route_as<T, 1, false>(logits, t, bias, ids, weights, stream);
      case 2: return route_as<T, 2, false>(logits, t, bias, ids, weights, stream);
      case 4: return route_as<T, 4, false>(logits, t, bias, ids, weights, stream);
      case 8: return route_as<T, 8, false>(logits, t, bias, ids, weights, stream);
      default: return route_as<T, 16, false>(logits, t, bias, ids, weights, stream);
    }
  }
  switch (lay_out(s, 64)) {  // more than one key: the groups take more than 32 lanes
    case 1: return route_as<T, 1, false>(logits, s, bias, ids, weights, stream);
    case 2: return route_as<T, 2, true>(logits, s, bias, ids, weights, stream);
    case 4: return route_as<T, 4, true>(logits, s, bias, ids, weights, stream);
    case 8: return route_as<T, 8, true>(logits, s, bias, ids, weights, stream);
    case 16: return route_as<T, 16, true>(logits, s, bias, ids, weights, stream);
    default: return route_as<T, 32, true>(logits, s, bias, ids, weights, stream);
  }
}

template <typename T>
ec_status back_of(const float* dweights, const void* logits, Layout s, const int32_t* ids,
                  void* dlogits, hipStream_t stream) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid_of(blocks_of(s)), dim3(kThreads), 0, stream, dweights,
                       (const T*)logits, s, ids, (T*)dlogits);
  };
  if (s.sigmoid || s.renormalize) {
    s.shift = 2, s.lane_shift = 0;
    while ((1u << s.shift) < s.choices) s.shift++;
    const uint32_t row = (uint32_t)ceil_div(s.experts, 16 / sizeof(T)) * (16 / sizeof(T)) * 4;
    hipLaunchKernelGGL((expert_route_back<T>), grid_of(blocks_of(s)), dim3(kThreads),
                       kThreads / 64 * row, stream, dweights, (const T*)logits, s, ids,
                       (T*)dlogits);
    return launched();
  }
  switch (lay_out(s, 64)) {  // one group: 16 keys at most
    case 1:
      if (s.shift == 6) go(expert_softmax_back<T, 1, true>);
      else go(expert_softmax_back<T, 1, false>);
      break;
    case 2: go(expert_softmax_back<T, 2, true>); break;
    case 4: go(expert_softmax_back<T, 4, true>); break;
    case 8: go(expert_softmax_back<T, 8, true>); break;
    default: go(expert_softmax_back<T, 16, true>);
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
