// Router with scores, a balance bias and expert groups, and its gradient.
// For a token's logits l_e (those above fp32's largest count as it; -inf and
// NaN mean that the expert is masked):
//   score   s_e = exp(l_e - max) / sum exp(l - max)   or   1 / (1 + exp(-l_e));   masked: 0
//   value   c_e = s_e + bias_e, in fp64; without a bias experts rank by l_e
//   groups  num_groups runs of consecutive experts; a group's grade is the sum
//           of its group_top largest values; the group_limit best groups stay
//   ids     the k largest values of the experts that stay, equal ones in the
//           order of their ids; -1 (weight 0) once no expert is left
//   weights scale s_id, or scale s_id / sum of the selected scores
// Values are fp64 because ids are compared, not rounded: in fp32 two experts
// whose values lie within a rounding of each other would change places with
// the exponential's last bit.
#include <climits>
#include <cmath>
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kTokensPerBlock = 4;   // one wave a token

template <bool F32>
__device__ __forceinline__ float load_logit(const void* p, size_t i) {
  return F32 ? static_cast<const float*>(p)[i] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}
constexpr float kMost = 3.402823466e38f;   // fp32's largest number
constexpr int kNanOrInf = 0x203;           // v_cmp_class: NaN or +inf
// NaN as -inf, +inf as the largest number (as integers: what lies above it is infinite or NaN)
__device__ __forceinline__ float cleaned(float l) {
  return l > -INFINITY ? __int_as_float(min(__float_as_int(l), __float_as_int(kMost))) : -INFINITY;
}

// Order-preserving integers; 0 is below every value.  -0 and +0 are equal.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ unsigned long long order_key(double v) {
  const long long u = __double_as_longlong(v + 0.0);
  return (unsigned long long)u ^ ((unsigned long long)(u >> 63) | 0x8000000000000000ull);
}

template <class V, class F>
__device__ __forceinline__ V wave_reduce(V v, F f) {
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) v = f(v, (V)__shfl_xor(v, off, kWave));
  return v;
}

// Reductions of 32-bit values on DPP moves (6 instructions, no LDS); the result
// is uniform. A lane without a source gets `none`.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t none, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xF, false);
}
template <class F>
__device__ __forceinline__ uint32_t reduce32(uint32_t v, uint32_t none, F f) {
  v = f(v, dpp<0x111, 0xF>(none, v));   // row_shr 1, 2, 4, 8: lane 15 of each row of 16 has its row's
  v = f(v, dpp<0x112, 0xF>(none, v));
  v = f(v, dpp<0x114, 0xF>(none, v));
  v = f(v, dpp<0x118, 0xF>(none, v));
  v = f(v, dpp<0x142, 0xA>(none, v));   // row_bcast 15 into rows 1 and 3, 31 into rows 2 and 3
  v = f(v, dpp<0x143, 0xC>(none, v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(reduce32(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  return reduce32(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float wave_max(float v) {   // of no NaN
  const uint32_t key = wave_max(order_key(v));
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ double wave_sum(double v) { return wave_reduce(v, [](double a, double b) { return a + b; }); }

// 2^(x log2 e) on the hardware's exponential: off by (1.25 |x| + 2) u of the value (the
// product's rounding |x| u, the constant's, the instruction's 2 u; 0.95 of that is the
// most found over [-87, 0]) and 0 below 2^-126.  Sums over all experts take it (16383 x
// 896 scores: the gradient 30 us with expf, 25 with it), selected weights expf.
__device__ __forceinline__ float quick_exp(float x) { return __expf(x); }

__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// v of a uniform lane
__device__ __forceinline__ float at_lane(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ double at_lane(double v, int lane) {
  const long long u = __double_as_longlong(v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __longlong_as_double((long long)((unsigned long long)hi << 32 | (uint32_t)__builtin_amdgcn_readlane((int)u, lane)));
}

// The groups that stay (bit g), from each expert's value over `total` (-INFINITY: none).
// gap: what separates the last that stays from the first that does not.
template <int PER, class V>
__device__ __forceinline__ unsigned long long open_groups(const SelectArgs& a, const V (&value)[PER], V* graded, int lane,
                                                          V& gap, double total = 1.0) {
#pragma unroll
  for (int j = 0; j < PER; ++j) graded[lane + kWave * j] = value[j];
  wave_lds_order();
  const int side = 1 << a.side, share = lane >> a.side;   // `side` lanes a group
  V first = -INFINITY, second = -INFINITY;                // the two largest of the lane's experts
  if (share < a.groups)
    for (int i = lane & (side - 1); i < a.per; i += side) {
      const V v = graded[share * a.per + i];
      second = max(second, min(first, v));
      first = max(first, v);
    }
  for (int off = 1; off < side; off *= 2) {
    const V f = __shfl_xor(first, off, kWave), s = __shfl_xor(second, off, kWave);
    second = max(min(first, f), max(second, s));
    first = max(first, f);
  }
  if constexpr (std::is_same_v<V, double>) {   // the order of the values is theirs before it too
    first /= total;
    second /= total;
  }
  const V sum = a.group_top == 2 && second > -INFINITY ? first + second : first;
  const V grade = __shfl(sum, lane << a.side & (kWave - 1), kWave);   // group g on lane g
  int better = 0;                                                     // groups that rank before it
  for (int o = 0; o < a.groups; ++o) {
    const V v = at_lane(grade, o);
    better += v > grade || (v == grade && o < lane);
  }
  const bool is = lane < a.groups;
  const int last = __ffsll((unsigned long long)__ballot(is && better == a.limit - 1)) - 1;
  const int next = __ffsll((unsigned long long)__ballot(is && better == a.limit)) - 1;
  gap = at_lane(grade, last & (kWave - 1)) - at_lane(grade, next & (kWave - 1));   // (none of a rank: NaN grades)
  return __ballot(is && better < a.limit);
}

// Sets what is not of an open group to `none`: bit g of `open` becomes the sign
// of the bits in reverse order, g to the left.
template <int PER, class V>
__device__ __forceinline__ void keep_open(const SelectArgs& a, unsigned long long open, int lane, V (&value)[PER],
                                          V none = (V)-INFINITY) {
  const float e = (float)lane + 0.5f;
  auto group = [&](int j) { return (uint32_t)((e + (float)(kWave * j)) * a.inverse); };   // exact below 1024 experts
  if (a.groups <= 32) {
    const uint32_t bits = __brev((uint32_t)open);
#pragma unroll
    for (int j = 0; j < PER; ++j) value[j] = (int32_t)(bits << (group(j) & 31)) < 0 ? value[j] : none;
  } else {
    const unsigned long long bits = __brevll(open);
#pragma unroll
    for (int j = 0; j < PER; ++j) value[j] = (long long)(bits << (group(j) & 63)) < 0 ? value[j] : none;
  }
}

// The fp64 values that groups are graded by (-inf: masked or switched off), and
// what they are to be divided by: scores are quotients, and sums of exponentials
// alone round, and tie, differently. With a bias they are divided here.
template <int PER, bool BIAS>
__device__ __forceinline__ double exact_values(const SelectArgs& a, const float (&l)[PER], const float (&b)[PER], float top,
                                               double (&v)[PER]) {
  double total = 1.0;
#pragma unroll
  for (int j = 0; j < PER; ++j) v[j] = (double)l[j];
  if (BIAS || (a.groups > a.limit && a.group_top == 2)) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const double x = (double)l[j];
      v[j] = a.score == 0 ? exp(x - (double)top) : 1.0 / (1.0 + exp(-x));
      sum += v[j];
    }
    if (a.score == 0) total = at_lane(wave_sum(sum), 0);   // (in scalar registers)
    if (BIAS) {
#pragma unroll
      for (int j = 0; j < PER; ++j) v[j] = v[j] / total + (double)b[j];
      total = 1.0;
    }
  }
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (l[j] == -INFINITY || (BIAS && !(b[j] > -INFINITY))) v[j] = -INFINITY;
  return total;
}

// The ids of a token's slots, slot r on lane r (-1: none), by k rounds of the
// best over the wave, every value exact: for rows that the quick way below
// cannot settle.
template <int PER, bool BIAS>
__device__ __forceinline__ int select_by_rounds(const SelectArgs& a, const float (&l)[PER], const float (&b)[PER], float top,
                                                double* graded, int lane) {
  using Key = std::conditional_t<BIAS, unsigned long long, uint32_t>;
  double v[PER];
  const double total = exact_values<PER, BIAS>(a, l, b, top, v);
  Key key[PER];   // 0: masked, taken or not there
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if constexpr (BIAS) key[j] = v[j] == -INFINITY ? 0 : order_key(v[j]);
    else key[j] = l[j] == -INFINITY ? 0 : order_key(l[j]);
  }
  if (a.groups > a.limit) {
    double gap;
    keep_open(a, open_groups<PER, double>(a, v, graded, lane, gap, total), lane, key, (Key)0);
  }
  int my_id = -1;
  for (int r = 0; r < a.top_k; ++r) {
    Key best = 0;
    int id = INT_MAX;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (key[j] > best) {
        best = key[j];
        id = lane + kWave * j;
      }
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) {
      const Key ok = __shfl_xor(best, off, kWave);
      const int oi = __shfl_xor(id, off, kWave);
      if (ok > best || (ok == best && oi < id)) {
        best = ok;
        id = oi;
      }
    }
    if (best == 0) break;   // the same on every lane
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (id == lane + kWave * j) key[j] = 0;
    if (lane == r) my_id = id;
  }
  return my_id;
}

// Whether logit j of every lane exists: E is above 64 (PER - 2), and 64 for PER 2.
template <int PER>
__device__ __forceinline__ bool there(int j) { return j < PER - 2; }

// One wave a token; PER logits per lane (expert lane + 64 j).
//   The quick way: of the lanes' largest values the k-th, found bit by bit with
// ballots, bounds the k-th largest of all from below; what reaches it, about
// k + 2 experts, is packed to one a lane, ordered exactly and ranked by
// comparison with every other. k rounds of the best over the wave took 80 us
// for 16383 tokens of 896 experts, top-16, where this takes 16.1;
// 4133 tokens of 384, top-8, sigmoid scores, a bias and four of eight groups: 19.2 and 7.6. Most of it is the
// issue of vector instructions (330 and 560 a wave, 70 % of the SIMDs' time).
//   With a bias the bound is taken in fp32 and lowered by twice what an fp32
// value can be off, so that no expert of the fp64 order is lost. The packed ones
// get fp64 values (one exponential a lane, softmax scores their sum in fp64
// too) where two of them are closer than that. Groups are graded in fp32 too
// where the grades at the border are further apart, else in fp64. Left to the
// rounds are rows of which more than 64 experts reach the bound, many equal ones.
template <int PER, bool BIAS, bool F32>
__global__ __launch_bounds__(kTokensPerBlock* kWave) void router_select(SelectArgs a) {
  __shared__ double shared[kTokensPerBlock][PER * kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int t = blockIdx.x * kTokensPerBlock + wave;
  if (t >= a.rows) return;   // whole waves
  const int E = a.experts, k = a.top_k;
  const bool softmax = a.score == 0, limited = a.groups > a.limit;
  const size_t row = (size_t)t * a.ld;
  float l[PER], b[PER];   // l: -inf where masked
  float top = -INFINITY;
  bool special = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + kWave * j;
    const bool in = there<PER>(j) || e < E;
    const int at = there<PER>(j) ? e : min(e, E - 1);   // loaded without a branch, which would wait
    l[j] = load_logit<F32>(a.logits, row + at);
    b[j] = BIAS ? a.bias[at] : 0.f;
    if (!in) l[j] = -INFINITY;
    special |= __builtin_amdgcn_classf(l[j], kNanOrInf);
  }
  if (__ballot(special)) {   // rare: one test a logit, where cleaning takes three instructions
#pragma unroll
    for (int j = 0; j < PER; ++j) l[j] = cleaned(l[j]);
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) top = fmaxf(top, l[j]);
  float total = 0.f;   // of exp(l - top)
  if (softmax) {
    top = wave_max(top);
    if (top == -INFINITY) top = 0.f;   // every expert masked
    if (!a.renormalize || BIAS) {
#pragma unroll
      for (int j = 0; j < PER; ++j) total += quick_exp(l[j] - top);
      total = wave_sum(total);
    }
  }

  // What experts are compared by: the logit, or an approximate score plus the bias, in fp32.
  // An approximate value v is off by less than off (1 + |v|): by u |v| of the bias's addition, and by what its score
  // is off, for which 8 u and 64 u are taken:
  //   sigmoid  (1.25 |x| + 2) u of the exponential reach the score times s (1 - s), 0.7 u at most; the rounding of
  //            1 + exp u, the reciprocal 2 u: 3.7 u
  //   softmax  x = l - top is rounded too, so (2.25 |x| + 2) u of an exponential: of the score's own, times s <=
  //            exp(-|x|), 2.1 u; of the sum's, whose average |x| is at most ln 1024, 17.6 u; the sum's 22 additions in
  //            a row 22 u; the reciprocal and the product 2 u: 44 u
  const float off = BIAS && softmax ? 0x1p-18f : 0x1p-21f;
  float value[PER];
  auto put_scores = [&](float (&to)[PER], float share) {   // -inf for masked experts
    auto put = [&](auto score) {
#pragma unroll
      for (int j = 0; j < PER; ++j) to[j] = l[j] == -INFINITY ? -INFINITY : score(l[j]);
    };
    if (softmax) put([&](float x) { return quick_exp(x - top) * share; });
    else put([&](float x) { return __builtin_amdgcn_rcpf(1.f + quick_exp(-x)); });
  };
  if constexpr (BIAS) {
    put_scores(value, 1.f / total);
#pragma unroll
    for (int j = 0; j < PER; ++j) value[j] = fmaxf(value[j] + b[j], -INFINITY);   // (NaN, by the bias: -inf)
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) value[j] = l[j];
  }
  if (limited) {
    const bool graded = !BIAS && a.group_top == 2;   // by the scores' sums, though experts rank by logit
    float grade[PER];
    if (graded) {
      put_scores(grade, 1.f);
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) grade[j] = value[j];
    }
    float gap;
    unsigned long long open = open_groups<PER, float>(a, grade, reinterpret_cast<float*>(shared[wave]), lane, gap);
    if (BIAS || graded) {
      float most = -INFINITY;
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (grade[j] > -INFINITY) most = fmaxf(most, fabsf(grade[j]));
      most = wave_max(most);
      // A gap between two sums of two values, each off by off (1 + most) and once rounded. One that could be
      // of the other sign is decided in fp64; a gap to a group without experts is infinite.
      if (most > -INFINITY && !(gap > 4.f * off * (1.f + most))) {
        double v[PER], exact_gap;
        const double total = exact_values<PER, BIAS>(a, l, b, top, v);
        wave_lds_order();
        open = open_groups<PER, double>(a, v, shared[wave], lane, exact_gap, total);
      }
    }
    keep_open(a, open, lane, value);
  }

  int id = -1, slot = lane;   // this lane's expert, and its place among the chosen
  float x = -INFINITY;
  // What a candidate reaches, from a key that k values reach.
  auto bound_of = [&](uint32_t key) {
    float v = __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
    if (BIAS) v -= 2.f * off * (1.f + fabsf(v));
    return v > -kMost ? v : -kMost;   // (NaN of an infinite bias: every expert is a candidate)
  };
  float bound = -kMost;
  uint32_t kth = 0;   // of the lanes' largest keys, the k-th or a little less; 0: fewer than k lanes have one
  // One logit a lane may all be candidates: without a search up to 16 experts (65536 tokens, top-8: 16 experts
  // 19.4 us without one and 19.7 with, 32 25.8 and 20.8, 64 40 and 22).
  if (PER > 1 || E > 16) {
    float most = value[0];
#pragma unroll
    for (int j = 1; j < PER; ++j) most = fmaxf(most, value[j]);
    uint32_t key = most > -INFINITY ? order_key(most) : 0;
    asm volatile("" : "+v"(key));   // (else the search does its selection in every step)
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t next = kth | 1u << bit;
      const int n = __popcll(__ballot(key >= next));
      if (n >= k) kth = next;
      if (n == k) break;
    }
    if (kth) bound = bound_of(kth);
  }
  int n;
  uint2* const packed = reinterpret_cast<uint2*>(shared[wave]);
  wave_lds_order();   // the grades have been read
  for (bool again = false;; again = true) {
    n = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const bool in = value[j] >= bound;
      const unsigned long long mask = __ballot(in);
      const int at = __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
      if (in) packed[n + at] = make_uint2(lane + kWave * j, __float_as_uint(l[j]));   // ids ascend; there is room for all
      n += __popcll(mask);
    }
    wave_lds_order();
    if (PER == 1 || n <= kWave || again || !kth) break;
    // More than a wave holds (top-32 of 1024: few rows of a thousand, but the rounds for them were the kernel's
    // time, 4096 tokens 20 to 29 us for 12 to 14): a higher bound from a search over every value, until k and no
    // more than the wave has reach it.
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t next = kth | 1u << bit;
      if (next == kth) continue;
      const float reach = __uint_as_float(next & 0x80000000u ? next ^ 0x80000000u : ~next);
      n = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) n += __popcll(__ballot(value[j] >= reach));
      if (n >= k) kth = next;
      if (n >= k && n < kWave - 8) break;
    }
    bound = bound_of(kth);
  }
  const bool settled = n <= kWave;
  if (settled) {
    if (lane < n) {
      const uint2 v = packed[lane];
      id = (int)v.x;
      x = __uint_as_float(v.y);
    }
    slot = 0;   // how many candidates rank before the lane's
    if constexpr (BIAS) {
      // In fp32 first, which settles the order unless two values are closer than both can be off.
      float v = softmax ? quick_exp(x - top) * (1.f / total) : __builtin_amdgcn_rcpf(1.f + quick_exp(-x));
      v = lane < n ? v + a.bias[id] : -INFINITY;
      const float near = 4.f * off * (1.f + fabsf(v));
      int close = 0;   // itself, and others
      for (int s = 0; s < n; ++s) {
        const float other = at_lane(v, s);
        slot += other > v;
        close += !(fabsf(other - v) > near);
      }
      if (__ballot(lane < n && close > 1)) {
        slot = 0;
        double score = 0.0;
        if (softmax) {
          double sum = 0.0;
#pragma unroll
          for (int j = 0; j < PER; ++j) sum += exp((double)l[j] - (double)top);
          score = exp((double)x - (double)top) / wave_sum(sum);
        } else {
          score = 1.0 / (1.0 + exp(-(double)x));
        }
        const unsigned long long key = lane < n ? order_key(score + (double)a.bias[id]) : 0;
        for (int s = 0; s < n; ++s) {
          const unsigned long long other = (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)(key >> 32), s) << 32 |
                                           (uint32_t)__builtin_amdgcn_readlane((int)key, s);
          slot += other > key || (other == key && s < lane);
        }
      }
    } else {
      const uint32_t high = order_key(x);
      const unsigned long long key = (unsigned long long)high << 32 | (uint32_t)(kWave - lane);
      for (int s = 0; s < n; ++s)
        slot += ((unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)high, s) << 32 | (uint32_t)(kWave - s)) > key;
    }
    if (lane >= n) slot = lane;   // an empty slot, if it is one
    else if (slot >= k) id = -1;
  }
  if (!settled) {
    wave_lds_order();
    id = select_by_rounds<PER, BIAS>(a, l, b, top, shared[wave], lane);
    slot = lane;
    x = id >= 0 ? cleaned(load_logit<F32>(a.logits, row + id)) : -INFINITY;
  }

  // weights
  const bool live = id >= 0;
  if (!live) x = -INFINITY;
  float w;
  if (softmax) {
    w = expf(x - (a.renormalize ? wave_max(x) : top));
    if (!a.renormalize) w /= total;
  } else {
    // renormalised weights are taken relative to the largest, so that small scores do not vanish
    const float shift = a.renormalize ? fminf(wave_max(x), 0.f) : 0.f;
    w = expf(fminf(x, 0.f) - shift) / (1.f + expf(-fabsf(x)));
  }
  if (!live) w = 0.f;
  if (a.renormalize) {
    const float sum = wave_sum(w);
    if (live) w /= sum;
  }
  if (slot < k) {
    a.ids[(size_t)t * k + slot] = id;
    a.weights[(size_t)t * k + slot] = w * a.scale;
  }
}

// The logits' gradient from the weights', ids fixed.  With g_j = scale dw_j of
// slot j (0 for an id outside [0, E) or a masked logit) and p_j = w_j / scale:
//   renormalised   dl_j = p_j (g_j - sum p g), times (1 - s_j) for sigmoid scores
//   sigmoid        dl_j = g_j s_j (1 - s_j)
//   softmax        dl_e = s_e (G_e - sum s_j g_j), G_e the sum of e's g_j
// An id that occurs twice gets both slots' terms; all other logits get 0.
template <int PER, bool F32>
__global__ __launch_bounds__(kTokensPerBlock* kWave) void router_select_backward(SelectBackwardArgs a) {
  __shared__ float rows[kTokensPerBlock][PER * kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int t = blockIdx.x * kTokensPerBlock + wave;
  if (t >= a.rows) return;   // whole waves
  const int E = a.experts, k = a.top_k;
  const bool softmax = a.score == 0, dense = softmax && !a.renormalize;
  float* const row = rows[wave];
#pragma unroll
  for (int j = 0; j < PER; ++j) row[lane + kWave * j] = 0.f;
  const int id = lane < k ? a.ids[(size_t)t * k + lane] : -1;
  const float x = id >= 0 && id < E ? cleaned(load_logit<F32>(a.logits, (size_t)t * a.ld + id)) : -INFINITY;
  const bool live = x > -INFINITY;
  const float g = live ? a.scale * a.dweights[(size_t)t * k + lane] : 0.f;

  float l[PER], top = 0.f, total = 1.f;
  if (dense) {
    top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane + kWave * j;
      l[j] = cleaned(load_logit<F32>(a.logits, (size_t)t * a.ld + (there<PER>(j) ? e : min(e, E - 1))));
      if (!there<PER>(j) && e >= E) l[j] = -INFINITY;
      top = fmaxf(top, l[j]);
    }
    top = wave_max(top);
    if (top == -INFINITY) top = 0.f;
    total = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      l[j] = quick_exp(l[j] - top);
      total += l[j];
    }
    total = wave_sum(total);
  }
  const float small = expf(-fabsf(x));                                        // sigmoid: of -|l|
  const float other = (x < 0.f ? 1.f : small) / (1.f + small);                // sigmoid: 1 - s
  float d, base = 0.f;
  if (a.renormalize) {
    const float most = wave_max(x);
    float p = softmax ? expf(x - most) : expf(fminf(x, 0.f) - fminf(most, 0.f)) / (1.f + small);
    if (!live) p = 0.f;
    const float sum = wave_sum(p);
    p = live ? p / sum : 0.f;
    const float mean = wave_sum(p * g);
    d = p * (g - mean);
    if (!softmax) d *= other;
  } else if (softmax) {
    d = g;
    base = wave_sum(live ? quick_exp(x - top) / total * g : 0.f);
  } else {
    d = g * other * (x < 0.f ? small : 1.f) / (1.f + small);
  }
  if (!live) d = 0.f;
  float mine = 0.f;   // the sum of every slot of this id, in slot order
  for (int s = 0; s < k; ++s) {
    const float v = __shfl(d, s, kWave);
    if (__shfl(id, s, kWave) == id) mine += v;
  }
  wave_lds_order();
  if (live) row[id] = mine;
  wave_lds_order();
  const float inverse = 1.f / total;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + kWave * j;
    if (!there<PER>(j) && e >= E) break;
    float v = row[e];
    if (dense) v = l[j] > 0.f ? l[j] * inverse * (v - base) : 0.f;
    if constexpr (F32) static_cast<float*>(a.dlogits)[(size_t)t * E + e] = v;
    else static_cast<uint16_t*>(a.dlogits)[(size_t)t * E + e] = f32_to_bf16_rne(v);
  }
}

// f(integral_constant PER): 1, or the smallest even number with 64 PER >= E
template <int PER = 1, class F>
void per_lane(int E, F f) {
  if constexpr (PER < kRouterMaxExperts / kWave) {
    if (E > kWave * PER) return per_lane<PER == 1 ? 2 : PER + 2>(E, f);
  }
  f(std::integral_constant<int, PER>{});
}

}  // namespace

hipError_t launch_router_select(SelectArgs a, bool f32, hipStream_t stream) {
  a.per = a.experts / a.groups;
  a.inverse = 1.f / (float)a.per;
  a.side = 6;
  for (int padded = 1; padded < a.groups; padded *= 2) --a.side;
  const dim3 grid((unsigned)((a.rows + kTokensPerBlock - 1) / kTokensPerBlock)), block(kTokensPerBlock * kWave);
  per_lane(a.experts, [&](auto per) {
    constexpr int PER = decltype(per)::value;
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
    if (a.bias) run(f32 ? router_select<PER, true, true> : router_select<PER, true, false>);
    else run(f32 ? router_select<PER, false, true> : router_select<PER, false, false>);
  });
  return hipGetLastError();
}

hipError_t launch_router_select_backward(const SelectBackwardArgs& a, bool f32, hipStream_t stream) {
  const dim3 grid((unsigned)((a.rows + kTokensPerBlock - 1) / kTokensPerBlock)), block(kTokensPerBlock * kWave);
  per_lane(a.experts, [&](auto per) {
    constexpr int PER = decltype(per)::value;
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
    run(f32 ? router_select_backward<PER, true> : router_select_backward<PER, false>);
  });
  return hipGetLastError();
}

}  // namespace moe
