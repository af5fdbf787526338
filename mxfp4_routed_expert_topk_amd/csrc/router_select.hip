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

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kTokensPerBlock = 4;   // one wave a token

__device__ __forceinline__ float load_logit(const void* p, bool f32, size_t i) {
  return f32 ? static_cast<const float*>(p)[i] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}
__device__ __forceinline__ bool is_masked(float l) { return !(l > -INFINITY); }
__device__ __forceinline__ float finite(float l) { return fminf(l, 3.402823466e38f); }

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
template <class V> __device__ __forceinline__ V wave_sum(V v) { return wave_reduce(v, [](V a, V b) { return a + b; }); }
template <class V> __device__ __forceinline__ V wave_max(V v) { return wave_reduce(v, [](V a, V b) { return a > b ? a : b; }); }

__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// PER: logits per lane (expert lane + 64 j).  KEY: uint32_t, or with a bias 64 bits.
template <int PER, bool BIAS>
__global__ __launch_bounds__(kTokensPerBlock* kWave) void router_select(SelectArgs a) {
  using Key = std::conditional_t<BIAS, unsigned long long, uint32_t>;
  __shared__ double graded[kTokensPerBlock][PER * kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int t = blockIdx.x * kTokensPerBlock + wave;
  if (t >= a.rows) return;   // whole waves
  const int E = a.experts;
  const bool softmax = a.score == 0, limited = a.groups > a.limit;
  float l[PER];   // -inf where masked
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + kWave * j;
    const float v = e < E ? load_logit(a.logits, a.f32, (size_t)t * a.ld + e) : -INFINITY;
    l[j] = is_masked(v) ? -INFINITY : finite(v);
    top = fmaxf(top, l[j]);
  }
  top = wave_max(top);
  if (top == -INFINITY) top = 0.f;   // every expert masked
  float total = 0.f;                 // of exp(l - top)
  if (softmax && !a.renormalize) {
#pragma unroll
    for (int j = 0; j < PER; ++j) total += expf(l[j] - top);
    total = wave_sum(total);
  }

  Key key[PER];   // 0: masked, taken or not there
  const bool wide = BIAS || (limited && a.group_top == 2);
  double s[PER];
  if (wide) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const double x = (double)l[j];
      s[j] = softmax ? exp(x - (double)top) : 1.0 / (1.0 + exp(-x));
      sum += s[j];
    }
    if (BIAS) {
      const double scale = softmax ? 1.0 / wave_sum(sum) : 1.0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int e = lane + kWave * j;
        const float b = e < E ? a.bias[e] : 0.f;
        if (!(b > -INFINITY)) l[j] = -INFINITY;   // switched off (its score has counted above)
        s[j] = s[j] * scale + (double)b;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if constexpr (BIAS) key[j] = l[j] == -INFINITY ? 0 : order_key(s[j]);
    else key[j] = l[j] == -INFINITY ? 0 : order_key(l[j]);
  }

  if (limited) {
    const int per = E / a.groups;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      graded[wave][lane + kWave * j] = key[j] == 0 ? -INFINITY : wide ? s[j] : (double)l[j];
    wave_lds_order();
    // `side` lanes a group, a power of two; each finds the two largest of its share
    int padded = 1;
    while (padded < a.groups) padded *= 2;
    const int side = kWave / padded, g = lane / side;
    double first = -INFINITY, second = -INFINITY;
    if (g < a.groups)
      for (int i = lane % side; i < per; i += side) {
        const double v = graded[wave][g * per + i];
        second = fmax(second, fmin(first, v));
        first = fmax(first, v);
      }
    for (int off = 1; off < side; off *= 2) {
      const double f = __shfl_xor(first, off, kWave), s2 = __shfl_xor(second, off, kWave);
      second = fmax(fmin(first, f), fmax(second, s2));
      first = fmax(first, f);
    }
    const double grade = a.group_top == 2 && second > -INFINITY ? first + second : first;
    int better = 0;   // groups that rank before this lane's
    for (int o = 0; o < a.groups; ++o) {
      const double v = __shfl(grade, o * side, kWave);
      better += v > grade || (v == grade && o < g);
    }
    const unsigned long long open = __ballot(g < a.groups && better < a.limit);   // bit side * g
    const float inverse = 1.f / (float)per;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int of = (int)(((float)(lane + kWave * j) + 0.5f) * inverse);   // exact below 1024 experts
      if (!((open >> (of * side & 63)) & 1)) key[j] = 0;
    }
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

  // weights, a slot a lane
  const bool live = my_id >= 0;
  const float x = live ? finite(load_logit(a.logits, a.f32, (size_t)t * a.ld + my_id)) : -INFINITY;
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
  if (lane < a.top_k) {
    a.ids[(size_t)t * a.top_k + lane] = my_id;
    a.weights[(size_t)t * a.top_k + lane] = w * a.scale;
  }
}

// The logits' gradient from the weights', ids fixed.  With g_j = scale dw_j of
// slot j (0 for an id outside [0, E) or a masked logit) and p_j = w_j / scale:
//   renormalised   dl_j = p_j (g_j - sum p g), times (1 - s_j) for sigmoid scores
//   sigmoid        dl_j = g_j s_j (1 - s_j)
//   softmax        dl_e = s_e (G_e - sum s_j g_j), G_e the sum of e's g_j
// An id that occurs twice gets both slots' terms; all other logits get 0.
template <int PER>
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
  float x = id >= 0 && id < E ? load_logit(a.logits, a.f32, (size_t)t * a.ld + id) : -INFINITY;
  const bool live = !is_masked(x);
  x = live ? finite(x) : -INFINITY;
  const float g = live ? a.scale * a.dweights[(size_t)t * k + lane] : 0.f;

  float l[PER], top = 0.f, total = 1.f;
  if (dense) {
    top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane + kWave * j;
      const float v = e < E ? load_logit(a.logits, a.f32, (size_t)t * a.ld + e) : -INFINITY;
      l[j] = is_masked(v) ? -INFINITY : finite(v);
      top = fmaxf(top, l[j]);
    }
    top = wave_max(top);
    if (top == -INFINITY) top = 0.f;
    total = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      l[j] = expf(l[j] - top);
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
    base = wave_sum(live ? expf(x - top) / total * g : 0.f);
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
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + kWave * j;
    if (e >= E) break;
    float v = row[e];
    if (dense) v = l[j] > 0.f ? l[j] / total * (v - base) : 0.f;
    if (a.f32) static_cast<float*>(a.dlogits)[(size_t)t * E + e] = v;
    else static_cast<uint16_t*>(a.dlogits)[(size_t)t * E + e] = f32_to_bf16_rne(v);
  }
}

// f(integral_constant PER) for the smallest power of two with 64 PER >= E
template <class F>
void per_lane(int E, F f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_router_select(const SelectArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.rows + kTokensPerBlock - 1) / kTokensPerBlock)), block(kTokensPerBlock * kWave);
  per_lane(a.experts, [&](auto per) {
    constexpr int PER = decltype(per)::value;
    if (a.bias) hipLaunchKernelGGL((router_select<PER, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((router_select<PER, false>), grid, block, 0, stream, a);
  });
  return hipGetLastError();
}

hipError_t launch_router_select_backward(const SelectBackwardArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.rows + kTokensPerBlock - 1) / kTokensPerBlock)), block(kTokensPerBlock * kWave);
  per_lane(a.experts, [&](auto per) {
    hipLaunchKernelGGL((router_select_backward<decltype(per)::value>), grid, block, 0, stream, a);
  });
  return hipGetLastError();
}

}  // namespace moe
