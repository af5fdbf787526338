// Each token's weighted sum of its routes' rows, and its gradients:
//   forward   out_t = sum over slots s of w[t,s] y[rowpos[t,s]]   (fp32, slots ascending, rounded once)
//   backward  dy_r   = w[t,s] dout_t of the route f = t k + s = perm[r]
//             dw[t,s] = <dout_t, y[rowpos[t,s]]>
// A rowpos outside [0, rows) is no route: it adds nothing and its dw is 0.
#include "moe_internal.h"

namespace moe {
namespace {

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
constexpr int kThreads = 256;
constexpr int kAhead = 8;   // slots whose rows are loaded together

__device__ __forceinline__ void unpack8(u32x4_t v, float (&f)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = __uint_as_float(v[q] << 16);
    f[2 * q + 1] = __uint_as_float(v[q] & 0xFFFF0000u);
  }
}

// A thread owns 8 columns; blockDim is (columns / 8, tokens).
template <bool F32>
__global__ __launch_bounds__(kThreads) void expert_combine(CombineArgs a) {
  const int t = blockIdx.x * blockDim.y + threadIdx.y;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
  if (t >= a.tokens || c >= a.hidden) return;
  const int32_t* const pos = a.rowpos + (size_t)t * a.top_k;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int s0 = 0; s0 < a.top_k; s0 += kAhead) {
    bool live[kAhead];
    u32x4_t v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = s0 + j < a.top_k ? pos[s0 + j] : -1;
      live[j] = r >= 0 && r < a.rows;
      if (live[j]) v[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(a.y + (size_t)r * a.ldy + c));
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (!live[j]) continue;
      const float w = a.weights ? a.weights[(size_t)t * a.top_k + s0 + j] : 1.f;
      float f[8];
      unpack8(v[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
    }
  }
  if constexpr (F32) {
    f32x4_t* const to = reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + (size_t)t * a.hidden + c);
    to[0] = f32x4_t{acc[0], acc[1], acc[2], acc[3]};
    to[1] = f32x4_t{acc[4], acc[5], acc[6], acc[7]};
  } else {
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + (size_t)t * a.hidden + c) =
        u32x4_t{bf16_pair(acc[0], acc[1]), bf16_pair(acc[2], acc[3]), bf16_pair(acc[4], acc[5]), bf16_pair(acc[6], acc[7])};
  }
}

// One workgroup a token; a thread owns columns 8 threadIdx.x + 8 blockDim.x i.
// A row of dy belongs to the route that perm names alone, whatever rowpos
// holds, so no two workgroups write one.
constexpr int kBackThreads = 1024;
template <bool F32>
__global__ __launch_bounds__(kBackThreads) void expert_combine_backward(CombineBackwardArgs a) {
  __shared__ float part[kBackThreads / kWave][kMaxTopK];
  const int t = blockIdx.x, lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  for (int s = 0; s < a.top_k; ++s) {
    const size_t f = (size_t)t * a.top_k + s;
    const int r = a.rowpos[f];
    const bool live = r >= 0 && r < a.rows;
    const bool owns = a.dy && live && a.perm[r] == (long long)f;
    const float w = live && a.weights ? a.weights[f] : 1.f;
    float dot = 0.f;
    if (live)
      for (int c = threadIdx.x * 8; c < a.hidden; c += blockDim.x * 8) {
        float d[8];
        if constexpr (F32) {
          const f32x4_t* const p = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(a.dout) + (size_t)t * a.lddout + c);
          const f32x4_t lo = p[0], hi = p[1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            d[i] = lo[i];
            d[4 + i] = hi[i];
          }
        } else {
          unpack8(*reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.dout) + (size_t)t * a.lddout + c), d);
        }
        if (a.dweights) {
          float v[8];
          unpack8(*reinterpret_cast<const u32x4_t*>(a.y + (size_t)r * a.ldy + c), v);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = fmaf(d[i], v[i], dot);
        }
        if (owns)
          *reinterpret_cast<u32x4_t*>(a.dy + (size_t)r * a.hidden + c) =
              u32x4_t{bf16_pair(w * d[0], w * d[1]), bf16_pair(w * d[2], w * d[3]), bf16_pair(w * d[4], w * d[5]),
                      bf16_pair(w * d[6], w * d[7])};
      }
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) dot += __shfl_xor(dot, off, kWave);
    if (lane == 0) part[wave][s] = dot;
  }
  __syncthreads();
  if (a.dweights && (int)threadIdx.x < a.top_k) {
    float sum = 0.f;
    for (int w = 0; w < (int)blockDim.x / kWave; ++w) sum += part[w][threadIdx.x];
    a.dweights[(size_t)t * a.top_k + threadIdx.x] = sum;
  }
}

}  // namespace

hipError_t launch_expert_combine(const CombineArgs& a, bool f32, hipStream_t stream) {
  const int chunks = a.hidden / 8, wide = chunks >= kThreads ? kThreads : (chunks + kWave - 1) / kWave * kWave;
  const dim3 block(wide, kThreads / wide);
  const dim3 grid((unsigned)((a.tokens + block.y - 1) / block.y), (unsigned)((chunks + wide - 1) / wide));
  if (f32) hipLaunchKernelGGL(expert_combine<true>, grid, block, 0, stream, a);
  else hipLaunchKernelGGL(expert_combine<false>, grid, block, 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_expert_combine_backward(const CombineBackwardArgs& a, bool f32, hipStream_t stream) {
  const int chunks = a.hidden / 8;
  const dim3 block(chunks >= kBackThreads ? kBackThreads : (chunks + kWave - 1) / kWave * kWave);
  if (f32) hipLaunchKernelGGL(expert_combine_backward<true>, dim3(a.tokens), block, 0, stream, a);
  else hipLaunchKernelGGL(expert_combine_backward<false>, dim3(a.tokens), block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace moe
