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
// STREAM: y and out pass the caches by, where y is larger than they are (4096
// tokens of 8 x 7168: 129 -> 116 us; 128 tokens, whose y the last kernel has just
// written, take 4.5 us without and 5.1 with).
template <bool F32, bool STREAM>
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
      if (live[j]) {
        const u32x4_t* const p = reinterpret_cast<const u32x4_t*>(a.y + (size_t)r * a.ldy + c);
        v[j] = STREAM ? __builtin_nontemporal_load(p) : *p;
      }
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
  auto store = [](auto v, auto* to) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, to);
    else *to = v;
  };
  if constexpr (F32) {
    f32x4_t* const to = reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + (size_t)t * a.hidden + c);
    store(f32x4_t{acc[0], acc[1], acc[2], acc[3]}, to);
    store(f32x4_t{acc[4], acc[5], acc[6], acc[7]}, to + 1);
  } else {
    store(u32x4_t{bf16_pair(acc[0], acc[1]), bf16_pair(acc[2], acc[3]), bf16_pair(acc[4], acc[5]), bf16_pair(acc[6], acc[7])},
          reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + (size_t)t * a.hidden + c));
  }
}

// A workgroup takes up to eight slots of a token (fewer where tokens are few:
// two tokens of 16 x 6712, 10.1 us in one each, 4.4); a thread owns columns
// 8 threadIdx.x + 8 blockDim.x i and keeps dout's in registers over the slots,
// whose rows of y are loaded eight together. dout is read once (with a loop
// over the slots outside, and a wait for each row, 4096 tokens of 8 x 7168 took
// 285 us, so 194: 1.0 GB at 5.1 TB/s). y passes the caches by and dy too (206
// and 208 us with plain loads or stores).
// A row of dy belongs to the route that perm names alone, whatever rowpos
// holds, so no two workgroups write one.
//   dweights: a thread's products in the order of its columns, then the wave's
// lanes and the waves in a fixed order.
constexpr int kBackThreads = 1024;

__device__ __forceinline__ float lanes_sum(float v) {   // on lane 63, by DPP moves
#define MOE_DPP_ADD(ctrl, rows) \
  v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, rows, 0xF, false))
  MOE_DPP_ADD(0x111, 0xF);   // row_shr 1, 2, 4, 8
  MOE_DPP_ADD(0x112, 0xF);
  MOE_DPP_ADD(0x114, 0xF);
  MOE_DPP_ADD(0x118, 0xF);
  MOE_DPP_ADD(0x142, 0xA);   // row_bcast 15, 31
  MOE_DPP_ADD(0x143, 0xC);
#undef MOE_DPP_ADD
  return v;
}

template <bool F32, bool DW>
__global__ __launch_bounds__(kBackThreads) void expert_combine_backward(CombineBackwardArgs a) {
  __shared__ float part[kBackThreads / kWave][kAhead];
  const int t = blockIdx.x, lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, k = a.top_k;
  const int s0 = blockIdx.y * a.slots, slots = min(a.slots, k - s0);
  // slot s0 + s on lane s: its row (-1: none), whether dy's row is its own, its weight
  int row = -1, own = 0;
  float weight = 1.f;
  if (lane < slots) {
    const size_t f = (size_t)t * k + s0 + lane;
    row = a.rowpos[f];
    if (row < 0 || row >= a.rows) row = -1;
    if (row >= 0) {
      own = a.dy && a.perm[row] == (long long)f;
      if (a.weights) weight = a.weights[f];
    }
  }
  float dot[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) dot[j] = 0.f;
  for (int c = threadIdx.x * 8; c < a.hidden; c += blockDim.x * 8) {
    u32x4_t v[kAhead];
    if (DW) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int r = __builtin_amdgcn_readlane(row, j);
        if (r >= 0) v[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(a.y + (size_t)r * a.ldy + c));
      }
    }
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
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int r = __builtin_amdgcn_readlane(row, j);
      if (r < 0) continue;
      if (__builtin_amdgcn_readlane(own, j)) {
        const float w = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(weight), j));
        const u32x4_t o = {bf16_pair(w * d[0], w * d[1]), bf16_pair(w * d[2], w * d[3]), bf16_pair(w * d[4], w * d[5]),
                           bf16_pair(w * d[6], w * d[7])};
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>(a.dy + (size_t)r * a.hidden + c));
      }
      if (DW) {
        float f[8];
        unpack8(v[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[j] = fmaf(d[i], f[i], dot[j]);
      }
    }
  }
  if (!DW) return;
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const float sum = lanes_sum(dot[j]);
    if (lane == kWave - 1) part[wave][j] = sum;
  }
  __syncthreads();
  if ((int)threadIdx.x < slots) {
    float sum = 0.f;
    for (int w = 0; w < (int)blockDim.x / kWave; ++w) sum += part[w][threadIdx.x];
    a.dweights[(size_t)t * k + s0 + threadIdx.x] = sum;
  }
}

}  // namespace

hipError_t launch_expert_combine(const CombineArgs& a, bool f32, hipStream_t stream) {
  const int chunks = a.hidden / 8, wide = chunks >= kThreads ? kThreads : (chunks + kWave - 1) / kWave * kWave;
  const dim3 block(wide, kThreads / wide);
  const dim3 grid((unsigned)((a.tokens + block.y - 1) / block.y), (unsigned)((chunks + wide - 1) / wide));
  const bool big = (size_t)a.rows * a.hidden * 2 > kL2Bytes;
  auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
  if (f32) run(big ? expert_combine<true, true> : expert_combine<true, false>);
  else run(big ? expert_combine<false, true> : expert_combine<false, false>);
  return hipGetLastError();
}

hipError_t launch_expert_combine_backward(CombineBackwardArgs a, bool f32, hipStream_t stream) {
  for (a.slots = kAhead; a.slots > 1 && (long long)a.tokens * ((a.top_k + a.slots - 1) / a.slots) < 256; a.slots /= 2) {}
  const int chunks = a.hidden / 8;
  const dim3 block(chunks >= kBackThreads ? kBackThreads : (chunks + kWave - 1) / kWave * kWave);
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(a.tokens, (a.top_k + a.slots - 1) / a.slots), block, 0, stream, a);
  };
  if (f32) run(a.dweights ? expert_combine_backward<true, true> : expert_combine_backward<true, false>);
  else run(a.dweights ? expert_combine_backward<false, true> : expert_combine_backward<false, false>);
  return hipGetLastError();
}

}  // namespace moe
