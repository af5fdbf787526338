// Product of bf16 rows with an MXFP4 matrix in checkpoint layout,
//   y [M, N] = x [M, K] W [N, K]^T,   W = code 2^(byte - 127)
// and, gated, silu(y[:, c]) y[:, c + N/2] for the fused w1||w3 of a shared
// expert.  A weight has at most two significant bits, so W is exact in bf16
// for every scale byte (0 is 2^-127, 255 NaN; 4 and 6 times 2^127 are infinite
// there as in fp32); products are summed in fp32 on v_mfma_f32_16x16x32_bf16,
// which keeps subnormal operands, and the sum is rounded once.
#include "moe_internal.h"

namespace moe {
namespace {

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// ---- few rows: W is streamed once per 16 MT rows of x.
//
// A workgroup owns 16 output columns and MT 16-row blocks of x; its kSplit
// waves take 256 K at a time in turn and their partial sums are added in wave
// order.  In 256 K a lane takes the 32 contiguous bytes of weight blocks 2q
// and 2q + 1 (q its quarter of the wave) and x's values alike: which K values
// share an MFMA does not matter to the sum.
constexpr int kSplit = 8;

__device__ __forceinline__ float gated(float g, float u) { return g / (1.f + expf(-g)) * u; }

template <int MT, bool GATE, bool F32>
__global__ __launch_bounds__(kSplit* kWave) void linear_rows(LinearArgs a) {
  constexpr int NB = GATE ? 2 : 1;   // weight rows an output column needs
  __shared__ f32x4_t part[kSplit][NB][MT][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int cols = GATE ? a.n / 2 : a.n, groups = a.k / 32;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * (16 * MT);
  // columns past the matrix repeat its last and are not stored
  const int n = min(n0 + r, cols - 1);
  f32x4_t acc[NB][MT];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[b][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int units = (groups + 7) / 8;
  for (int u = wave; u < units; u += kSplit) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = 8 * u + 2 * q + h;
      const bool in = g < groups;
      u32x4_t w[NB];
      float s[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const size_t at = (size_t)(n + b * cols) * groups + g;
        w[b] = in ? *reinterpret_cast<const u32x4_t*>(a.codes + at * 16) : u32x4_t{0, 0, 0, 0};
        s[b] = e8m0_to_f32(in ? a.scales[at] : 127);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8_t x[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int m = m0 + 16 * i + r;
          x[i] = bf16x8_t{};
          if (in && m < a.m) x[i] = *reinterpret_cast<const bf16x8_t*>(a.x + (size_t)m * a.ldx + 32 * g + 8 * j);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const bf16x8_t v = dequant8(w[b][j], s[b]);
#pragma unroll
          for (int i = 0; i < MT; ++i) acc[b][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, x[i], acc[b][i], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][b][i][lane] = acc[b][i];
  __syncthreads();
  if (wave >= MT) return;   // wave i adds and stores row block i
  f32x4_t v[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    v[b] = part[0][b][wave][lane];
#pragma unroll
    for (int w = 1; w < kSplit; ++w) v[b] += part[w][b][wave][lane];
  }
  const int m = m0 + 16 * wave + r, c = n0 + 4 * q;
  if (m >= a.m) return;
  const size_t at = (size_t)m * cols + c;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (c + e >= cols) break;
    const float f = GATE ? gated(v[0][e], v[NB - 1][e]) : v[0][e];
    if (F32) static_cast<float*>(a.out)[at + e] = f;
    else static_cast<uint16_t*>(a.out)[at + e] = f32_to_bf16_rne(f);
  }
}

template <int MT>
hipError_t launch_rows(const LinearArgs& a, bool gate, bool f32, hipStream_t stream) {
  const int cols = gate ? a.n / 2 : a.n;
  const dim3 grid((cols + 15) / 16, (a.m + 16 * MT - 1) / (16 * MT)), block(kSplit * kWave);
  if (gate && f32) hipLaunchKernelGGL((linear_rows<MT, true, true>), grid, block, 0, stream, a);
  else if (gate) hipLaunchKernelGGL((linear_rows<MT, true, false>), grid, block, 0, stream, a);
  else if (f32) hipLaunchKernelGGL((linear_rows<MT, false, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((linear_rows<MT, false, false>), grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mxfp4_linear(const LinearArgs& a, bool gate, bool f32, hipStream_t stream) {
  if (a.m <= 16) return launch_rows<1>(a, gate, f32, stream);
  if (a.m <= 32) return launch_rows<2>(a, gate, f32, stream);
  return launch_rows<4>(a, gate, f32, stream);
}

}  // namespace moe
