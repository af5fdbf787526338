// Product of two MXFP4 matrices, y [M, N] = A [M, K] B [N, K]^T:
//   y[m, n] = sum over blocks g of 32 K of  2^(ea + eb) sum_i a_i b_i
// on v_mfma_scale_f32_16x16x128_f8f6f4 with both operands E2M1.  A block's 32
// products are multiples of 1/4 and their sum is exact; the instruction adds
// the blocks to an fp32 accumulator (checked against 64 bits: the error of a
// step is below 2^-20 of its largest term, an E8M0 byte 0xFF gives NaN and
// byte 0 counts as 2^-127).
//
// Operand order of the instruction: lane l holds row l%16 and the 32
// consecutive K values 32 (l/16) + [0, 32) of each operand, with the scale of
// exactly that block: 16 contiguous bytes and one byte of the row-major
// matrices.  B goes in as the first operand, so a lane ends with four
// consecutive columns n of one row m.
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kSplit = 4;   // waves per workgroup, each a share of K

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4_t mfma_fp4(u32x4_t b, u32x4_t a, f32x4_t c, int sb, int sa) {
  const i32x8_t B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  const i32x8_t A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(B, A, c, 4, 4, 0, sb, 0, sa);
}

// One workgroup per 16 x 16 outputs.  groups: K / 32.
template <bool F32>
__global__ __launch_bounds__(kSplit* kWave) void matmul_mxfp4(const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as,
                                                              const uint8_t* __restrict__ bc, const uint8_t* __restrict__ bs,
                                                              int M, int N, int groups, void* __restrict__ out) {
  __shared__ f32x4_t part[kSplit - 1][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
  // rows past the matrix repeat its last row and are not stored
  const size_t arow = (size_t)min(m0 + r, M - 1) * groups, brow = (size_t)min(n0 + r, N - 1) * groups;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  const int steps = (groups + 3) / 4;
  for (int s = wave; s < steps; s += kSplit) {
    const int g = 4 * s + q;             // this lane's block of 32
    u32x4_t a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
    int sa = 127, sb = 127;
    if (g < groups) {
      a = *reinterpret_cast<const u32x4_t*>(ac + (arow + g) * 16);
      b = *reinterpret_cast<const u32x4_t*>(bc + (brow + g) * 16);
      sa = as[arow + g];
      sb = bs[brow + g];
    }
    acc = mfma_fp4(b, a, acc, sb, sa);
  }
  if (wave) part[wave - 1][lane] = acc;
  __syncthreads();
  if (wave) return;
  for (int w = 0; w < kSplit - 1; ++w) acc += part[w][lane];
  const int m = m0 + r;
  if (m >= M) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + 4 * q + i;
    if (n >= N) break;
    if (F32) static_cast<float*>(out)[(size_t)m * N + n] = acc[i];
    else static_cast<uint16_t*>(out)[(size_t)m * N + n] = f32_to_bf16_rne(acc[i]);
  }
}

}  // namespace

hipError_t launch_mxfp4_matmul(const uint8_t* ac, const uint8_t* as, const uint8_t* bc, const uint8_t* bs, int M, int N,
                               int K, bool f32, void* out, hipStream_t stream) {
  const dim3 grid((N + 15) / 16, (M + 15) / 16);
  if (f32) hipLaunchKernelGGL(matmul_mxfp4<true>, grid, dim3(kSplit * kWave), 0, stream, ac, as, bc, bs, M, N, K / 32, out);
  else hipLaunchKernelGGL(matmul_mxfp4<false>, grid, dim3(kSplit * kWave), 0, stream, ac, as, bc, bs, M, N, K / 32, out);
  return hipGetLastError();
}

}  // namespace moe
