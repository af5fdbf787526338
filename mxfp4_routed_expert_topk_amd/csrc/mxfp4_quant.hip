// MXFP4 quantisation of a matrix and the values its codes stand for.
//
// Quantiser, per 32 consecutive elements of a row (the OCP Microscaling v1.0
// rule for E2M1, whose largest power of two is 4 = 2^2):
//   e = clamp(floor(log2(amax)) - 2, -125, 125), -125 for a block of zeros;
//   code = nearest-even E2M1 of x 2^-e, saturated to +-6;  byte = e + 127.
// The clamp keeps every byte in 2..252, which moe_mxfp4_plan accepts for both
// activation types: the bf16 values stay normal and finite.  For a normal amax
// the byte is its fp32 exponent field minus 2, so no logarithm is taken.
// x 2^-e is exact in fp32 (a power of two; an element that underflows is far
// below half a step), so codes and bytes have one right answer.  A block that
// holds a NaN or an infinity gets byte 0xFF (E8M0's NaN) and codes 0: the plan
// refuses it by name, a product with it gives NaN.
//
// Four lanes share a block: each loads 8 elements (16 or 32 bytes, adjacent
// lanes adjacent addresses), the block's amax is two shuffles away, and each
// lane stores one dword of codes.
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPerLane = 8;              // elements per lane: one dword of codes
// A launch holds fewer than 2^32 threads; a lane past kMaxBlocks workgroups'
// takes its turn in a loop.
constexpr long long kMaxBlocks = 1 << 23;

unsigned blocks_for(long long lanes) {
  const long long b = (lanes + kThreads - 1) / kThreads;
  return (unsigned)(b < kMaxBlocks ? b : kMaxBlocks);
}

__device__ __forceinline__ void load8(const uint16_t* p, uint32_t (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = d[i] << 16;
    v[2 * i + 1] = d[i] & 0xFFFF0000u;
  }
}
__device__ __forceinline__ void load8(const float* p, uint32_t (&v)[8]) {
  const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
  const uint32_t d[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = d[i];
}

// STRIDED: rows of lanes_per_row lanes lie ld elements apart; else the matrix is contiguous.
template <class T, bool STRIDED>
__global__ __launch_bounds__(kThreads) void quant_mxfp4(const T* __restrict__ x, long long lanes, int lanes_per_row,
                                                        long long ld, uint32_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
  // a block's four lanes stay together: lanes and the stride are multiples of 4
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < lanes; i += (long long)gridDim.x * kThreads) {
    long long at = i * kPerLane;
    if constexpr (STRIDED) {
      const long long row = i / lanes_per_row;
      at = row * ld + (i - row * lanes_per_row) * kPerLane;
    }
    uint32_t v[8];
    load8(x + at, v);
    uint32_t amax = 0;                     // as bits: a NaN ranks above every finite value
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, v[j] & 0x7FFFFFFFu);
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1, kWave));
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2, kWave));
    const bool bad = amax >= 0x7F800000u;
    const int byte = max((int)(amax >> 23) - 2, 2);
    const float scale = __uint_as_float((uint32_t)byte << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v[0]), __uint_as_float(v[1]), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v[2]), __uint_as_float(v[3]), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v[4]), __uint_as_float(v[5]), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v[6]), __uint_as_float(v[7]), scale, 3);
    codes[i] = bad ? 0u : c;
    if ((threadIdx.x & 3) == 0) scales[i >> 2] = bad ? 0xFFu : (uint8_t)byte;
  }
}

// E8M0 byte -> its value: 2^(b-127) (byte 0 is the subnormal 2^-127), NaN for 0xFF.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : b == 0xFFu ? 0x7FC00000u : b << 23);
}

// A code times its scale is exact in fp32 and in bf16 (two significant bits;
// 4 and 6 times 2^127 overflow to infinity in both), so bf16 takes the upper
// half of the fp32 value.  A lane makes 16 bytes of output (8 bf16 or 4 fp32
// values), so that a wave's store is 1 KB of whole lines.  STREAM: an output
// beyond the L2s passes the caches by (16384 x 7168: 62 -> 41 us, 7.1 TB/s).
template <bool F32, bool STREAM>
__global__ __launch_bounds__(kThreads) void dequant_mxfp4(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, long long lanes,
                                                          uint4* __restrict__ out) {
  constexpr int kN = F32 ? 4 : 8;        // elements per lane
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < lanes; i += (long long)gridDim.x * kThreads) {
    uint32_t c;
    if constexpr (F32) c = reinterpret_cast<const uint16_t*>(codes)[i];
    else c = reinterpret_cast<const uint32_t*>(codes)[i];
    const float s = e8m0_value(scales[i / (32 / kN)]);
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    uint32_t v[kN];
    auto pair = [&](int j, f32x2_t p) {
      v[2 * j] = __float_as_uint(p[0] * s);
      v[2 * j + 1] = __float_as_uint(p[1] * s);
    };
    pair(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0));
    pair(1, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1));
    u32x4_t o;
    if constexpr (F32) {
      o = u32x4_t{v[0], v[1], v[2], v[3]};
    } else {
      pair(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2));
      pair(3, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3));
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = (v[2 * j] >> 16) | (v[2 * j + 1] & 0xFFFF0000u);
    }
    if constexpr (STREAM) __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>(out) + i);
    else reinterpret_cast<u32x4_t*>(out)[i] = o;
  }
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, bool f32, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                                 uint8_t* scales, hipStream_t stream) {
  const long long per_row = cols / kPerLane, lanes = rows * per_row;
  const dim3 grid(blocks_for(lanes));
  uint32_t* const c = reinterpret_cast<uint32_t*>(codes);
  auto run = [&](auto* src) {
    using T = std::remove_pointer_t<decltype(src)>;
    if (ld == cols || rows == 1)
      hipLaunchKernelGGL((quant_mxfp4<std::remove_const_t<T>, false>), grid, dim3(kThreads), 0, stream, src, lanes,
                         (int)per_row, ld, c, scales);
    else
      hipLaunchKernelGGL((quant_mxfp4<std::remove_const_t<T>, true>), grid, dim3(kThreads), 0, stream, src, lanes,
                         (int)per_row, ld, c, scales);
  };
  if (f32) run(static_cast<const float*>(x));
  else run(static_cast<const uint16_t*>(x));
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, bool f32,
                                   void* out, hipStream_t stream) {
  const long long lanes = rows * cols / (f32 ? 4 : 8);
  const dim3 grid(blocks_for(lanes));
  const bool stream_out = lanes * 16 > (long long)kL2Bytes;
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, codes, scales, lanes, static_cast<uint4*>(out));
  };
  if (f32) run(stream_out ? dequant_mxfp4<true, true> : dequant_mxfp4<true, false>);
  else run(stream_out ? dequant_mxfp4<false, true> : dequant_mxfp4<false, false>);
  return hipGetLastError();
}

}  // namespace moe
