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
#include <type_traits>

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

// ---- many rows: BM x BN output tiles, operands staged through LDS.
//
// One stage is 128 K: 64 bytes of codes per row, copied global -> LDS by
// buffer_load ... lds (16 rows per wave instruction) into a ring of four
// stages, three ahead.  The four 16-byte chunks of a staged row are permuted
// by chunk ^ ((row >> 2) & 3): the sixteen rows of a quarter-wave's
// ds_read_b128 then cover all 64 banks once.  Copies past an edge get an
// out-of-range offset and write zeros.
// A group of four stages (512 K) has 16 scale bytes per row.  Thread t loads
// those of row t one group ahead, transposes them to four dwords (dword q:
// the bytes of blocks q, q + 4, q + 8, q + 12, that is lane quarter q's
// scales of the four stages) and stores them in LDS; a wave reads one dword
// per lane, 16-row block and group, and each stage's MFMA picks its byte.
typedef __attribute__((address_space(3))) void lds_void_t;

constexpr int kRing = 4;
constexpr uint32_t kPastEnd = 0x80000000u;   // beyond every buffer resource below

#define MOE_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | ((((n) >> 4) & 3) << 14))

__device__ __forceinline__ int swz4(int c, int r) { return c ^ ((r >> 2) & 3); }

template <int BM_, int BN_, int WM_, int WN_>
struct MxShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, kWaves = WM * WN;
  static constexpr int MI = BM / WM / 16, NJ = BN / WN / 16;
  static constexpr int kRows = BM + BN;                 // staged rows: A's, then B's
  static constexpr int kStageBytes = kRows * 64;
  static constexpr int kCopies = kRows / 16 / kWaves;   // copies per wave and stage
  static constexpr int kScaleBytes = kRows * 16;        // one group
  static constexpr int kSmem = kRing * kStageBytes + 2 * kScaleBytes;
  static_assert(kCopies * kWaves * 16 == kRows && (BM / 16) % kWaves == 0 && kRows % (kWaves * kWave) == 0, "even split");
};

// the four dwords of a row's 16 scale bytes: dword q holds bytes q, 4 + q, 8 + q, 12 + q
__device__ __forceinline__ u32x4_t transpose4(u32x4_t v) {
  const uint32_t a = __builtin_amdgcn_perm(v[1], v[0], 0x05010400u), b = __builtin_amdgcn_perm(v[3], v[2], 0x05010400u);
  const uint32_t c = __builtin_amdgcn_perm(v[1], v[0], 0x07030602u), d = __builtin_amdgcn_perm(v[3], v[2], 0x07030602u);
  return u32x4_t{__builtin_amdgcn_perm(b, a, 0x05040100u), __builtin_amdgcn_perm(b, a, 0x07060302u),
                 __builtin_amdgcn_perm(d, c, 0x05040100u), __builtin_amdgcn_perm(d, c, 0x07060302u)};
}

template <int OP>
__device__ __forceinline__ f32x4_t mfma_fp4_sel(u32x4_t b, u32x4_t a, f32x4_t c, uint32_t sb, uint32_t sa) {
  const i32x8_t B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  const i32x8_t A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(B, A, c, 4, 4, OP, (int)sb, OP, (int)sa);
}

template <class C, bool F32>
__device__ __forceinline__ void matmul_tile(uint8_t* smem, const uint8_t* ac, const uint8_t* as, const uint8_t* bc,
                                            const uint8_t* bs, int M, int N, int groups, int tm, int tn, void* out) {
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  // workgroups go to the XCDs in turn: XCD x takes the x-th eighth of the
  // tiles, walked in bands of eight tile rows so that its concurrent tiles
  // share operand panels in its L2
  const int total = tm * tn, chunk = (total + kXcds - 1) / kXcds;
  const int id = (int)(blockIdx.x % kXcds) * chunk + (int)(blockIdx.x / kXcds);
  if ((int)(blockIdx.x / kXcds) >= chunk || id >= total) return;
  constexpr int kBand = 8;
  const int band = id / (kBand * tn), in = id - band * kBand * tn;
  const int high = min(kBand, tm - band * kBand);
  const int m0 = (band * kBand + in % high) * C::BM, n0 = in / high * C::BN;
  const int mrows = min(C::BM, M - m0), nrows = min(C::BN, N - n0);
  const uint32_t pitch = (uint32_t)groups * 16;   // bytes of a row's codes
  const int stages = (groups + 3) / 4;

  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(ac) + (size_t)m0 * pitch, (short)0, (int)(mrows * pitch), kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(bc) + (size_t)n0 * pitch, (short)0, (int)(nrows * pitch), kRsrcWord3);
  // copy j of this wave fills staged rows 16 (wave + kWaves j) ..; the first BM rows are A's
  constexpr int kCopiesA = C::BM / 16 / C::kWaves;
  uint32_t off[C::kCopies];
  int chunk_of[C::kCopies];
#pragma unroll
  for (int j = 0; j < C::kCopies; ++j) {
    const int r = 16 * (wave + C::kWaves * j) + (lane >> 2) - (j < kCopiesA ? 0 : C::BM);
    chunk_of[j] = swz4(lane & 3, r);
    off[j] = r < (j < kCopiesA ? mrows : nrows) ? (uint32_t)r * pitch + 16 * chunk_of[j] : kPastEnd;
  }
  auto issue = [&](int slot, int s) {
#pragma unroll
    for (int j = 0; j < C::kCopies; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          j < kCopiesA ? ra : rb, (lds_void_t*)(smem + slot * C::kStageBytes + (wave + C::kWaves * j) * 1024), 16,
          4 * s + chunk_of[j] < groups ? off[j] : kPastEnd, s < stages ? s * 64 : 0, 0, 0);
  };
  // scales: kPer rows per thread, 16 bytes each
  constexpr int kPer = C::kRows / (C::kWaves * kWave);
  const uint8_t* srow[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = t + i * C::kWaves * kWave;
    srow[i] = r < C::BM ? as + (size_t)(m0 + min(r, mrows - 1)) * groups
                        : bs + (size_t)(n0 + min(r - C::BM, nrows - 1)) * groups;
  }
  uint8_t* const sscale = smem + kRing * C::kStageBytes;
  u32x4_t sreg[kPer];
  auto load_scales = [&](int g) {   // a whole group
#pragma unroll
    for (int i = 0; i < kPer; ++i) __builtin_memcpy(&sreg[i], srow[i] + 16 * g, 16);
  };
  auto load_last_scales = [&](int g) {   // fewer than 16 blocks: the others as 2^0 (times zeros)
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        uint32_t w = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int at = 16 * g + 4 * d + b;
          w |= (at < groups ? (uint32_t)srow[i][min(at, groups - 1)] : 127u) << (8 * b);
        }
        sreg[i][d] = w;
      }
  };
  auto store_scales = [&](int g) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      *reinterpret_cast<u32x4_t*>(sscale + (g & 1) * C::kScaleBytes + (t + i * C::kWaves * kWave) * 16) = transpose4(sreg[i]);
  };

  const int wm = wave / C::WN, wn = wave % C::WN;
  const int rl = lane & 15, q = lane >> 4;
  const int arow = wm * (16 * C::MI) + rl, brow = C::BM + wn * (16 * C::NJ) + rl;
  f32x4_t acc[C::MI][C::NJ];
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int full = groups / 16;   // groups of four whole stages
  if (full) load_scales(0);
  else load_last_scales(0);
  store_scales(0);
#pragma unroll
  for (int d = 0; d < kRing - 1; ++d) issue(d, d);

  uint32_t sa[C::MI], sb[C::NJ];
  auto run_stage = [&](auto jc, int g) {
    constexpr int j4 = decltype(jc)::value;
    const int s = 4 * g + j4;
    // this wave's copies of stage s have landed (two stages' copies came after
    // them; a scale load among those only makes the wait stricter) and its
    // LDS accesses are done; the barrier extends both to every wave
    MOE_WAIT_VM(2 * C::kCopies);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (j4 == 0 && g + 1 < full) load_scales(g + 1);
    issue((j4 + kRing - 1) % kRing, s + kRing - 1);
    if (j4 == 0) {
      const uint8_t* sc = sscale + (g & 1) * C::kScaleBytes + q * 4;
#pragma unroll
      for (int i = 0; i < C::MI; ++i) sa[i] = *reinterpret_cast<const uint32_t*>(sc + (arow + 16 * i) * 16);
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) sb[j] = *reinterpret_cast<const uint32_t*>(sc + (brow + 16 * j) * 16);
    }
    const uint8_t* buf = smem + j4 * C::kStageBytes;
    u32x4_t fb[C::NJ], fa[C::MI];
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
      fb[j] = *reinterpret_cast<const u32x4_t*>(buf + (brow + 16 * j) * 64 + swz4(q, rl) * 16);
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
      fa[i] = *reinterpret_cast<const u32x4_t*>(buf + (arow + 16 * i) * 64 + swz4(q, rl) * 16);
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) acc[i][j] = mfma_fp4_sel<j4>(fb[j], fa[i], acc[i][j], sb[j], sa[i]);
    if (j4 == 3 && g + 1 < full) store_scales(g + 1);
    // the stage's MFMAs stay in their stage (left free, the compiler collects
    // several stages' operands first and spills)
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) pin(acc[i][j][0]);
  };
  for (int g = 0; g < full; ++g) {
    run_stage(std::integral_constant<int, 0>{}, g);
    run_stage(std::integral_constant<int, 1>{}, g);
    run_stage(std::integral_constant<int, 2>{}, g);
    run_stage(std::integral_constant<int, 3>{}, g);
  }
  if (4 * full < stages) {   // K is not a multiple of 512
    if (full) {
      load_last_scales(full);
      store_scales(full);
    }
    run_stage(std::integral_constant<int, 0>{}, full);
    if (4 * full + 1 < stages) run_stage(std::integral_constant<int, 1>{}, full);
    if (4 * full + 2 < stages) run_stage(std::integral_constant<int, 2>{}, full);
    if (4 * full + 3 < stages) run_stage(std::integral_constant<int, 3>{}, full);
  }
  MOE_WAIT_VM(0);   // the copies past the end still write LDS

  // lane holds row rl, columns 4q .. 4q + 3 of each 16 x 16 block
#pragma unroll
  for (int i = 0; i < C::MI; ++i) {
    const int m = wm * (16 * C::MI) + 16 * i + rl;
    if (m >= mrows) continue;
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) {
      const int n = wn * (16 * C::NJ) + 16 * j + 4 * q;
      const size_t at = (size_t)(m0 + m) * N + n0 + n;
      if (!F32 && N % 4 == 0) {
        if (n < nrows)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
              make_uint2(f32_to_bf16_rne(acc[i][j][0]) | ((uint32_t)f32_to_bf16_rne(acc[i][j][1]) << 16),
                         f32_to_bf16_rne(acc[i][j][2]) | ((uint32_t)f32_to_bf16_rne(acc[i][j][3]) << 16));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (n + e >= nrows) break;
          if (F32) static_cast<float*>(out)[at + e] = acc[i][j][e];
          else static_cast<uint16_t*>(out)[at + e] = f32_to_bf16_rne(acc[i][j][e]);
        }
      }
    }
  }
}

template <class C, bool F32>
__global__ __launch_bounds__(C::kWaves* kWave) void matmul_mxfp4_tiles(const uint8_t* ac, const uint8_t* as,
                                                                       const uint8_t* bc, const uint8_t* bs, int M, int N,
                                                                       int groups, int tm, int tn, void* out) {
  __shared__ __align__(1024) uint8_t smem[C::kSmem];
  matmul_tile<C, F32>(smem, ac, as, bc, bs, M, N, groups, tm, tn, out);
}

template <class C>
hipError_t launch_tiles(const uint8_t* ac, const uint8_t* as, const uint8_t* bc, const uint8_t* bs, int M, int N, int K,
                        bool f32, void* out, hipStream_t stream) {
  const int tm = (M + C::BM - 1) / C::BM, tn = (N + C::BN - 1) / C::BN;
  const dim3 grid((unsigned)(((long long)tm * tn + kXcds - 1) / kXcds * kXcds)), block(C::kWaves * kWave);
  if (f32)
    hipLaunchKernelGGL((matmul_mxfp4_tiles<C, true>), grid, block, 0, stream, ac, as, bc, bs, M, N, K / 32, tm, tn, out);
  else
    hipLaunchKernelGGL((matmul_mxfp4_tiles<C, false>), grid, block, 0, stream, ac, as, bc, bs, M, N, K / 32, tm, tn, out);
  return hipGetLastError();
}

using Mx256 = MxShape<256, 256, 2, 4>;

}  // namespace

hipError_t launch_mxfp4_matmul(const uint8_t* ac, const uint8_t* as, const uint8_t* bc, const uint8_t* bs, int M, int N,
                               int K, bool f32, void* out, hipStream_t stream) {
  if (M > 128) return launch_tiles<Mx256>(ac, as, bc, bs, M, N, K, f32, out, stream);
  const dim3 grid((N + 15) / 16, (M + 15) / 16);
  if (f32) hipLaunchKernelGGL(matmul_mxfp4<true>, grid, dim3(kSplit * kWave), 0, stream, ac, as, bc, bs, M, N, K / 32, out);
  else hipLaunchKernelGGL(matmul_mxfp4<false>, grid, dim3(kSplit * kWave), 0, stream, ac, as, bc, bs, M, N, K / 32, out);
  return hipGetLastError();
}

}  // namespace moe
