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

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4_t mfma_fp4(u32x4_t b, u32x4_t a, f32x4_t c, int sb, int sa) {
  const i32x8_t B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  const i32x8_t A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(B, A, c, 4, 4, 0, sb, 0, sa);
}

// ---- few rows: B is streamed once per 16 MT rows of A.
//
// A workgroup owns 16 columns and MT 16-row blocks; its kSplit waves take 256
// K at a time in turn and their partial sums are added in wave order.  In 256
// K a lane takes the 32 contiguous bytes of blocks 2q and 2q + 1 (of A alike),
// one MFMA step each, so that a row's 128 bytes are fetched as a whole line;
// which blocks share a step does not matter to the sum.  Two such units are
// in flight per wave.
constexpr int kSplit = 8;

// 16 bytes of codes, a chunk past K as zeros with scale 2^0
struct Operand4 {
  u32x4_t v[2];
  int s[2];
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, size_t row, int unit, int q, int groups) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int g = 8 * unit + 2 * q + i;
      v[i] = u32x4_t{0, 0, 0, 0};
      s[i] = 127;
      if (g < groups) {
        v[i] = *reinterpret_cast<const u32x4_t*>(codes + (row * groups + g) * 16);
        s[i] = scales[row * groups + g];
      }
    }
  }
};

// groups: K / 32
template <int MT, bool F32>
__global__ __launch_bounds__(kSplit* kWave) void matmul_mxfp4_rows(const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as,
                                                                   const uint8_t* __restrict__ bc, const uint8_t* __restrict__ bs,
                                                                   int M, int N, int groups, void* __restrict__ out) {
  __shared__ f32x4_t part[kSplit][MT][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * (16 * MT);
  // rows past the matrix repeat its last row and are not stored
  const size_t brow = min(n0 + r, N - 1);
  f32x4_t acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int units = (groups + 7) / 8;
  for (int u = wave; u < units; u += 2 * kSplit) {
    Operand4 b[2], a[2][MT];
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      b[d].load(bc, bs, brow, u + d * kSplit, q, groups);
#pragma unroll
      for (int i = 0; i < MT; ++i) a[d][i].load(ac, as, min(m0 + 16 * i + r, M - 1), u + d * kSplit, q, groups);
    }
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = mfma_fp4(b[d].v[h], a[d][i].v[h], acc[i], b[d].s[h], a[d][i].s[h]);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave >= MT) return;   // wave i adds and stores row block i
  f32x4_t v = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < kSplit; ++w) v += part[w][wave][lane];
  const int m = m0 + 16 * wave + r, n = n0 + 4 * q;
  if (m >= M) return;
  const size_t at = (size_t)m * N + n;
  if (N % 4 == 0) {
    if (n >= N) return;
    if constexpr (F32) *reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + at) = v;
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
        make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (n + e >= N) break;
    if (F32) static_cast<float*>(out)[at + e] = v[e];
    else static_cast<uint16_t*>(out)[at + e] = f32_to_bf16_rne(v[e]);
  }
}

// ---- many rows: BM x BN output tiles, operands staged through LDS.
//
// One stage is 256 K: 128 bytes of codes per row, whole cache lines, copied
// global -> LDS by buffer_load ... lds (8 rows per wave instruction) into one
// of two buffers while the other multiplies.  (With 128 K a stage, half lines,
// the copies took 62 us against 59 at 4096 x 4096 x 7168.)  The eight 16-byte
// chunks of a staged row are permuted by chunk ^ (row >> 1): the sixteen lanes
// that ds_read_b128 serves at once, eight rows of one chunk and the other eight
// of its neighbour (lanes 0-3, 12-15, 20-27), then cover all 64 banks
// once.  Copies past an edge get an out-of-range offset and write zeros.
// A pair of stages (512 K) has 16 scale bytes per row.  Thread t loads those
// of row t one pair ahead, transposes them to four dwords (dword q: the bytes
// of blocks q, q + 4, q + 8, q + 12, that is lane quarter q's scales of the
// pair's four MFMA steps) and stores them in LDS; a wave reads one dword per
// lane, 16-row block and pair, and each step's MFMA picks its byte.
typedef __attribute__((address_space(3))) void lds_void_t;

constexpr uint32_t kPastEnd = 0x80000000u;   // beyond every buffer resource below

#define MOE_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | ((((n) >> 4) & 3) << 14))

__device__ __forceinline__ int swz(int c, int r) { return c ^ ((r >> 1) & 7); }

template <int BM_, int BN_, int WM_, int WN_>
struct MxShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, kWaves = WM * WN;
  static constexpr int MI = BM / WM / 16, NJ = BN / WN / 16;
  static constexpr int kRows = BM + BN;                 // staged rows: A's, then B's
  static constexpr int kStageBytes = kRows * 128;
  static constexpr int kCopies = kRows / 8 / kWaves;    // copies per wave and stage
  static constexpr int kScaleBytes = kRows * 16;        // one pair of stages
  static constexpr int kSmem = 2 * kStageBytes + 2 * kScaleBytes;
  static_assert(kCopies * kWaves * 8 == kRows && (BM / 8) % kWaves == 0 && kWaves % 2 == 0 && kRows == kWaves * kWave && BM % kWave == 0, "even split");
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
  // whole pairs of stages: what is past K multiplies zeros
  const int pairs = (groups + 15) / 16;

  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(ac) + (size_t)m0 * pitch, (short)0, (int)(mrows * pitch), kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(bc) + (size_t)n0 * pitch, (short)0, (int)(nrows * pitch), kRsrcWord3);
  // copy j of this wave fills staged rows 8 (wave + kWaves j) ..; the first BM rows are A's
  constexpr int kCopiesA = C::BM / 8 / C::kWaves;
  uint32_t off[C::kCopies];
  const int chunk_of = swz(lane & 7, 8 * wave + (lane >> 3));   // the same in every copy: 16 rows apart
#pragma unroll
  for (int j = 0; j < C::kCopies; ++j) {
    const int r = 8 * (wave + C::kWaves * j) + (lane >> 3) - (j < kCopiesA ? 0 : C::BM);
    off[j] = r < (j < kCopiesA ? mrows : nrows) ? (uint32_t)r * pitch + 16 * chunk_of : kPastEnd;
  }
  auto issue = [&](int slot, int s, int j) {   // copy j of stage s
    const bool in = 8 * s + chunk_of < groups;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        j < kCopiesA ? ra : rb, (lds_void_t*)(smem + slot * C::kStageBytes + (wave + C::kWaves * j) * 1024), 16,
        in ? off[j] : kPastEnd, 8 * s < groups ? s * 128 : 0, 0, 0);   // never past the resource by itself
  };
  // scales: thread t's row of the staged ones (a wave's are all A's or all B's)
  const bool of_a = wave < C::BM / kWave;
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(of_a ? as + (size_t)m0 * groups : bs + (size_t)n0 * groups), (short)0,
      (of_a ? mrows : nrows) * groups, kRsrcWord3);
  const uint32_t srow = (uint32_t)(of_a ? min(t, mrows - 1) : min(t - C::BM, nrows - 1)) * groups;
  uint8_t* const sscale = smem + 2 * C::kStageBytes;
  u32x4_t sreg;
  // pair g's 16 bytes of the row; of a last pair that is not whole, the row's last 16
  auto load_scales = [&](int g) { sreg = __builtin_amdgcn_raw_buffer_load_b128(rs, srow, max(min(16 * g, groups - 16), 0), 0); };
  auto load_few_scales = [&] {   // K below 512: byte by byte, those past K as 2^0 (times zeros)
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t w = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int at = 4 * d + b;
        w |= (at < groups ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rs, srow, at, 0) : 127u) << (8 * b);
      }
      sreg[d] = w;
    }
  };
  // moves the last 16 bytes of a row down to where its last pair starts; what
  // follows counts as 2^0 (times zeros)
  auto align_scales = [&](u32x4_t v) {
    const int past = 16 * pairs - groups;   // bytes of the pair before it
#pragma unroll
    for (int w = 0; w < 3; ++w)
      if (4 * w + 4 <= past) v = u32x4_t{v[1], v[2], v[3], 0x7F7F7F7Fu};
    const uint32_t by = past & 3;
    return u32x4_t{__builtin_amdgcn_alignbyte(v[1], v[0], by), __builtin_amdgcn_alignbyte(v[2], v[1], by),
                   __builtin_amdgcn_alignbyte(v[3], v[2], by), __builtin_amdgcn_alignbyte(0x7F7F7F7Fu, v[3], by)};
  };
  auto store_scales = [&](int g) {
    const u32x4_t v = g > 0 && 16 * g + 16 > groups ? align_scales(sreg) : sreg;
    *reinterpret_cast<u32x4_t*>(sscale + (g & 1) * C::kScaleBytes + t * 16) = transpose4(v);
  };

  const int wm = wave / C::WN, wn = wave % C::WN;
  const int rl = lane & 15, q = lane >> 4;
  const int arow = wm * (16 * C::MI) + rl, brow = C::BM + wn * (16 * C::NJ) + rl;
  f32x4_t acc[C::MI][C::NJ];
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (groups >= 16) load_scales(0);
  else load_few_scales();
  store_scales(0);
#pragma unroll
  for (int j = 0; j < C::kCopies; ++j) issue(0, 0, j);

  // A stage has two MFMA steps of 128 K, each two lists: the wave's upper and
  // lower row blocks.  Behind each MFMA stands a share of the LDS reads of the
  // list after it (and, early in the stage, of the next stage's copies), so
  // that no run of reads holds an MFMA up; the last list of a stage runs after
  // the next stage's barrier, over that stage's first reads.  Before the first
  // stage its operands are zeros with scales of 2^0.
  constexpr int kHalf = C::MI / 2, kM = kHalf * C::NJ;
  static_assert(C::MI % 2 == 0 && kM >= C::NJ + kHalf && kM >= C::kCopies, "a list has room for its reads and copies");
  uint32_t sa[C::MI], sb[C::NJ];
  u32x4_t fa[C::MI], fb[2][C::NJ];
#pragma unroll
  for (int i = 0; i < C::MI; ++i) {
    fa[i] = u32x4_t{0, 0, 0, 0};
    sa[i] = 0x7F7F7F7Fu;
  }
#pragma unroll
  for (int j = 0; j < C::NJ; ++j) {
    fb[0][j] = fb[1][j] = u32x4_t{0, 0, 0, 0};
    sb[j] = 0x7F7F7F7Fu;
  }
  auto run_stage = [&](auto pc, int g) {   // stage p of pair g
    constexpr int p = decltype(pc)::value;
    // this wave's copies of the stage have landed and its LDS accesses are
    // done; the barrier extends both to every wave
    MOE_WAIT_VM(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const uint8_t* buf = smem + p * C::kStageBytes;
    const uint8_t* sc = sscale + (g & 1) * C::kScaleBytes + q * 4;
    unrolled<4>([&](auto hc) {
      // list h - 1 (h = 0: the previous stage's last) over the operands of list h
      constexpr int h = decltype(hc)::value, k = h / 2;
      constexpr int pk = (2 * p + (h + 1) / 2 + 3) % 4;   // the step of the list that multiplies, in its pair
      constexpr int pb = pk % 2, lo = (h + 1) % 2;
      const uint8_t* at = buf + swz(4 * k + q, rl) * 16;
      unrolled<kM>([&](auto mc) {
        constexpr int m = decltype(mc)::value, i = lo * kHalf + m / C::NJ, j = m % C::NJ;
        acc[i][j] = mfma_fp4_sel<pk>(fb[pb][j], fa[i], acc[i][j], sb[j], sa[i]);
        if constexpr (h % 2 == 0) {          // B and the upper blocks of step k
          if constexpr (m < C::NJ) {
            fb[k][m] = *reinterpret_cast<const u32x4_t*>(at + (brow + 16 * m) * 128);
          } else if constexpr (m < C::NJ + kHalf) {
            constexpr int r = m - C::NJ;
            fa[r] = *reinterpret_cast<const u32x4_t*>(at + (arow + 16 * r) * 128);
            if constexpr (p == 0 && h == 0) sa[r] = *reinterpret_cast<const uint32_t*>(sc + (arow + 16 * r) * 16);
          }
        } else if constexpr (m < kHalf) {    // its lower blocks
          constexpr int r = kHalf + m;
          fa[r] = *reinterpret_cast<const u32x4_t*>(at + (arow + 16 * r) * 128);
          if constexpr (p == 0 && h == 1) sa[r] = *reinterpret_cast<const uint32_t*>(sc + (arow + 16 * r) * 16);
        }
        if constexpr (h == 0 && m < C::kCopies) issue(1 - p, 2 * g + p + 1, m);
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (p == 0 && h == 0) {
#pragma unroll
        for (int j = 0; j < C::NJ; ++j) sb[j] = *reinterpret_cast<const uint32_t*>(sc + (brow + 16 * j) * 16);
        load_scales(g + 1);
      }
    });
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) pin(acc[i][j][0]);
    if constexpr (p == 1) store_scales(g + 1);   // after the last pair: into the half no one reads
  };
  for (int g = 0; g < pairs; ++g) {
    run_stage(std::integral_constant<int, 0>{}, g);
    run_stage(std::integral_constant<int, 1>{}, g);
  }
  unrolled<kM>([&](auto mc) {   // the last list of the last stage
    constexpr int m = decltype(mc)::value, i = kHalf + m / C::NJ, j = m % C::NJ;
    acc[i][j] = mfma_fp4_sel<3>(fb[1][j], fa[i], acc[i][j], sb[j], sa[i]);
  });
  MOE_WAIT_VM(0);   // the copies past the end still write LDS
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();   // every wave is done reading the ring
  asm volatile("" ::: "memory");

  // Lane holds row rl, columns 4q .. 4q + 3 of each 16 x 16 block.  The wave's
  // blocks pass through its part of the ring, 32 rows at a time, and leave as
  // whole rows of 16-byte chunks (permuted by chunk ^ row for the banks) or,
  // where the output's rows are not 16-byte aligned, of single values, a row's
  // side by side (4096 x 4097 x 1024: 36 us; from the MFMA layout 57).
  constexpr int kSize = F32 ? 4 : 2, kRowBytes = C::NJ * 16 * kSize, kChunks = kRowBytes / 16;
  constexpr int kMask = kChunks < 16 ? kChunks - 1 : 15;
  constexpr int kShift = kRowBytes >= 256 ? 0 : 1;   // rows side by side in the banks
  auto place = [](int r, int c) { return (c ^ ((r >> kShift) & kMask)) * 16; };   // chunk c of row r
  static_assert(C::kWaves * 32 * kRowBytes <= C::kSmem && 64 % kChunks == 0, "two blocks of every wave fit");
  const bool rows_aligned = N % (16 / kSize) == 0;
  uint8_t* const stg = smem + wave * (32 * kRowBytes);
  const int mw = wm * (16 * C::MI), nw = wn * (16 * C::NJ);
#pragma unroll
  for (int i = 0; i < C::MI; i += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) {
        const f32x4_t v = acc[i + h][j];
        uint8_t* const at = stg + (16 * h + rl) * kRowBytes;
        if constexpr (F32)
          *reinterpret_cast<f32x4_t*>(at + place(rl, 4 * j + q)) = v;
        else
          *reinterpret_cast<uint2*>(at + place(rl, 2 * j + (q >> 1)) + 8 * (q & 1)) =
              make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
      }
    asm volatile("" ::: "memory");
    if (rows_aligned) {
#pragma unroll
      for (int k = 0; k < kChunks / 2; ++k) {   // 64 / kChunks rows at a time
        const int r = k * (64 / kChunks) + lane / kChunks, c = lane % kChunks;
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(stg + r * kRowBytes + place(r, c));
        const int m = mw + 16 * i + r, n = nw + c * (16 / kSize);
        if (m < mrows && n < nrows)
          *reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(out) + ((size_t)(m0 + m) * N + n0 + n) * kSize) = v;
      }
    } else {
      using V = std::conditional_t<F32, float, uint16_t>;
      static_assert(C::NJ * 16 == kWave, "a row a wave");
      const int n = nw + lane, c = lane / (16 / kSize);
      for (int r = 0; r < 32 && mw + 16 * i + r < mrows; ++r) {
        const V v = *reinterpret_cast<const V*>(stg + r * kRowBytes + place(r, c) + lane % (16 / kSize) * kSize);
        if (n < nrows) static_cast<V*>(out)[(size_t)(m0 + mw + 16 * i + r) * N + n0 + n] = v;
      }
    }
    asm volatile("" ::: "memory");
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
using Mx128 = MxShape<128, 128, 2, 2>;

template <int MT>
hipError_t launch_rows(const uint8_t* ac, const uint8_t* as, const uint8_t* bc, const uint8_t* bs, int M, int N, int K,
                       bool f32, void* out, hipStream_t stream) {
  const dim3 grid((N + 15) / 16, (M + 16 * MT - 1) / (16 * MT)), block(kSplit * kWave);
  if (f32)
    hipLaunchKernelGGL((matmul_mxfp4_rows<MT, true>), grid, block, 0, stream, ac, as, bc, bs, M, N, K / 32, out);
  else
    hipLaunchKernelGGL((matmul_mxfp4_rows<MT, false>), grid, block, 0, stream, ac, as, bc, bs, M, N, K / 32, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mxfp4_matmul(const uint8_t* ac, const uint8_t* as, const uint8_t* bc, const uint8_t* bs, int M, int N,
                               int K, bool f32, void* out, hipStream_t stream) {
  // Row blocks per workgroup of the streaming kernel: the fewest whose
  // workgroups still fit one to a CU (K 7168 to 4096 columns, 32 rows: 14.5,
  // 11.3, 12.9 us with 1, 2, 4; K 4096 to 512, 64 rows: 5.5, 7.3, 10.9).
  const int nb = (N + 15) / 16, mb = (M + 15) / 16;
  const int mt = mb == 1 || nb * mb <= 256 ? 1 : mb == 2 || nb * ((mb + 1) / 2) <= 256 ? 2 : 4;
  // It reads mt + 1 row blocks of K/2 bytes per workgroup from the L2s at about
  // 4.6 TB/s; up to 256 tiles of 128 x 128 take about 4.5 us and 0.4 us per 256
  // K.  The two meet about where the count below does (K 7168 to 4096 columns:
  // 32 rows 11.3 against 16.5 us, 48 rows 15.5 against 16.5, 64 rows 17.9
  // against 16.5; K 2048 to 7168: 17 rows 5.9 against 6.9, 48 rows 10.5 against
  // 7.0; K 480 to 2048: 256 rows 4.3 against 5.2).
  const long long blocks = (long long)nb * ((mb + mt - 1) / mt) * (mt + 1);
  if (blocks <= 900 + 800000 / K) {
    if (mt == 1) return launch_rows<1>(ac, as, bc, bs, M, N, K, f32, out, stream);
    if (mt == 2) return launch_rows<2>(ac, as, bc, bs, M, N, K, f32, out, stream);
    return launch_rows<4>(ac, as, bc, bs, M, N, K, f32, out, stream);
  }
  // 256 x 256 once they fill most of the 256 CUs: half the copies per product
  // (K 7168 to 4096 columns: 2048 rows, 128 large tiles, 49 against 41 us;
  // 4096 rows, 256 of them, 59 against 84; K 2048 to 7168: 2048 rows, 224 of
  // them, 20.8 against 28.9).
  if ((long long)((M + 255) / 256) * ((N + 255) / 256) >= 192)
    return launch_tiles<Mx256>(ac, as, bc, bs, M, N, K, f32, out, stream);
  return launch_tiles<Mx128>(ac, as, bc, bs, M, N, K, f32, out, stream);
}

}  // namespace moe
