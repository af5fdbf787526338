// Product of bf16 rows with an MXFP4 matrix in checkpoint layout,
//   y [M, N] = x [M, K] W [N, K]^T,   W = code 2^(byte - 127)
// and, gated, silu(y[:, c]) y[:, c + N/2] for the fused w1||w3 of a shared
// expert.  A weight has at most two significant bits, so W is exact in bf16
// for every scale byte (0 is 2^-127, 255 NaN; 2^128 and above, of bytes 253 and 254,
// is infinite there as in fp32); products are summed in fp32 on v_mfma_f32_16x16x32_bf16,
// which keeps subnormal operands, and the sum is rounded once.
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void_t;

constexpr uint32_t kPastEnd = 0x80000000u;   // beyond every buffer resource below

// vmcnt <= n and lgkmcnt 0
#define MOE_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | ((((n) >> 4) & 3) << 14))

// silu(g) u of four values.  exp(-g) is infinite in fp32 below -88.7, where silu is a
// number down to -104 and further down its product with a large u: there, where
// 1 + exp(g) is 1, it is g u exp(g), by halves of the exponent, which fp32 holds.
// (One rare branch behind all four: one a value costs 1024 rows of 4096 x 7168
// 62.8 us for 60.6.)
__device__ __forceinline__ f32x4_t gated(f32x4_t g, f32x4_t u) {
  f32x4_t v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = g[e] / (1.f + expf(-g[e])) * u[e];
  if (__ballot(fminf(fminf(g[0], g[1]), fminf(g[2], g[3])) < -64.f)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float half = expf(0.5f * g[e]);
      if (g[e] < -64.f) v[e] = g[e] * half * u[e] * half;
    }
  }
  return v;
}

// ---- few rows: the waves of a workgroup split K.
//
// A workgroup owns MT 16-row blocks of x and RB 16-row blocks of W; each of its
// SPLIT waves has its part of K to itself, in chunks of 128, and their sums are
// added in wave order. No barrier until then; DEPTH chunks are in flight.
//   Everything passes through LDS, because a load serves sixteen consecutive
// lanes at a time and costs a clock for every line that they touch: 64 for the
// MFMA's own order, which has sixteen rows side by side (W and scales loaded so:
// 64 columns of W over 8192 K, 25.7 us a workgroup, 11 GB/s). A copy of x is four
// rows of 256 bytes, one of W sixteen rows of 64; the scales of a workgroup's
// rows, one run of memory, come first and all at once.
//   x: a row's 16-byte pieces are permuted by piece ^ 2 (row & 7), W's by piece ^
// 2 (row >> 3): of the sixteen lanes that ds_read_b128 serves at once, eight rows
// of one piece and the other eight of the next (lanes 0-3, 12-15, 20-27), no two
// then share a bank.
//   Lane quarter q reads the 16 bytes of block q of its row of W; two swaps of
// 32-lane halves and two of 16-lane rows transpose them between the quarters,
// dword q of block j for MFMA step j.
//   With a gate and RB 1 the block is eight rows of w1 and the same eight of w3
// (the lanes of an output's two values are 32 apart), else blocks alternate.
// Byte j of s where the scaled converter reads it: bits 30:23, whatever the
// others hold (checked for every byte).
__device__ __forceinline__ float scale_byte(uint32_t s, int j) { return __uint_as_float(j < 3 ? s << (23 - 8 * j) : s >> 1); }

// dword i of quarter q's lanes to dword q of quarter i's
__device__ __forceinline__ void transpose_quarters(u32x4_t& v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  v = u32x4_t{c[0], c[1], d[0], d[1]};
}

// COPIES: of x for a chunk, four rows each.
// GROUPS: the most scales a row has here.
template <int MT, int RB, int SPLIT, int DEPTH, int COPIES, int GROUPS, bool GATE>
__device__ __forceinline__ void linear_rows_block(uint8_t* smem, uint32_t* scale, const LinearArgs& a, bool f32) {
  constexpr int kXBytes = COPIES * 1024, kPlace = kXBytes + RB * 1024;   // a chunk of x, and of W behind it
  constexpr int kCols = GATE ? 8 * RB : 16 * RB;   // output columns
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int cols = GATE ? a.n / 2 : a.n, groups = a.k / 32, c0 = blockIdx.x * kCols, m0 = blockIdx.y * (16 * MT);
  const int chunks = (groups + 3) / 4, per = (chunks + SPLIT - 1) / SPLIT;
  const int first = wave * per, mine = min(max(chunks - first, 0), per);   // the wave's chunks
  // row of W of a block's row i; columns past the matrix repeat its last and are not stored
  auto matrix_row = [&](int b, int i) {
    const int col = c0 + (GATE ? (RB == 1 ? i & 7 : 16 * (b >> 1) + i) : 16 * b + i);
    return min(col, cols - 1) + (GATE ? (RB == 1 ? i >> 3 : b & 1) * cols : 0);
  };

  // Scales: dword d of row i holds blocks 4 d .. 4 d + 3, those past K as 0 (2^-127).
  const int scales = a.n * groups;
  const __amdgpu_buffer_rsrc_t ss =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.scales), (short)0, scales, kRsrcWord3);
  constexpr int kLine = SPLIT * kWave / 16, kTurns = GROUPS / 4 / kLine;   // thread -> row, and every kLine-th dword of it
  uint32_t sv[RB][kTurns];
  const int srow = threadIdx.x / kLine, sd = threadIdx.x % kLine;
  auto scale_at = [&](int b, int j) { return matrix_row(b, srow) * groups + 4 * (sd + kLine * j); };
#pragma unroll
  for (int j = 0; j < kTurns; ++j)
    if (kLine * j < chunks) {
#pragma unroll
      for (int b = 0; b < RB; ++b)   // the matrix may end inside a dword: its last four bytes then
        sv[b][j] = __builtin_amdgcn_raw_buffer_load_b32(ss, min(scale_at(b, j), scales - 4), 0, 0);
    }

  // Copies of x: lane -> row 4 t + lane / 16 and a piece of it. Rows past the
  // matrix read as zeros, and so does what is past K.
  const int mrows = min(16 * MT, a.m - m0);
  const uint16_t* const xbase = a.x + (size_t)m0 * a.ldx;
  const int xrange = (int)(((mrows - 1) * a.ldx + a.k) * 2);
  auto xpiece = [&](int t) { return r ^ (2 * ((4 * t + q) & 7)); };
  uint32_t xoff[COPIES];
#pragma unroll
  for (int t = 0; t < COPIES; ++t)
    xoff[t] = 4 * t + q < mrows ? (uint32_t)((4 * t + q) * a.ldx * 2) + 16 * xpiece(t) : kPastEnd;
  uint8_t* const ring = smem + wave * DEPTH * kPlace;
  // W's copies: lane -> row lane / 4, piece lane % 4 in its place. With a gate, w1
  // and w3 have a resource each, but with RB 1 one reaches both, from w1's first row of the
  // block to the end of w3's eighth: (n / 2 + 8) pitch bytes, which the launcher keeps below 2^31.
  const uint32_t pitch = (uint32_t)groups * 16;
  constexpr int kHalves = GATE && RB > 1 ? 2 : 1;
  const int wpiece = (lane & 3) ^ (2 * (lane >> 5));
  uint32_t woff[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b)
    woff[b] = (uint32_t)(matrix_row(b, lane >> 2) - matrix_row(b % kHalves, 0)) * pitch + 16 * wpiece;
  auto issue = [&](auto whole, int d, int c) {   // chunk c into place d; one that K ends in or before is not whole
    uint8_t* const to = ring + d * kPlace;
    const int c_ = whole ? c : 0;   // else offsets count from the rows' start
    __amdgpu_buffer_rsrc_t ws[kHalves];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
      ws[h] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.codes) + (size_t)matrix_row(h, 0) * pitch + 64 * c_,
                                                (short)0, 0x7FFFFFFF, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t xs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(xbase) + 128 * c_, (short)0,
                                                                        xrange - 256 * c_, kRsrcWord3);
    auto copy_w = [&](int b, uint32_t at) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ws[b % kHalves], (lds_void_t*)(to + kXBytes + b * 1024), 16, at, 0, 0, 0);
    };
    auto copy_x = [&](int t, uint32_t at) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xs, (lds_void_t*)(to + t * 1024), 16, at, 0, 0, 0);
    };
    if constexpr (whole) {
#pragma unroll
      for (int b = 0; b < RB; ++b) copy_w(b, woff[b]);
#pragma unroll
      for (int t = 0; t < COPIES; ++t) copy_x(t, xoff[t]);
    } else {   // a block past K repeats the last one (its scale is 0)
#pragma unroll
      for (int b = 0; b < RB; ++b) copy_w(b, woff[b] + 16 * (min(4 * c + wpiece, groups - 1) - wpiece));
#pragma unroll
      for (int t = 0; t < COPIES; ++t) copy_x(t, 128 * c + 8 * xpiece(t) < a.k ? xoff[t] + 256 * c : kPastEnd);
    }
  };
  constexpr int kEach = RB + COPIES;   // copies of a chunk
  static_assert((DEPTH - 1) * kEach < 64, "vmcnt counts them");
  // chunks past the wave's last are copied too (from the last one's lines): the waits below count on it
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) issue(std::false_type{}, d, first + d);   // (no branch: the scales' wait counts them)
#pragma unroll
  for (int j = 0; j < kTurns; ++j)
    if (kLine * j < chunks) {
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int at = scale_at(b, j), d = sd + kLine * j, live = groups - 4 * d;
        const uint32_t v = sv[b][j] >> (8 * (at - min(at, scales - 4)) & 31);
        if (d < chunks) scale[(16 * b + srow) * chunks + d] = live >= 4 ? v : v & ((1u << (8 * live)) - 1);
      }
    }
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));   // lgkmcnt 0: this wave's scales are in LDS
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

  f32x4_t acc[RB][MT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[b][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int xr = COPIES < 4 ? r & (4 * COPIES - 1) : r;   // rows that are not staged repeat others and are not stored
  int d = 0;   // place of chunk i
  for (int i = 0; i < mine; ++i) {
    MOE_WAIT_VM((DEPTH - 1) * kEach);   // the chunk has landed; those after it may be in flight
    asm volatile("" ::: "memory");
    const uint8_t* const at = ring + d * kPlace;
    u32x4_t w[RB];
    uint32_t sc[RB];
    bf16x8_t x[MT][4];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      w[b] = *reinterpret_cast<const u32x4_t*>(at + kXBytes + b * 1024 + r * 64 + (q ^ (2 * (r >> 3))) * 16);
      sc[b] = scale[(16 * b + r) * chunks + first + i];
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[t][j] = *reinterpret_cast<const bf16x8_t*>(at + t * 4096 + xr * 256 + ((4 * j + q) ^ (2 * (xr & 7))) * 16);
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));   // lgkmcnt 0: the place has been read
    asm volatile("" ::: "memory");
    const int c = first + i + DEPTH;
    if (4 * c + 4 <= groups) issue(std::true_type{}, d, c);
    else issue(std::false_type{}, d, c);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      transpose_quarters(w[b]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8_t v = dequant8(w[b][j], scale_byte(sc[b], j));
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, x[t][j], acc[b][t], 0, 0, 0);
      }
    }
    d = d + 1 == DEPTH ? 0 : d + 1;
  }
  MOE_WAIT_VM(0);    // the copies past the end still write LDS
  __syncthreads();   // every wave is done with its ring
  f32x4_t* const part = reinterpret_cast<f32x4_t*>(smem);
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < MT; ++i) part[((wave * RB + b) * MT + i) * kWave + lane] = acc[b][i];
  __syncthreads();
  auto sum = [&](int b, int i) {
    f32x4_t v = part[(b * MT + i) * kWave + lane];
#pragma unroll
    for (int w = 1; w < SPLIT; ++w) v += part[((w * RB + b) * MT + i) * kWave + lane];
    return v;
  };
  // a wave adds and stores a 16 x 16 block, with a gate a pair of them
  constexpr int kPairs = GATE && RB > 1 ? RB / 2 : RB;
  for (int task = wave; task < MT * kPairs; task += SPLIT) {
    const int i = task / kPairs, b = task % kPairs, m = 16 * i + r;
    f32x4_t v;
    if constexpr (GATE) {
      f32x4_t u;
      if constexpr (RB > 1) {
        v = sum(2 * b, i);
        u = sum(2 * b + 1, i);
      } else {
        v = sum(0, i);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = __shfl_xor(v[e], 32, kWave);
      }
      v = gated(v, u);
      if (RB == 1 && q >= 2) continue;   // the lanes of w3
    } else {
      v = sum(b, i);
    }
    const int c = c0 + 16 * b + 4 * q;
    if (m >= mrows || c >= cols) continue;
    const size_t at = (size_t)(m0 + m) * cols + c;
    if (cols % 4 == 0) {
      if (f32) *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + at) = v;
      else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
      continue;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (c + e >= cols) break;
      if (f32) static_cast<float*>(a.out)[at + e] = v[e];
      else static_cast<uint16_t*>(a.out)[at + e] = f32_to_bf16_rne(v[e]);
    }
  }
}

template <int MT, int RB, int SPLIT, int DEPTH, int COPIES, int GROUPS, bool GATE>
__global__ __launch_bounds__(SPLIT* kWave) void linear_rows(LinearArgs a, bool f32) {
  constexpr int kParts = SPLIT * RB * MT * 1024;   // the waves' sums, in the ring's memory after it
  constexpr int kRing = SPLIT * DEPTH * (COPIES + RB) * 1024;
  // One array: the compiler lets reads of a ring wait for every copy in flight
  // (vmcnt(0)) once there are two.
  constexpr int kMost = kRing > kParts ? kRing : kParts;
  __shared__ __align__(1024) uint8_t smem[kMost + RB * 16 * GROUPS];
  linear_rows_block<MT, RB, SPLIT, DEPTH, COPIES, GROUPS, GATE>(smem, reinterpret_cast<uint32_t*>(smem + kMost), a, f32);
}

template <int MT, int RB, int SPLIT, int DEPTH, int COPIES, int GROUPS>
hipError_t launch_rows(const LinearArgs& a, bool gate, bool f32, hipStream_t stream) {
  const int cols = gate ? a.n / 2 : a.n, wide = (gate ? 8 : 16) * RB;
  const dim3 grid((cols + wide - 1) / wide, (a.m + 16 * MT - 1) / (16 * MT)), block(SPLIT * kWave);
  if (gate) hipLaunchKernelGGL((linear_rows<MT, RB, SPLIT, DEPTH, COPIES, GROUPS, true>), grid, block, 0, stream, a, f32);
  else hipLaunchKernelGGL((linear_rows<MT, RB, SPLIT, DEPTH, COPIES, GROUPS, false>), grid, block, 0, stream, a, f32);
  return hipGetLastError();
}

// ---- many rows: BM x BN tiles, operands staged through LDS.
//
// A stage is 64 K. x comes as it lies, 128 bytes a row, into a ring of
// stages; W comes as packed codes, 128 K at a time (a unit, 64 bytes a row),
// into a ring of units: both by buffer_load ... lds copies of 1 KB a wave
// instruction, past an edge as zeros. A wave turns the codes of its columns
// into bf16 fragments in registers on the scaled converter, so a staged weight
// costs a quarter of a bf16 one's LDS traffic, and x, which every weight row
// shares, is what the tile shape saves.
//   In a stage lane quarter q has the 16 K values 16 q + [0, 16): 8 bytes of
// codes in one read, with one scale, that of block q / 2; MFMA step j takes
// 8 j + [0, 8) of them, of x alike.
//   x rows are 128 bytes, half the banks; their 16-byte chunks are permuted by
// chunk ^ f(row), f = (row >> 1 & 1) | (row >> 3 & 1) << 2. The sixteen lanes
// that ds_read_b128 serves at once are eight rows of one quarter's chunk and
// the other eight of its neighbour's (lanes 0-3, 12-15, 20-27), that is chunks
// 2 apart: f takes 0, 1, 4, 5 on either eight's even rows, so together they
// cover all eight places.
//   W rows are 64 bytes: chunk ^ (row >> 2 & 3) puts the rows four apart, which
// share banks, into different places.
//   Scales, a byte per row and block, go straight to registers, four a unit and row.
//   With a gate the tile's 16-row blocks of W alternate between w1 and w3, so
// that a lane holds both values of an output.
__device__ __forceinline__ int swz_x(int c, int r) { return c ^ (((r >> 1) & 1) | ((r >> 1) & 4)); }
__device__ __forceinline__ int swz_w(int c, int r) { return c ^ ((r >> 2) & 3); }

// NX stages in x's ring (odd), NW units in W's.
template <int BM_, int BN_, int WM_, int WN_, int PER_CU_, int NX_, int NW_>
struct LinearShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, kWaves = WM * WN, kPerCU = PER_CU_, NX = NX_, NW = NW_;
  static constexpr int MI = BM / WM / 16, NJ = BN / WN / 16;
  static constexpr int kXBytes = BM * 128, kWBytes = BN * 64;
  static constexpr int kX = BM / 8 / kWaves, kW = BN / 16 / kWaves;   // copies per wave: a stage's x, a unit's W
  static constexpr int kSmem = NX * kXBytes + NW * kWBytes;
  // copies and scale loads that a wave issues after a stage's x and before that stage starts
  static constexpr int kSc = (NJ + 3) / 4;   // loads of a unit's scales
  static constexpr int kAfter = (NX - 2) * kX + (kW + kSc) * (NX - 1) / 2;
  static_assert(kX * kWaves * 8 == BM && kW * kWaves * 16 == BN && kWaves % 2 == 0, "even split");
  static_assert(kPerCU * kSmem <= 160 * 1024 && MI % 2 == 0 && NJ % 2 == 0, "rings fit");
  static_assert(4 * (kX - 1) < 3 * (kX + kW), "a stage's x before its scales");
  static_assert(NX % 2 == 1 && 2 * NW > NX + 1 && kAfter < 64, "W lands before x of its stage; vmcnt counts them");
};

template <class C, bool GATE, bool F32>
__device__ __forceinline__ void linear_tile(uint8_t* smem, const LinearArgs& a, int tm, int tn) {
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  // workgroups go to the XCDs in turn: XCD x takes the x-th eighth of the
  // tiles, walked in bands of tile rows so that its concurrent tiles share
  // operand panels in its L2
  const int total = tm * tn, chunk = (total + kXcds - 1) / kXcds;
  const int id = (int)(blockIdx.x % kXcds) * chunk + (int)(blockIdx.x / kXcds);
  if ((int)(blockIdx.x / kXcds) >= chunk || id >= total) return;
  constexpr int kBand = 4;
  const int band = id / (kBand * tn), in = id - band * kBand * tn;
  const int high = min(kBand, tm - band * kBand);
  constexpr int kCols = GATE ? C::BN / 2 : C::BN;   // output columns of a tile
  const int cols = GATE ? a.n / 2 : a.n, groups = a.k / 32;
  const int m0 = (band * kBand + in % high) * C::BM, c0 = in / high * kCols;
  const int mrows = min(C::BM, a.m - m0), ncols = min(kCols, cols - c0);
  const uint32_t pitch = (uint32_t)groups * 16;   // bytes of a row's codes
  const int units = (groups + 3) / 4;

  uint8_t* const ring_w = smem + C::NX * C::kXBytes;
  // Copies: lane -> (row, place in the row); the permutation repeats every 16
  // rows, so a lane has one offset for all its copies, whose resources start
  // at their own rows (offsets of each copy's own would be spilled) and end
  // with the live ones.
  const int xrow = 8 * wave + (lane >> 3), xchunk = swz_x(lane & 7, xrow);
  const uint32_t xpitch = (uint32_t)a.ldx * 2, xoff = (lane >> 3) * xpitch + 16 * xchunk;
  // a W copy is one 16-row block; with a gate a wave's blocks are all w1's or all w3's
  const int wrow = lane >> 2, wchunk = swz_w(lane & 3, wrow);
  const uint32_t woff = wrow * pitch + 16 * wchunk;
  const uint8_t* const xbase = reinterpret_cast<const uint8_t*>(a.x + (size_t)m0 * a.ldx);
  const uint8_t* const wbase = a.codes + (size_t)(c0 + (GATE && (wave & 1) ? cols : 0)) * pitch;
  auto issue_x = [&](uint8_t* buf, int s, int j) {   // copy j of stage s
    const int row = 8 * (wave + C::kWaves * j);
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(xbase) + (size_t)row * xpitch + (size_t)s * 128, (short)0,
        max((mrows - row) * (int)xpitch - s * 128, 0), kRsrcWord3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(buf + (wave + C::kWaves * j) * 1024), 16,
                                             64 * s + 8 * xchunk < a.k ? xoff : kPastEnd, 0, 0, 0);
  };
  auto issue_w = [&](uint8_t* buf, int u, int j) {   // copy j of unit u
    const int b = wave + C::kWaves * j, row = 16 * (GATE ? b >> 1 : b);
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(wbase) + (size_t)row * pitch + (size_t)u * 64, (short)0,
        max((ncols - row) * (int)pitch - u * 64, 0), kRsrcWord3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(buf + b * 1024), 16,
                                             woff, 0, 0, 0);   // past K: whatever follows, times x's zeros
  };

  const int wm = wave / C::WN, wn = wave % C::WN, rl = lane & 15, q = lane >> 4;
  // Scales: a lane loads the four bytes of a unit's blocks of one row, of the
  // wave's 16-row block lane / 16 (and 4 more, ..), and the lanes that multiply
  // that row take them from it. (A lane that loads its own rows' makes every
  // load touch sixteen lines four times over, 64 clocks.) They are loaded two
  // units ahead (one: 1024 rows of 4096 x 7168 take 62.8 us for 59.9). The
  // matrix's last four bytes may start before the unit's and are moved down; past
  // K they are 0, so that codes there are finite whatever they are (x is 0).
  constexpr int kSc = C::kSc;
  const int scales = a.n * groups, last = max(scales - 4, 0);
  const __amdgpu_buffer_rsrc_t srsrc =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.scales), (short)0, scales, kRsrcWord3);
  int srow[kSc];   // offset of the lane's rows; rows past the matrix repeat its last
#pragma unroll
  for (int i = 0; i < kSc; ++i) {
    const int b = wn * C::NJ + min(4 * i + q, C::NJ - 1);
    srow[i] = (min(c0 + 16 * (GATE ? b >> 1 : b) + rl, cols - 1) + (GATE && (b & 1) ? cols : 0)) * groups;
  }
  uint32_t sc[C::NJ], next[kSc], far[kSc];   // in use, of the next unit, of the one after it
  auto load_scale = [&](int i, int u) {
    far[i] = __builtin_amdgcn_raw_buffer_load_b32(srsrc, min(srow[i] + 4 * u, last), 0, 0);
  };
  // the byte of lane quarter q's block of the unit's first stage in bits 7:0, of the second in 23:16
  auto take_scales = [&](int u) {
    const int live = groups - 4 * u;
    const uint32_t mask = live >= 4 ? ~0u : (1u << (8 * live)) - 1;
#pragma unroll
    for (int i = 0; i < kSc; ++i) next[i] = next[i] >> (8 * max(srow[i] + 4 * u - last, 0) & 31) & mask;
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
      sc[j] = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (16 * (j % 4) + rl), (int)next[j / 4]) >> (8 * (q >> 1));
  };

  f32x4_t acc[C::MI][C::NJ];
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // A unit's first stage issues its copies of W and its scales beside its x,
  // so what is issued between a stage's x and its start does not depend on
  // which of the two it is. The rings' fill keeps that order, as if stages
  // 1 - NX .. -1 had issued it.
  constexpr int kHalf = C::MI / 2, kM = kHalf * C::NJ;
  constexpr int kUnits = (C::NX - 1) / 2;   // those stages' units
  unrolled<C::NW - 1 - kUnits>([&](auto u) {
#pragma unroll
    for (int j = 0; j < C::kW; ++j) issue_w(ring_w + u * C::kWBytes, u, j);
  });
  if (scales >= 4) {
#pragma unroll
    for (int i = 0; i < kSc; ++i) load_scale(i, 0);
  } else {   // one unit, byte by byte
    uint32_t v = 0;
    for (int g = 0; g < scales; ++g) v |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(srsrc, g, 0, 0) << (8 * g);
#pragma unroll
    for (int i = 0; i < kSc; ++i) far[i] = v;
  }
#pragma unroll
  for (int i = 0; i < kSc; ++i) next[i] = far[i];
  unrolled<C::NX - 1>([&](auto vc) {
    constexpr int v = decltype(vc)::value, u = C::NW - 1 - kUnits + v / 2;
#pragma unroll
    for (int j = 0; j < C::kX; ++j) issue_x(smem + v * C::kXBytes, v, j);
    if constexpr (v % 2 == 0) {
#pragma unroll
      for (int j = 0; j < C::kW; ++j) issue_w(ring_w + u * C::kWBytes, u, j);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (v % 2 == 0) {
#pragma unroll
      for (int j = 0; j < kSc; ++j) load_scale(j, max(2 - kUnits + v / 2, 0));
    }
    __builtin_amdgcn_sched_barrier(0);
  });

  // A stage is four lists of MFMAs: steps 0 and 1, the wave's upper and lower
  // row blocks. Behind each MFMA stands a share of the LDS reads and
  // conversions for the lists after it and of the copies; the last list of a
  // stage runs after the next stage's barrier, over that stage's first reads.
  // Before the first stage its operands are zeros.
  bf16x8_t fx[C::MI], fw[2][C::NJ];
  u32x2_t raw[C::NJ];
#pragma unroll
  for (int i = 0; i < C::MI; ++i) fx[i] = bf16x8_t{};
#pragma unroll
  for (int j = 0; j < C::NJ; ++j) fw[1][j] = bf16x8_t{};
  // LDS offsets of the lane's operands; the others differ in one bit
  int xat = wm * C::MI * 2048 + rl * 128 + swz_x(2 * q, rl) * 16;
  int wat = wn * C::NJ * 1024 + rl * 64 + swz_w(q >> 1, rl) * 16 + (q & 1) * 8;
  auto keep = [&] {
    unrolled<C::MI * C::NJ>([&](auto mc) {
      f32x4_t& v = acc[decltype(mc)::value / C::NJ][decltype(mc)::value % C::NJ];
      pin(v[0]);
    });
  };
  int ix = 0, iw = 0;   // the ring places of stage s and unit u
  auto run_stage = [&](auto pc, int u) {   // stage p of unit u
    constexpr int p = decltype(pc)::value;
    const int s = 2 * u + p;
    // This wave's copies of the stage have landed and its LDS reads are done;
    // the barrier extends both to every wave.
    MOE_WAIT_VM(C::kAfter);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const uint8_t* const bx = smem + ix * C::kXBytes;
    const uint8_t* const bw = ring_w + iw * C::kWBytes;
    uint8_t* const to_x = smem + (ix ? ix - 1 : C::NX - 1) * C::kXBytes;
    uint8_t* const to_w = ring_w + (iw ? iw - 1 : C::NW - 1) * C::kWBytes;
    asm volatile("" : "+v"(xat), "+v"(wat));   // derived anew in each stage: held over the loop, they would be spilled
    auto read_x = [&](auto ic, auto jc) {
      constexpr int i = decltype(ic)::value, j = decltype(jc)::value;
      fx[i] = *reinterpret_cast<const bf16x8_t*>(bx + (xat ^ (16 * j)) + i * 2048);
    };
    auto read_w = [&](auto jc) {
      constexpr int j = decltype(jc)::value;
      raw[j] = *reinterpret_cast<const u32x2_t*>(bw + (wat ^ (32 * p)) + j * 1024);
    };
    auto convert = [&](auto jc, auto step) {
      constexpr int j = decltype(jc)::value, k = decltype(step)::value;
      fw[k][j] = dequant8(raw[j][k], scale_byte(sc[j], 2 * p));
    };
    unrolled<4>([&](auto hc) {
      constexpr int h = decltype(hc)::value;
      constexpr int step = h == 0 || h == 3 ? 1 : 0, lo = h % 2 == 0;   // the list that multiplies
      if constexpr (p == 0 && h == 0) take_scales(u);
      unrolled<kM>([&](auto mc) {
        constexpr int m = decltype(mc)::value, i = lo * kHalf + m / C::NJ, j = m % C::NJ;
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[step][j], fx[i], acc[i][j], 0, 0, 0);
        // reads of the next list's x blocks; W's at the stage's start
        if constexpr (h == 0) {
          unrolled<C::NJ>([&](auto b) { if constexpr (b * (kM / 4) / C::NJ == m) read_w(b); });
          unrolled<kHalf>([&](auto b) {
            if constexpr (kM / 4 + b * (kM / 4) / kHalf == m)
              read_x(std::integral_constant<int, decltype(b)::value>{}, std::integral_constant<int, 0>{});
          });
          unrolled<C::NJ>([&](auto b) {
            if constexpr (kM / 2 + b * (kM / 2) / C::NJ == m) convert(b, std::integral_constant<int, 0>{});
          });
        } else {
          constexpr int to = h == 2 ? 0 : kHalf;   // h 1: lower, step 0; 2: upper, step 1; 3: lower, step 1
          unrolled<kHalf>([&](auto b) {
            if constexpr (b * (kM / 2) / kHalf == m)
              read_x(std::integral_constant<int, to + decltype(b)::value>{}, std::integral_constant<int, (h > 1)>{});
          });
          if constexpr (h == 1)
            unrolled<C::NJ>([&](auto b) {
              if constexpr (b * kM / C::NJ == m) convert(b, std::integral_constant<int, 1>{});
            });
        }
        // copies over the whole stage, x's first, then W's, then the scales
        constexpr int kG = C::kX + (p ? 0 : C::kW);
        unrolled<kG>([&](auto cc) {
          constexpr int c = decltype(cc)::value;
          if constexpr (c * 4 * kM / kG == h * kM + m) {
            if constexpr (c < C::kX) issue_x(to_x, s + C::NX - 1, c);
            else issue_w(to_w, u + C::NW - 1, c - C::kX);
          }
        });
        if constexpr (p == 0 && h == 3) {
          unrolled<kSc>([&](auto b) {
            if constexpr (b * kM / kSc == m) {
              next[b] = far[b];
              asm volatile("" : "+v"(next[b]));   // here and not earlier, where it would wait for them
              load_scale(b, u + 2);
            }
          });
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    keep();
    ix = ix == C::NX - 1 ? 0 : ix + 1;
    if constexpr (p == 1) iw = iw == C::NW - 1 ? 0 : iw + 1;
  };
  for (int u = 0; u < units; ++u) {
    run_stage(std::integral_constant<int, 0>{}, u);
    run_stage(std::integral_constant<int, 1>{}, u);
  }
  unrolled<kM>([&](auto mc) {   // the last list of the last stage
    constexpr int m = decltype(mc)::value, i = kHalf + m / C::NJ, j = m % C::NJ;
    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[1][j], fx[i], acc[i][j], 0, 0, 0);
  });
  MOE_WAIT_VM(0);   // the copies past the end still write LDS
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();   // every wave is done reading the rings
  asm volatile("" ::: "memory");

  // Lane holds row rl, columns 4q .. 4q + 3 of each 16 x 16 block. The wave's
  // blocks pass through its part of LDS, 32 rows at a time, and leave as whole
  // rows of 16-byte chunks (permuted by chunk ^ row for the banks) or, where
  // the output's rows are not 16-byte aligned, of single values.
  // (The addresses below are made here: taken over the K loop in registers, they
  // would be spilled.)
  int lane_ = lane;
  asm volatile("" : "+v"(lane_));
  const int rl_ = lane_ & 15, q_ = lane_ >> 4;
  constexpr int kBlocks = GATE ? C::NJ / 2 : C::NJ;
  constexpr int kSize = F32 ? 4 : 2, kRowBytes = kBlocks * 16 * kSize, kChunks = kRowBytes / 16;
  constexpr int kMask = kChunks < 16 ? kChunks - 1 : 15;
  constexpr int kShift = kRowBytes >= 256 ? 0 : kRowBytes == 128 ? 1 : 2;   // rows side by side in the banks
  auto place = [](int r, int c) { return (c ^ ((r >> kShift) & kMask)) * 16; };   // chunk c of row r
  static_assert(C::kWaves * 32 * kRowBytes <= C::kSmem && 64 % kChunks == 0, "two blocks of every wave fit");
  const bool rows_aligned = cols % (16 / kSize) == 0;
  uint8_t* const stg = smem + wave * (32 * kRowBytes);
  const int mw = wm * (16 * C::MI), cw = wn * (16 * kBlocks);
#pragma unroll
  for (int i = 0; i < C::MI; i += 2) {
    if (mw + 16 * i >= mrows) break;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) {
        f32x4_t v = acc[i + h][GATE ? 2 * j : j];
        if constexpr (GATE) v = gated(v, acc[i + h][2 * j + 1]);
        uint8_t* const at = stg + (16 * h + rl_) * kRowBytes;
        if constexpr (F32)
          *reinterpret_cast<f32x4_t*>(at + place(16 * h + rl_, 4 * j + q_)) = v;
        else
          *reinterpret_cast<u32x2_t*>(at + place(16 * h + rl_, 2 * j + (q_ >> 1)) + 8 * (q_ & 1)) =
              u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
      }
    asm volatile("" ::: "memory");
    if (rows_aligned) {
#pragma unroll
      for (int k = 0; k < kChunks / 2; ++k) {   // 64 / kChunks rows at a time
        const int r = k * (64 / kChunks) + lane_ / kChunks, c = lane_ % kChunks;
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(stg + r * kRowBytes + place(r, c));
        const int m = mw + 16 * i + r, n = cw + c * (16 / kSize);
        if (m < mrows && n < ncols)
          *reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(a.out) + ((size_t)(m0 + m) * cols + c0 + n) * kSize) = v;
      }
    } else {
      using V = std::conditional_t<F32, float, uint16_t>;
      constexpr int kWide = kBlocks * 16;
#pragma unroll 8
      for (int k = 0; k < 32 * kWide / kWave; ++k) {
        const int r = (k * kWave + lane_) / kWide, n = (k * kWave + lane_) % kWide, m = mw + 16 * i + r;
        const V v = *reinterpret_cast<const V*>(stg + r * kRowBytes + place(r, n / (16 / kSize)) + n % (16 / kSize) * kSize);
        if (m < mrows && cw + n < ncols) static_cast<V*>(a.out)[(size_t)(m0 + m) * cols + c0 + cw + n] = v;
      }
    }
    asm volatile("" ::: "memory");
  }
}

template <class C, bool GATE, bool F32>
__global__ __launch_bounds__(C::kWaves* kWave, C::kPerCU* C::kWaves / 4) void linear_tiles(LinearArgs a, int tm, int tn) {
  __shared__ __align__(1024) uint8_t smem[C::kSmem];
  linear_tile<C, GATE, F32>(smem, a, tm, tn);
}

template <class C>
hipError_t launch_tiles(const LinearArgs& a, bool gate, bool f32, hipStream_t stream) {
  const int cols = gate ? a.n / 2 : a.n, wide = gate ? C::BN / 2 : C::BN;
  const int tm = (a.m + C::BM - 1) / C::BM, tn = (cols + wide - 1) / wide;
  const dim3 grid((unsigned)(((long long)tm * tn + kXcds - 1) / kXcds * kXcds)), block(C::kWaves * kWave);
  if (gate && f32) hipLaunchKernelGGL((linear_tiles<C, true, true>), grid, block, 0, stream, a, tm, tn);
  else if (gate) hipLaunchKernelGGL((linear_tiles<C, true, false>), grid, block, 0, stream, a, tm, tn);
  else if (f32) hipLaunchKernelGGL((linear_tiles<C, false, true>), grid, block, 0, stream, a, tm, tn);
  else hipLaunchKernelGGL((linear_tiles<C, false, false>), grid, block, 0, stream, a, tm, tn);
  return hipGetLastError();
}

// Four waves of 64 x 64 for the smaller tile: in eight of 64 x 32, which read x from
// LDS twice as often, 1900 rows of 4096 x 7168 take 109 us for 102, up to 300 rows the
// same. (Eight of 128 x 64 for the larger one: four of 128 x 128 take 227 for 168.)
using Linear256 = LinearShape<256, 256, 2, 4, 1, 3, 3>;
using Linear128 = LinearShape<128, 128, 2, 2, 2, 3, 3>;

}  // namespace

hipError_t launch_mxfp4_linear(const LinearArgs& a, bool gate, bool f32, hipStream_t stream) {
  const int groups = a.k / 32;
  const long long mb = (a.m + 15) / 16, blocks = mb * ((a.n + 15) / 16);   // 16 x 16 outputs, gated ones counted twice
  // The streaming kernel reads scales four at a time and reaches both halves
  // of a gated matrix from one address: the eight rows of w3 end (n / 2 + 8)
  // rows behind w1's first, within a resource of 2^31 - 1 bytes. Its rows of W hold
  // up to 512 scales (2048 in the form for up to 16 rows).
  const bool streams = (long long)a.n * groups >= 4 && (!gate || (a.n / 2 + 8ll) * groups * 16 < (1ll << 31));
  // Up to 4096 blocks it beats the 128 x 128 tiles, over a long K up to 8192 (K 7168
  // to 4096 columns: 512 rows, 8192 blocks, 43 against 58 us, 1024 rows 81 against
  // 59; K 2048 to 7168: 128 rows, 3584 blocks, 11.8 against 19.7, 256 rows 20.3
  // against 19.7; K 512 to 1024: 2048 rows, 8192 blocks, 11.0 against 7.8).
  if (streams && blocks <= (a.k > 4096 ? 8192 : 4096) && (groups <= 512 || a.m <= 16)) {
    if (groups > 512) return launch_rows<1, 1, 8, 3, 4, 2048>(a, gate, f32, stream);
    // up to four rows one copy of x a chunk, and room for a second chunk (one row, K 7168
    // to 4096 columns: 6.3 us, with four copies and one chunk 7.4)
    if (a.m <= 4) return launch_rows<1, 1, 8, 2, 1, 512>(a, gate, f32, stream);
    // The smallest share of a workgroup that keeps the workgroups to one a CU or
    // two: less of W or x is loaded twice with a larger one, and more CUs work with
    // a smaller. us for shares of 1 x 1, 1 x 2, 2 x 2, 2 x 4, 4 x 4 blocks of x and W
    // (in each row the one taken is the fastest measured):
    //   K 7168 to 4096   16 rows (256 blocks)    8.8 10.4 12.5 17.7 21.6
    //                    32 rows (512)          12.7 10.2 13.9 18.7 22.9
    //                    37 rows (768)          15.3 13.3 11.0 16.1 23.6
    //                    128 rows (2048)        32.1 23.7 21.9 17.0 23.7
    //                    256 rows (4096)        58.8 41.6 39.4 29.0 23.5
    //   K 2048 to 7168   16 rows (448)           5.9  4.9  5.6  7.4 10.8
    //                    32 rows (896)           8.2  6.8  6.2  7.7 11.2
    //                    37 rows (1344)         10.0  8.7  9.3  7.7 11.4
    //                    128 rows (3584)        20.5 16.3 17.0 13.0 11.8
    // One block of rows is not spread over two: 1 x 4 from 513 blocks.
    if (blocks <= 256) return launch_rows<1, 1, 8, 1, 4, 512>(a, gate, f32, stream);
    if (blocks <= 512) return launch_rows<1, 2, 8, 1, 4, 512>(a, gate, f32, stream);
    if (mb == 1) return launch_rows<1, 4, 8, 1, 4, 512>(a, gate, f32, stream);
    if (blocks <= 1024) return launch_rows<2, 2, 8, 1, 8, 512>(a, gate, f32, stream);
    if (blocks <= 2048 || mb == 2) return launch_rows<2, 4, 8, 1, 8, 512>(a, gate, f32, stream);
    return launch_rows<4, 4, 4, 1, 16, 512>(a, gate, f32, stream);
  }
  // 256 x 256 tiles once they fill most of the CUs (K 7168 to 4096 columns: 2048
  // rows, 128 of them, 140 against 99 us, 2560 rows, 160, 141 against 143; K 2048 to 7168:
  // 1500 rows, 168 of them, 44.4 against 44.7, 1792 rows, 196, 44 against 55), but not where
  // a second round of them would run on few CUs (K 7168 to 4096: 4352 rows, 272 tiles, 278
  // against 230, 5632 rows, 352, 282 against 275, 6000 rows, 384, 284 against 285; K 2048 to
  // 7168: 2560 rows, 280 tiles, 86 against 69, 3000 rows, 336, 87 against 82, 3584 rows, 392,
  // 88 against 96). With more rounds the last weighs less.
  const long long large = (long long)((a.m + 255) / 256) * ((a.n + 255) / 256);
  if (large >= 160 && !(large > 256 && large <= 352)) return launch_tiles<Linear256>(a, gate, f32, stream);
  return launch_tiles<Linear128>(a, gate, f32, stream);
}

}  // namespace moe
