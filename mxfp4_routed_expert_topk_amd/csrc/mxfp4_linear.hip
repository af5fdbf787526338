// Product of bf16 rows with an MXFP4 matrix in checkpoint layout,
//   y [M, N] = x [M, K] W [N, K]^T,   W = code 2^(byte - 127)
// and, gated, silu(y[:, c]) y[:, c + N/2] for the fused w1||w3 of a shared
// expert.  A weight has at most two significant bits, so W is exact in bf16
// for every scale byte (0 is 2^-127, 255 NaN; 4 and 6 times 2^127 are infinite
// there as in fp32); products are summed in fp32 on v_mfma_f32_16x16x32_bf16,
// which keeps subnormal operands, and the sum is rounded once.
#include <type_traits>

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

// ---- many rows: BM x BN tiles, operands staged through LDS.
//
// A stage is 64 K. x comes as it lies, 128 bytes a row, into a ring of three
// stages; W comes as packed codes, 128 K at a time (a unit, 64 bytes a row),
// into a ring of three units: both by buffer_load ... lds copies of 1 KB a wave
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
//   Scales, a byte per row and block, go straight to registers, four a unit.
//   With a gate the tile's 16-row blocks of W alternate between w1 and w3, so
// that a lane holds both values of an output.
typedef __attribute__((address_space(3))) void lds_void_t;
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

constexpr uint32_t kPastEnd = 0x80000000u;   // beyond every buffer resource below
constexpr int kMaxRange = 0x7FFFFFFF;

// vmcnt <= n and lgkmcnt 0
#define MOE_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | ((((n) >> 4) & 3) << 14))

__device__ __forceinline__ int swz_x(int c, int r) { return c ^ (((r >> 1) & 1) | ((r >> 1) & 4)); }
__device__ __forceinline__ int swz_w(int c, int r) { return c ^ ((r >> 2) & 3); }

template <int BM_, int BN_, int WM_, int WN_, int PER_CU_>
struct LinearShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, kWaves = WM * WN, kPerCU = PER_CU_;
  static constexpr bool kAlone = kWaves * kPerCU == 4;    // a wave has its SIMD, and 512 registers, to itself
  static constexpr int MI = BM / WM / 16, NJ = BN / WN / 16;
  static constexpr int kXBytes = BM * 128, kWBytes = BN * 64;
  static constexpr int kX = BM / 8 / kWaves, kW = BN / 16 / kWaves;   // copies per wave: a stage's x, a unit's W
  static constexpr int kSmem = 3 * (kXBytes + kWBytes);
  static_assert(kX * kWaves * 8 == BM && kW * kWaves * 16 == BN && kW % 2 == 0 && kWaves % 2 == 0, "even split");
  static_assert(kPerCU * kSmem <= 160 * 1024 && MI % 2 == 0 && NJ % 2 == 0, "rings fit");
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

  uint8_t* const ring_w = smem + 3 * C::kXBytes;
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
  // Scales: the four bytes of a unit's blocks of each of the wave's 16-row
  // blocks. A last unit that is not whole takes the row's last four bytes,
  // moved down; what follows is 0, so that codes past K are finite whatever they
  // are (x is zero there).
  uint32_t sc[C::NJ], next[C::NJ];
  __amdgpu_buffer_rsrc_t srsrc[GATE ? 2 : 1];   // rows past the matrix read as 0
#pragma unroll
  for (int h = 0; h < (GATE ? 2 : 1); ++h)
    srsrc[h] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.scales) + (size_t)(c0 + h * cols) * groups, (short)0,
                                                 ncols * groups, kRsrcWord3);
  const uint32_t srow = rl * groups;
  auto scale_at = [&](int j, int g) {   // byte g of block j's rows
    const int b = wn * C::NJ + j;
    return srow + (uint32_t)(16 * (GATE ? b >> 1 : b) * groups + g);
  };
  auto load_scale = [&](int j, int u) {
    next[j] = __builtin_amdgcn_raw_buffer_load_b32(srsrc[GATE ? j & 1 : 0], scale_at(j, max(min(4 * u, groups - 4), 0)), 0, 0);
  };
  // the byte of lane quarter q's block of the unit's first stage in bits 7:0, of the second in 23:16
  auto take_scales = [&](int u) {
    const int past = groups >= 4 ? 8 * max(4 * u + 4 - groups, 0) : 0;
    const uint32_t by = (uint32_t)min(past, 31) + 8 * (q >> 1);
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) sc[j] = (uint32_t)((unsigned long long)next[j] >> by);
  };

  f32x4_t acc[C::MI][C::NJ];
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // The rings' fill, in the order that a stage's wait counts on: unit 1's W and
  // the scales as if stages before the first had issued them.
  constexpr int kHalf = C::MI / 2, kM = kHalf * C::NJ, kWh = C::kW / 2, kG = C::kX + kWh;
#pragma unroll
  for (int j = 0; j < C::kW; ++j) issue_w(ring_w, 0, j);
#pragma unroll
  for (int j = 0; j < C::kX; ++j) issue_x(smem, 0, j);
#pragma unroll
  for (int j = 0; j < kWh; ++j) issue_w(ring_w + C::kWBytes, 1, j);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < C::NJ; ++j) {
    if (groups >= 4) {
      load_scale(j, 0);
    } else {   // K below 128: one unit, byte by byte
      next[j] = 0;
      for (int g = 0; g < groups; ++g)
        next[j] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(srsrc[GATE ? j & 1 : 0], scale_at(j, g), 0, 0) << (8 * g);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < C::kX; ++j) issue_x(smem + C::kXBytes, 1, j);
#pragma unroll
  for (int j = kWh; j < C::kW; ++j) issue_w(ring_w + C::kWBytes, 1, j);

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
      if constexpr (C::kAlone) pin_agpr(v);
      else pin(v[0]);
    });
  };
  if constexpr (C::kAlone) keep();
  int ix = 0, iw = 0;   // the ring places of stage s and unit u
  auto run_stage = [&](auto pc, int u) {   // stage p of unit u
    constexpr int p = decltype(pc)::value;
    const int s = 2 * u + p;
    // This wave's copies of the stage have landed and its LDS reads are done;
    // the barrier extends both to every wave. After the stage's x copies it has
    // issued the W copies beside them, a stage's copies and a unit's scales.
    MOE_WAIT_VM(2 * kWh + C::kX + C::NJ);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const uint8_t* const bx = smem + ix * C::kXBytes;
    const uint8_t* const bw = ring_w + iw * C::kWBytes;
    uint8_t* const to_x = smem + (ix ? ix - 1 : 2) * C::kXBytes;
    uint8_t* const to_w = ring_w + (iw ? iw - 1 : 2) * C::kWBytes;
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
      fw[k][j] = dequant8(raw[j][k], e8m0_to_f32((p ? sc[j] >> 16 : sc[j]) & 0xFFu));
    };
    unrolled<4>([&](auto hc) {
      constexpr int h = decltype(hc)::value;
      constexpr int step = h == 0 || h == 3 ? 1 : 0, lo = h % 2 == 0;   // the list that multiplies
      if constexpr (p == 0 && h == 0) take_scales(u);
      unrolled<kM>([&](auto mc) {
        constexpr int m = decltype(mc)::value, i = lo * kHalf + m / C::NJ, j = m % C::NJ;
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[step][j], fx[i], acc[i][j], 0, 0, 0);
        if constexpr (C::kAlone) pin_agpr(acc[i][j]);
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
        unrolled<kG>([&](auto cc) {
          constexpr int c = decltype(cc)::value;
          if constexpr (c * 4 * kM / kG == h * kM + m) {
            if constexpr (c < C::kX) issue_x(to_x, s + 2, c);
            else issue_w(to_w, u + 2, p * kWh + c - C::kX);
          }
        });
        if constexpr (p == 0 && h == 3) {
          unrolled<C::NJ>([&](auto b) { if constexpr (b * kM / C::NJ == m) load_scale(b, u + 1); });
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    keep();
    ix = ix == 2 ? 0 : ix + 1;
    if constexpr (p == 1) iw = iw == 2 ? 0 : iw + 1;
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
        if constexpr (GATE)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = gated(v[e], acc[i + h][2 * j + 1][e]);
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
      for (int r = 0; r < 32 && mw + 16 * i + r < mrows; ++r)
        for (int n = lane_; n < kBlocks * 16; n += kWave) {
          const V v = *reinterpret_cast<const V*>(stg + r * kRowBytes + place(r, n / (16 / kSize)) + n % (16 / kSize) * kSize);
          if (cw + n < ncols) static_cast<V*>(a.out)[(size_t)(m0 + mw + 16 * i + r) * cols + c0 + cw + n] = v;
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

using Linear256 = LinearShape<256, 256, 2, 4, 1>;
using Linear128 = LinearShape<128, 128, 2, 2, 2>;

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
  if (a.m > 64) {
    if ((long long)((a.m + 255) / 256) * ((a.n + 255) / 256) >= 192) return launch_tiles<Linear256>(a, gate, f32, stream);
    return launch_tiles<Linear128>(a, gate, f32, stream);
  }
  if (a.m <= 16) return launch_rows<1>(a, gate, f32, stream);
  if (a.m <= 32) return launch_rows<2>(a, gate, f32, stream);
  return launch_rows<4>(a, gate, f32, stream);
}

}  // namespace moe
