// Products of ragged groups of rows with one bf16 matrix per group (a routed
// layer's unquantised experts), and their gradients.  Rows offsets[e] ..
// offsets[e+1]-1 of x [R, K] belong to group e with w_e [N, K]:
//   forward    y_r  = w_e x_r                       reduction over K
//   dx         dx_r = dy_r w_e                      reduction over N
//   dw         dw_e = sum over e's rows dy_r x_r^T  reduction over the rows
// One tile kernel on v_mfma_f32_16x16x32_bf16 serves the three: an output tile
// of BM x BN is the product of a row operand P (output rows) and a column
// operand Q (output columns).  An operand
// lies in memory either along its reduction ("plain": x and w forward, dy for
// dx) or across it ("crossed": w for dx; dy and x for dw); a crossed operand
// is staged as it lies and read through ds_read_b64_tr_b16, which hands each
// lane one column's four consecutive reduction values, so nothing is
// transposed in memory.
//
// Staging: buffer_load ... lds copies of 1 KB per wave instruction, STEP of the
// reduction at a time, into one ring of tiles for Q and one for P.  Q is the
// operand that comes from HBM (the weights) and has the longer ring, P the rows
// that a tile's column slices share in L2.  Addresses past an edge (rows past
// the group, reduction past its length, columns past the matrix) get an
// out-of-range offset, for which the copy writes zeros: no other group's row,
// NaN or not, enters a sum.
//   plain tile: rows of STEP reduction values (128 bytes, half the banks) whose
//     16-byte chunks are permuted by chunk ^ (row >> 1).  The sixteen lanes that
//     ds_read_b128 serves at once are eight rows of one chunk and the other
//     eight of its neighbour (lanes 0-3, 12-15, 20-27): the eight even rows
//     then take all eight places, and the odd ones.  (chunk ^ row ^ (row >> 3)
//     is right for lanes in order only: every read took twice the cycles.)
//   crossed tile: STEP rows (the reduction) of BM or BN columns whose 64-byte
//     units are permuted by unit ^ (row & 3) and whose halves of a unit by
//     (row >> 3) & 1: the eight rows that half a wave's transposed read takes
//     lie in eight different halves, again all 64 banks.
// Both operands number the reduction alike, so every output is one fp32 sum
// in ascending order of 32 values an MFMA, whatever the tile; in a split
// reduction each part is such a sum and the parts are added in their order.
//
// Q is the instruction's first operand: a lane then ends with four
// consecutive columns of one output row, stored together.
#include <algorithm>
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr int kCusPerXcd = 32;
constexpr uint32_t kPastEnd = 0x80000000u;     // beyond every buffer resource below
constexpr int kMaxRange = 0x7FFFFFFF;          // bytes a resource covers

// vmcnt <= n and lgkmcnt 0
#define MOE_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | ((((n) >> 4) & 3) << 14))

// LDS place of 16-byte chunk c in a plain tile's row r.
__device__ __forceinline__ int swz(int c, int r) { return c ^ ((r >> 1) & 7); }

// Four reduction values of one column (see Operand::read).  The __restrict__
// matters: without alias information on the read the compiler takes it to
// depend on every LDS copy in flight and waits for all of them (vmcnt(0)).
__device__ __forceinline__ s16x4_t read_crossed(const uint8_t* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p));
}

// One operand's tile of B rows (plain) or columns (crossed), `count` of them
// live, over `length` of the reduction; `base` is its first element and `ld`
// the elements from one memory row to the next.
// NT: read past the caches.
template <bool CROSSED, int B, int WAVES, int STEP, bool NT>
struct Operand {
  static constexpr int kBytes = B * STEP * 2;
  static constexpr int kCopies = kBytes / 1024 / WAVES;   // copies per wave and stage
  static constexpr int kChunks = B / 8;                   // crossed: 16-byte chunks per staged row
  static_assert(!CROSSED || B >= 128, "four 64-byte units to permute");
  static_assert(kCopies * WAVES * 1024 == kBytes, "copies split evenly");

  const uint16_t* base;
  long long ld;
  int length;
  int wave;
  // Copies of a wave lie 8 kRows or more staged rows apart, so a lane's chunk is
  // the same in all of them.  Plain: each copy has its own memory row; crossed:
  // the same columns of rows that lie kApart apart.
  static constexpr int kPerRow = CROSSED ? kChunks : STEP / 8;   // chunks per staged row
  static constexpr int kRows = 64 / kPerRow;                     // staged rows per copy
  static constexpr int kApart = kRows * WAVES;
  static_assert(kApart % 16 == 0 || kCopies == 1, "the permutation repeats");
  static constexpr int kOffs = CROSSED ? 1 : kCopies;
  uint32_t off[kOffs];     // byte offset of this lane's chunk at stage 0 (kPastEnd: not live)
  int red;                 // reduction index of its first value at stage 0 (of copy 0)

  __device__ __forceinline__ Operand(const uint16_t* b, long long l, int count, int len, int w, int lane)
      : base(b), ld(l), length(len), wave(w) {
    const int r = kRows * wave + lane / kPerRow;
    if constexpr (CROSSED) {
      const int c = (lane % kPerRow) ^ ((r & 3) << 2) ^ (((r >> 3) & 1) << 1);
      red = r;
      off[0] = 8 * c < count ? (uint32_t)((long long)r * ld * 2) + 16 * c : kPastEnd;
    } else {
      const int c = swz(lane % kPerRow, r);
      red = 8 * c;
#pragma unroll
      for (int j = 0; j < kCopies; ++j)
        off[j] = r + kApart * j < count ? (uint32_t)((long long)(r + kApart * j) * ld * 2) + 16 * c : kPastEnd;
    }
  }

  // copy j of stage s into `buf`
  __device__ __forceinline__ void issue(uint8_t* buf, int s, int j) const {
    const long long skip = CROSSED ? ((long long)s * STEP + kApart * j) * ld : (long long)s * STEP;
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base + skip), (short)0, kMaxRange, kRsrcWord3);
    const int at = red + s * STEP + (CROSSED ? kApart * j : 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(buf + (wave + WAVES * j) * 1024), 16,
                                             at < length ? off[CROSSED ? 0 : j] : kPastEnd, 0, 0, NT ? 2 : 0);
  }

  // MFMA operand of 16-row block b, 32-deep step k, from a staged tile
  static __device__ __forceinline__ bf16x8_t read(const uint8_t* buf, int b, int k, int lane) {
    const int i = lane & 15, q = lane >> 4;   // row and the step's q-th eight values
    if constexpr (!CROSSED) {
      return *reinterpret_cast<const bf16x8_t*>(buf + (b * 16 + i) * (2 * STEP) + swz(4 * k + q, i) * 16);
    } else {
      // lane i of 16 points at row i/4 and columns 4 (i%4).. of a 4 x 16 block
      const uint8_t* p = buf + (32 * k + 8 * q + (i >> 2)) * (B * 2) +
                         (((b >> 1) ^ (i >> 2)) * 4 + 2 * ((b ^ q) & 1) + ((i >> 1) & 1)) * 16 + (i & 1) * 8;
      const s16x4_t lo = read_crossed(p), hi = read_crossed(p + 4 * (B * 2));
      const s16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      return __builtin_bit_cast(bf16x8_t, v);
    }
  }
};

// Row tiles (of bm rows, groups in order) and the place of one of them.
// Offsets are clamped to [0, rows] and count at least as much as every one
// before them: none leads outside the tensors, no two groups share a row, so
// that no two workgroups write one (nor one row's parts of a split sum), and
// there are never more tiles than the grid was made for.  Every wave counts by
// itself: a lane takes ceil(groups / 64) groups, a wave scan gives each lane
// its first tile.
struct Tile { int e, row0, rows; };
struct RowTiles {
  const int32_t* offsets;
  int rows, bm, e0, e1, from, first, mine, total;   // from: group e0's rows start there or later

  __device__ __forceinline__ int clamped(int e) const { return min(max(offsets[e], 0), rows); }
  // Counts the lane's tiles; last: where the last one ends.  True if an offset
  // is below the one before it.
  __device__ __forceinline__ bool count(int& last) {
    bool falls = false;
    mine = 0;
    last = from;
    for (int e = e0; e < e1; ++e) {
      const int lo = max(clamped(e), last), to = clamped(e + 1);
      falls |= to < lo;
      last = max(to, lo);
      mine += (last - lo + bm - 1) / bm;
    }
    return falls;
  }
  __device__ __forceinline__ RowTiles(const int32_t* o, int groups, int r, int b, int lane)
      : offsets(o), rows(r), bm(b), from(0) {
    const int per = (groups + kWave - 1) / kWave;
    e0 = min(lane * per, groups);
    e1 = min(e0 + per, groups);
    int last;
    if (__any(count(last))) {   // each lane starts from the largest offset of the lanes before it
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const int v = __shfl_up(last, d, kWave);
        if (lane >= d) last = max(last, v);
      }
      const int before = __shfl_up(last, 1, kWave);
      if (lane > 0) from = before;
      count(last);
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int v = __shfl_up(upto, d, kWave);
      if (lane >= d) upto += v;
    }
    first = upto - mine;
    total = __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  // tile in [0, total)
  __device__ __forceinline__ Tile place(int tile) const {
    Tile t = {0, 0, 0};
    const bool here = tile >= first && tile < first + mine;
    if (here) {
      int at = first, hi = from;
      for (int e = e0; e < e1; ++e) {
        const int lo = max(clamped(e), hi);
        hi = max(clamped(e + 1), lo);
        const int n = (hi - lo + bm - 1) / bm;
        if (tile < at + n) {
          t.e = e;
          t.row0 = lo + (tile - at) * bm;
          t.rows = min(bm, hi - t.row0);
          break;
        }
        at += n;
      }
    }
    const int src = __ffsll((unsigned long long)__ballot(here)) - 1;
    t.e = __builtin_amdgcn_readlane(t.e, src);
    t.row0 = __builtin_amdgcn_readlane(t.row0, src);
    t.rows = __builtin_amdgcn_readlane(t.rows, src);
    return t;
  }
};

// W waves as WM x WN.  A wave's 32-row blocks are every WM-th one, so that the
// blocks past a tile's last row, which are skipped, are spread over the waves;
// its 32-column blocks lie side by side.
// NP and NQ tiles of the rings; PER_CU workgroups fit a CU.  NT: Q is read by
// one workgroup only and passes the caches by.
template <int BM_, int BN_, int WM_, int WN_, int STEP_, int NP_, int NQ_, int PER_CU_, bool NT_ = false>
struct Shape {
  static constexpr bool NT = NT_;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STEP = STEP_, NP = NP_, NQ = NQ_;
  static constexpr int kWaves = WM * WN, kPerCU = PER_CU_;
  static constexpr bool kAlone = kWaves * kPerCU == 4;   // a wave has its SIMD, and 512 registers, to itself
  static constexpr int MI = BM / WM / 32, NJ = BN / WN / 32;
  static constexpr int kSmem = 2 * STEP * (BM * NP + BN * NQ);
  static_assert(NQ >= NP && NP >= 2 && kPerCU * kSmem <= 160 * 1024, "rings fit");
};

// The operands of a tile in shape C.
template <class C, bool PX, bool QX>
struct Operands {
  using P = Operand<PX, C::BM, C::kWaves, C::STEP, false>;
  using Q = Operand<QX, C::BN, C::kWaves, C::STEP, C::NT>;
  P p;
  Q q;
  // Stage s issues P of stage s + NP - 1 and Q of stage s + NQ - 1 into the
  // tiles that stage s - 1 has read; the stages before 0 fill the rings.
  __device__ __forceinline__ void fill(uint8_t* smem) const {
    uint8_t* const ring_p = smem + C::NQ * Q::kBytes;
    unrolled<C::NQ - 1>([&](auto d) {
      constexpr int v = decltype(d)::value, sp = v - (C::NQ - C::NP);
      if constexpr (sp >= 0) unrolled<P::kCopies>([&](auto c) { p.issue(ring_p + sp * P::kBytes, sp, c); });
      unrolled<Q::kCopies>([&](auto c) { q.issue(smem + v * Q::kBytes, v, c); });
    });
  }
};

// Stores of a full tile's epilogue that a K loop's first wait may leave in
// flight (they follow the fill it waits for).
constexpr int kLater = 32;

// The K loop over a wave's first LIVE row blocks, the rings filled.  later: the
// wave has issued kLater stores or more since the fill.
template <class C, bool PX, bool QX, int LIVE>
struct Reduce {
  static __device__ __forceinline__ void run(uint8_t* smem, const Operands<C, PX, QX>& o, int stages, int wm, int wn,
                                             int lane, bool later, f32x4_t (&acc)[2 * C::MI][2 * C::NJ]) {
    using P = typename Operands<C, PX, QX>::P;
    using Q = typename Operands<C, PX, QX>::Q;
    constexpr int kG = P::kCopies + Q::kCopies;
    uint8_t* const ring_q = smem;
    uint8_t* const ring_p = smem + C::NQ * Q::kBytes;

    // A stage has STEP / 32 steps, each two lists of MFMAs: the upper and the
    // lower half of the wave's live 16-row blocks.  Behind each MFMA stands a
    // share of the LDS reads of the list after it and of the global copies: a
    // run of reads would fill the LDS queue from eight waves at once and hold
    // up the MFMAs behind it.  A stage's last list therefore runs after the
    // next stage's barrier, over that stage's first reads.  Before the first
    // stage its operands are zeros (0 * 0 leaves the accumulators at +0).
    constexpr int kSteps = C::STEP / 32;
    static_assert(kSteps % 2 == 0, "two sets of Q operands in turn");
    constexpr int kH = LIVE, kB = 2 * C::NJ, kM = kH * kB;   // P and Q blocks and MFMAs of a list
    // With two waves a SIMD the copies stand in a stage's first quarter (P,
    // needed one stage on) and third quarter (Q): 1431 us for eight groups of
    // 4096 x 4096 x 7168, 1445 with all of them in the first half, 1471 over the
    // whole stage; a wave alone takes that (1412 against 1422).  P's come first,
    // as the wait below counts.
    constexpr int kQuarter = 2 * kSteps * kM / 4;
    constexpr int kRows = LIVE ? 2 * LIVE : 1;
    bf16x8_t fp[kRows], fq[2][kB];
#pragma unroll
    for (int i = 0; i < kRows; ++i) fp[i] = bf16x8_t{};
#pragma unroll
    for (int j = 0; j < kB; ++j) fq[1][j] = bf16x8_t{};
    // the accumulators stay where they are: those of a wave alone are 256, all
    // of the AGPRs (unasked, the compiler moved them about: 2170 us for 1412)
    auto keep = [&] {
      unrolled<2 * kM>([&](auto mc) {
        f32x4_t& a = acc[decltype(mc)::value / kB][decltype(mc)::value % kB];
        if constexpr (C::kAlone) pin_agpr(a);
        else pin(a[0]);
      });
    };
    if constexpr (C::kAlone) keep();
    int iq = 0, ip = 0;   // stage s's tiles
    for (int s = 0; s < stages; ++s) {
      // this wave's copies of stage s have landed (what was issued after them
      // may be in flight) and its reads of stage s - 1 are done; the barrier
      // extends both to every wave
      constexpr int kAfter = (C::NP - 2) * kG + (C::NQ > C::NP ? Q::kCopies : 0);
      if (s == 0 && later) MOE_WAIT_VM(kAfter + kLater);
      else MOE_WAIT_VM(kAfter);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const uint8_t* bq = ring_q + iq * Q::kBytes;
      const uint8_t* bp = ring_p + ip * P::kBytes;
      uint8_t* const to_q = ring_q + (iq ? iq - 1 : C::NQ - 1) * Q::kBytes;
      uint8_t* const to_p = ring_p + (ip ? ip - 1 : C::NP - 1) * P::kBytes;
      auto row_block = [&](int i) { return 2 * ((i >> 1) * C::WM + wm) + (i & 1); };   // of the tile
      auto copy = [&](auto c) {
        constexpr int i = decltype(c)::value;
        if constexpr (i < P::kCopies) o.p.issue(to_p, s + C::NP - 1, i);
        else o.q.issue(to_q, s + C::NQ - 1, i - P::kCopies);
      };
      unrolled<2 * kSteps>([&](auto hc) {
        // the MFMAs of the list before (the last one of stage s - 1 first) over the reads of list h
        constexpr int h = decltype(hc)::value, k = h / 2, half = h % 2;
        constexpr int before = half ? k : (k + kSteps - 1) % kSteps;   // its step
        constexpr int kR = half ? kH : kH + kB;                        // reads, over 3/4 of the MFMAs
        unrolled<kM>([&](auto mc) {
          constexpr int m = decltype(mc)::value, i = (1 - half) * kH + m / kB, j = m % kB;
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[before % 2][j], fp[i], acc[i][j], 0, 0, 0);
          unrolled<kR>([&](auto rc) {   // q0, p0, the other q's, the other p's
            constexpr int r = decltype(rc)::value;
            if constexpr (r * 3 * kM / (4 * kR) == m) {
              constexpr int p = half ? r : r == 1 ? 0 : r - kB, q = r ? r - 1 : 0;
              if constexpr (half || r == 1 || r > kB)
                fp[half * kH + p] = P::read(bp, row_block(half * kH + p), k, lane);
              else
                fq[k % 2][q] = Q::read(bq, wn * kB + q, k, lane);
            }
          });
          unrolled<kG>([&](auto cc) {
            constexpr int c = decltype(cc)::value, q = c - P::kCopies;
            constexpr int at = C::kAlone ? c * 4 * kQuarter / kG
                               : q < 0   ? c * kQuarter / P::kCopies
                                         : 2 * kQuarter + q * kQuarter / Q::kCopies;
            if constexpr (at == h * kM + m) copy(cc);
          });
          __builtin_amdgcn_sched_barrier(0);
        });
      });
      if constexpr (LIVE == 0) unrolled<kG>([&](auto c) { copy(c); });
      keep();
      iq = iq + 1 == C::NQ ? 0 : iq + 1;
      ip = ip + 1 == C::NP ? 0 : ip + 1;
    }
    unrolled<kM>([&](auto mc) {
      constexpr int m = decltype(mc)::value, i = kH + m / kB, j = m % kB;
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[1][j], fp[i], acc[i][j], 0, 0, 0);
    });
    MOE_WAIT_VM(0);   // the copies past the end still write LDS
  }
};

// The product of a tile with `rows` live rows: the K loop with the wave's share
// of the live row blocks.
template <class C, bool PX, bool QX>
__device__ __forceinline__ void multiply(uint8_t* smem, const Operands<C, PX, QX>& o, int rows, int length, int wave,
                                         int lane, bool later, f32x4_t (&acc)[2 * C::MI][2 * C::NJ]) {
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int stages = (length + C::STEP - 1) / C::STEP;
#pragma unroll
  for (int i = 0; i < 2 * C::MI; ++i)
#pragma unroll
    for (int j = 0; j < 2 * C::NJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  static_assert(C::MI == 1 || C::MI == 2 || C::MI == 4, "cases below");
  const int blocks = (rows + 31) / 32, live = (blocks - wm + C::WM - 1) / C::WM;   // this wave's
  if (live >= C::MI) Reduce<C, PX, QX, C::MI>::run(smem, o, stages, wm, wn, lane, later, acc);
  else if (C::MI > 3 && live == 3) Reduce<C, PX, QX, C::MI - 1>::run(smem, o, stages, wm, wn, lane, later, acc);
  else if (C::MI > 2 && live == 2) Reduce<C, PX, QX, 2>::run(smem, o, stages, wm, wn, lane, later, acc);
  else if (live == 1) Reduce<C, PX, QX, 1>::run(smem, o, stages, wm, wn, lane, later, acc);
  else Reduce<C, PX, QX, 0>::run(smem, o, stages, wm, wn, lane, later, acc);
}

// Workgroup barrier after a K loop: every wave is done reading the rings.
__device__ __forceinline__ void rings_free() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Stores a tile: rows 0..rows-1, columns 0..cols-1 from `out` on.  STREAM: the
// output passes the caches by.
//   16x16 D layout with Q first: lane holds output row l%16, columns
// 4 (l/16) + [0, 4).  The wave's blocks pass through LDS (the rings' last
// tiles, which a fill leaves alone), 32 rows at a time, and leave as whole
// rows, 16 bytes a lane: stored from the MFMA layout a row's line would be
// written in four parts (non-temporal stores of such parts took dw from 1.4 to
// 4.4 ms).  Chunks are permuted by chunk ^ row, for the banks.
template <class C, bool F32, bool STREAM>
__device__ __forceinline__ void store_tile(uint8_t* smem, const f32x4_t (&acc)[2 * C::MI][2 * C::NJ], int rows, int cols,
                                           int wave, int lane, void* out, long long ldo) {
  // the addresses below are made anew for every tile: kept across a K loop in
  // registers (they do not change with it), they would be spilled
  asm volatile("" : "+v"(lane));
  const int wm = wave / C::WN, wn = wave % C::WN;
  constexpr int kSize = F32 ? 4 : 2, kRowBytes = C::NJ * 32 * kSize, kChunks = kRowBytes / 16;
  constexpr int kMask = kChunks < 16 ? kChunks - 1 : 15;
  constexpr int kShift = kRowBytes >= 256 ? 0 : kRowBytes == 128 ? 1 : 2;   // rows side by side in the banks
  auto place = [](int r, int c) { return (c ^ ((r >> kShift) & kMask)) * 16; };   // chunk c of row r
  constexpr int kHalf = C::kWaves / 2, kQ = C::BN * C::STEP * 2, kP = C::BM * C::STEP * 2;   // waves, tile bytes
  static_assert(kHalf * 32 * kRowBytes <= kQ && kHalf * 32 * kRowBytes <= kP && 64 % kChunks == 0,
                "a block of every wave fits");
  // the last Q tile, and the end of the last P tile
  uint8_t* const stg = smem + (wave < kHalf ? (C::NQ - 1) * kQ + wave * (32 * kRowBytes)
                                            : C::kSmem - (wave - kHalf + 1) * (32 * kRowBytes));
  const int q = lane >> 4;
#pragma unroll
  for (int i = 0; i < C::MI; ++i) {
    const int r0 = (i * C::WM + wm) * 32;
    if (r0 >= rows) break;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 2 * C::NJ; ++j) {
        const f32x4_t& a = acc[2 * i + h][j];
        const int r = 16 * h + (lane & 15);
        uint8_t* const at = stg + r * kRowBytes;
        if constexpr (F32) *reinterpret_cast<f32x4_t*>(at + place(r, 4 * j + q)) = a;
        else *reinterpret_cast<uint2*>(at + place(r, 2 * j + (q >> 1)) + 8 * (q & 1)) =
            make_uint2(bf16_pair(a[0], a[1]), bf16_pair(a[2], a[3]));
      }
    asm volatile("" ::: "memory");
#pragma unroll
    for (int k = 0; k < kChunks / 2; ++k) {   // 64 / kChunks rows at a time
      const int r = k * (64 / kChunks) + lane / kChunks, c = lane % kChunks;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(stg + r * kRowBytes + place(r, c));
      const int col = wn * (C::NJ * 32) + c * (16 / kSize);
      u32x4_t* const to = reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(out) + ((long long)(r0 + r) * ldo + col) * kSize);
      if (r0 + r < rows && col < cols) {   // cols is a multiple of 8
        if constexpr (STREAM) __builtin_nontemporal_store(v, to);
        else *to = v;
      }
    }
    asm volatile("" ::: "memory");
  }
}

// How the (row tile, column slice) items are dealt to the XCDs: to `parts`
// (4, 2 or 1) shares of the slices and kXcds / parts turns of the row tiles.
// Each weight then crosses to kXcds / parts L2s only, and 32 concurrent
// workgroups of an XCD (one per CU) hold e.g. 8 row tiles x 4 slices: 12
// operand tiles to fetch per stage where 2 x 16 (every XCD all slices) need 18.
struct Deal {
  int slices, parts, share;   // share: slices per part, the last part may have fewer
};
inline Deal deal(int slices) {
  const int parts = slices % 4 == 0 || slices > 12 ? 4 : slices % 2 == 0 || slices > 4 ? 2 : 1;
  return {slices, parts, (slices + parts - 1) / parts};
}

// Item i of XCD `xcd`'s list: its row tile and column slice; false past the end.
template <class C>
__device__ __forceinline__ bool rows_place(const int32_t* offsets, int rows, int groups, const Deal& d, int xcd, int i,
                                           Tile& t, int& slice) {
  const int turn = i / d.share;
  slice = xcd % d.parts * d.share + i - turn * d.share;
  // a turn's tiles go round: groups of 1.5 tiles would else give one XCD the
  // full and another the half ones (dx of 32 groups of 384 rows: 821 -> 720 us)
  const int turns = kXcds / d.parts, tile = turn * turns + (xcd / d.parts + turn) % turns;
  if (slice >= d.slices) return false;
  const RowTiles tiles(offsets, groups, rows, C::BM, threadIdx.x & 63);
  if (tile >= tiles.total) return false;
  t = tiles.place(tile);
  return true;
}

// A reduction in `parts` parts of whole stages: part `part` of one of `length`.
template <int STEP>
__device__ __forceinline__ void part_range(int length, int parts, int part, int& from, int& len) {
  const int per = ((length + STEP - 1) / STEP + parts - 1) / parts * STEP;
  from = min(part * per, length);
  len = min(length - from, per);
}

// SPLIT: item i / parts, the part i % parts of its reduction, to `partial`
// [parts, rows, cols].
template <class C, bool QX, bool SPLIT>
struct RowsItem {
  static __device__ __forceinline__ void run(uint8_t* smem, const uint16_t* p, long long ldp, const uint16_t* w,
                                            const int32_t* offsets, int rows, int groups, int cols, int length, Deal d,
                                            uint16_t* out, int parts, float* partial, int xcd, int i) {
    Tile t;
    int slice, from = 0, len = length;
    const int part = SPLIT ? i % parts : 0;
    if (!rows_place<C>(offsets, rows, groups, d, xcd, SPLIT ? i / parts : i, t, slice)) return;
    if (SPLIT) part_range<C::STEP>(length, parts, part, from, len);
    const int c0 = slice * C::BN;
    const uint16_t* we = w + (size_t)t.e * cols * length + (QX ? (size_t)from * cols + c0 : (size_t)c0 * length + from);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int live_cols = min(C::BN, cols - c0);
    using O = Operands<C, false, QX>;
    const O o = {typename O::P(p + (long long)t.row0 * ldp + from, ldp, t.rows, len, wave, lane),
                 typename O::Q(we, QX ? cols : length, live_cols, len, wave, lane)};
    f32x4_t acc[2 * C::MI][2 * C::NJ];
    o.fill(smem);
    multiply(smem, o, t.rows, len, wave, lane, false, acc);
    rings_free();
    if constexpr (SPLIT)
      store_tile<C, true, false>(smem, acc, t.rows, live_cols, wave, lane,
                                 partial + ((size_t)part * rows + t.row0) * cols + c0, cols);
    else
      store_tile<C, false, false>(smem, acc, t.rows, live_cols, wave, lane, out + (long long)t.row0 * cols + c0, cols);
  }
};

// The sum of `parts` values `stride` apart, in the parts' order.
__device__ __forceinline__ f32x4_t join(const float* p, size_t stride, int parts) {
  f32x4_t v = *reinterpret_cast<const f32x4_t*>(p);
  for (int i = 1; i < parts; ++i) v += *reinterpret_cast<const f32x4_t*>(p + i * stride);
  return v;
}
__device__ __forceinline__ uint2 bf16_quad(f32x4_t v) {
  return make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
}

// Joins the parts of every item of the same deal: rows outside every group are
// left alone here too.
template <class C>
__global__ __launch_bounds__(C::kWaves* kWave) void grouped_join_rows(const float* partial, int parts,
                                                                      const int32_t* offsets, int rows, int groups,
                                                                      int cols, Deal d, uint16_t* out) {
  Tile t;
  int slice;
  if (!rows_place<C>(offsets, rows, groups, d, blockIdx.x % kXcds, blockIdx.x / kXcds, t, slice)) return;
  const int c0 = slice * C::BN, quads = min(C::BN, cols - c0) / 4;
  for (int i = threadIdx.x; i < t.rows * quads; i += C::kWaves * kWave) {
    const int r = i / quads;
    const size_t at = (size_t)(t.row0 + r) * cols + c0 + 4 * (i - r * quads);
    *reinterpret_cast<uint2*>(out + at) = bf16_quad(join(partial + at, (size_t)rows * cols, parts));
  }
}

template <bool F32>
__global__ __launch_bounds__(256) void grouped_join_dw(const float* partial, int parts, size_t total, void* dw) {
  const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= total) return;   // a multiple of 64
  const f32x4_t v = join(partial + at, total, parts);
  if constexpr (F32) *reinterpret_cast<f32x4_t*>(static_cast<float*>(dw) + at) = v;
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dw) + at) = bf16_quad(v);
}

// y = x w_e^T
template <class C, bool SPLIT>
__global__ __launch_bounds__(C::kWaves* kWave, C::kPerCU* C::kWaves / 4) void grouped_forward(
    const uint16_t* x, long long ldx, const uint16_t* w, const int32_t* offsets, int rows, int groups, int n, int k,
    Deal d, uint16_t* out, int parts, float* partial) {
  __shared__ __align__(1024) uint8_t smem[C::kSmem];
  RowsItem<C, false, SPLIT>::run(smem, x, ldx, w, offsets, rows, groups, n, k, d, out, parts, partial, blockIdx.x % kXcds,
                             blockIdx.x / kXcds);
}

struct BackwardArgs {
  const uint16_t *dy, *x, *w;
  long long lddy, ldx;
  const int32_t* offsets;
  int rows, groups, n, k;
  uint16_t* dx;
  void* dw;
  Deal dx_deal;
  int dx_items, dw_items;   // per XCD (dx: at most)
  int dw_groups;            // workgroups that share an XCD's dw items
  int dx_parts, dw_parts;   // parts of a reduction, each a dx or dw item
  float *dx_partial, *dw_partial;   // [parts] dx and dw in fp32
};

// Tile `id` of dw: a group's tiles in bands of eight tile rows, whose
// concurrent ones share their columns of dy and x.
// A group's own two offsets count, clamped: every group has an output of its own.
struct DwTile {
  int e, n0, k0, lo, length, rows, cols, part;
};
template <class C>
__device__ __forceinline__ DwTile dw_tile(const BackwardArgs& a, int id) {
  const int mtiles = (a.n + C::BM - 1) / C::BM, ntiles = (a.k + C::BN - 1) / C::BN, per = mtiles * ntiles;
  DwTile t;
  t.e = id / per;
  const int j = id - t.e * per;
  constexpr int kBand = 8;
  const int band = j / (kBand * ntiles), in = j - band * kBand * ntiles, high = min(kBand, mtiles - band * kBand);
  t.n0 = (band * kBand + in % high) * C::BM;
  t.k0 = in / high * C::BN;
  t.lo = min(max(a.offsets[t.e], 0), a.rows);
  t.length = min(max(a.offsets[t.e + 1], t.lo), a.rows) - t.lo;
  t.rows = min(C::BM, a.n - t.n0);
  t.cols = min(C::BN, a.k - t.k0);
  return t;
}

// dw: workgroup i of its XCD's `stride` takes tiles i, i + stride, .. of the
// XCD's share.  A tile is short (384 rows are six stages) and its output large
// (256 KB in fp32), so the next tile's rings are filled before this one is
// stored: the fill's latency and the stores overlap.
template <class C, bool F32, bool STREAM, bool SPLIT>
__device__ __forceinline__ void dw_share(uint8_t* smem, const BackwardArgs& a, int xcd, int i, int stride) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = ((a.n + C::BM - 1) / C::BM) * ((a.k + C::BN - 1) / C::BN);
  const int parts = SPLIT ? a.dw_parts : 1, end = min((xcd + 1) * a.dw_items, a.groups * per * parts);
  auto tile = [&](int id) {
    DwTile t = dw_tile<C>(a, SPLIT ? id / parts : id);
    t.part = 0;
    if (SPLIT) {
      int from, len;
      t.part = id % parts;
      part_range<C::STEP>(t.length, parts, t.part, from, len);
      t.lo += from;
      t.length = len;
    }
    return t;
  };
  int id = xcd * a.dw_items + i;
  if (id >= end) return;
  using O = Operands<C, true, true>;
  auto operands = [&](const DwTile& t) {
    return O{typename O::P(a.dy + (long long)t.lo * a.lddy + t.n0, a.lddy, t.rows, t.length, wave, lane),
             typename O::Q(a.x + (long long)t.lo * a.ldx + t.k0, a.ldx, t.cols, t.length, wave, lane)};
  };
  DwTile t = tile(id);
  O o = operands(t);
  o.fill(smem);
  bool later = false;
  for (;;) {
    f32x4_t acc[2 * C::MI][2 * C::NJ];
    multiply(smem, o, t.rows, t.length, wave, lane, later, acc);
    rings_free();
    id += stride;
    const DwTile done = t;
    if (id < end) {
      t = tile(id);
      o = operands(t);
      o.fill(smem);
    }
    const size_t at = ((size_t)(done.part * a.groups + done.e) * a.n + done.n0) * a.k + done.k0;
    float* const f32 = SPLIT ? a.dw_partial : static_cast<float*>(a.dw);
    void* to = F32 ? static_cast<void*>(f32 + at) : static_cast<void*>(static_cast<uint16_t*>(a.dw) + at);
    store_tile<C, F32, STREAM>(smem, acc, done.rows, done.cols, wave, lane, to, a.k);
    if (id >= end) return;
    // every store of a full tile was issued, so the next K loop's first wait need not cover them
    later = F32 && C::MI * C::NJ * 4 >= kLater && done.rows == C::BM && done.cols == C::BN;
  }
}

// Both gradients in one launch, an XCD's dx items (tiles in shape X) and then
// its dw workgroups, whose stores end the launch: 32 groups of 384 rows,
// 4096 x 7168, take 1838 us, dw first 1860; 4 groups of 75 rows, 2048 x 1024,
// 19.6 and 22.7.  (Mixed in proportion, so that some CUs would write while
// others multiply, was no better than dw first.)
template <class C, class X, bool F32, bool STREAM, bool SPLIT_DX, bool SPLIT_DW>
__global__ __launch_bounds__(C::kWaves* kWave, C::kPerCU* C::kWaves / 4) void grouped_backward(BackwardArgs a) {
  static_assert(C::kWaves == X::kWaves, "one workgroup size");
  __shared__ __align__(1024) uint8_t smem[C::kSmem > X::kSmem ? C::kSmem : X::kSmem];
  const int xcd = blockIdx.x % kXcds, i = blockIdx.x / kXcds;
  if (i < a.dx_items)
    RowsItem<X, true, SPLIT_DX>::run(smem, a.dy, a.lddy, a.w, a.offsets, a.rows, a.groups, a.k, a.n, a.dx_deal, a.dx,
                                 a.dx_parts, a.dx_partial, xcd, i);
  else dw_share<C, F32, STREAM, SPLIT_DW>(smem, a, xcd, i - a.dx_items, a.dw_groups);
}

// items per XCD there can be with row tiles of bm rows
long long items_per_xcd(const GroupedArgs& a, int bm, const Deal& d) {
  const int turns = kXcds / d.parts;
  return ((long long)a.rows / bm + std::min(a.groups, a.rows) + turns - 1) / turns * d.share;
}

template <int WN>
using Large = Shape<256, 256, 2, WN, 64, 2, 3, 1>;
template <bool NT>
using Middle = Shape<128, 128, 2, 2, 64, 2, 3, 2, NT>;
template <bool NT>
using Small = Shape<64, 128, 1, 4, 64, 3, 3, 2, NT>;

// items there will be, about: half the groups end in a partial tile
template <class C>
long long items(const GroupedArgs& a, int cols) {
  return ((long long)a.rows / C::BM + (std::min(a.groups, a.rows) + 1) / 2) * ((cols + C::BN - 1) / C::BN);
}

// Parts of a reduction of `stages` stages for a launch of `items` workgroups:
// few items leave CUs idle, each taking 0.3 us a stage (dw 0.5).  The second
// launch and the workspace cost the host 5 us, so only long sums gain (718 rows,
// 6672 -> 64, 12 items of 105 stages: 28.9 -> 14.6 us; dw of 6566 rows, 584 x
// 184, 10 of 103: 58 -> 19; dx of 100 rows in two groups, 4096 x 512, 8 of 64:
// 24.9 -> 16.7), not short ones (300 rows in two groups, 2048 -> 2048, 32
// stages: 12.7 -> 20.6) or many items, which fill the memory (10 rows in 18
// groups, 5552 -> 2216, 90 of 87: 53 -> 60).
int parts_for(long long items, long long stages) {
  if (items > 64 || stages < 50) return 1;
  return (int)std::min(stages / 8, 256 / std::max(items, 1LL));
}

struct Parts {
  int dx = 1, dw = 1;   // dx: of the forward product's y too
  size_t dx_floats = 0, dw_floats = 0;
  size_t bytes() const { return (dx > 1 ? dx * dx_floats : 0) * 4 + (dw > 1 ? dw * dw_floats : 0) * 4; }
};
Parts forward_parts(const GroupedArgs& a) {
  Parts p;
  p.dx_floats = (size_t)a.rows * a.n;
  p.dx = parts_for(items<Small<false>>(a, a.n), (a.k + 63) / 64);
  return p;
}
Parts backward_parts(const GroupedArgs& a, bool dx, bool dw) {
  Parts p;
  p.dx_floats = (size_t)a.rows * a.k;
  p.dw_floats = (size_t)a.groups * a.n * a.k;
  if (dx) p.dx = parts_for(items<Small<false>>(a, a.k), (a.n + 63) / 64);
  if (dw)
    p.dw = parts_for((long long)a.groups * ((a.n + 127) / 128) * ((a.k + 127) / 128), a.rows / a.groups / 64);
  return p;
}

template <class C>
hipError_t launch_join_rows(const GroupedArgs& a, int cols, const Deal& d, int parts, const float* partial, void* out,
                            hipStream_t stream) {
  hipLaunchKernelGGL((grouped_join_rows<C>), dim3((unsigned)(items_per_xcd(a, C::BM, d) * kXcds)),
                     dim3(C::kWaves * kWave), 0, stream, partial, parts, a.offsets, a.rows, a.groups, cols, d,
                     static_cast<uint16_t*>(out));
  return hipGetLastError();
}

template <class C, bool SPLIT = false>
hipError_t launch_forward(const GroupedArgs& a, const void* x, int64_t ldx, void* y, hipStream_t stream, int parts = 1,
                          float* partial = nullptr) {
  // a weight read once is best read beside its neighbours: one share
  const int slices = (a.n + C::BN - 1) / C::BN;
  const Deal d = C::NT ? Deal{slices, 1, slices} : deal(slices);
  hipLaunchKernelGGL((grouped_forward<C, SPLIT>), dim3((unsigned)(items_per_xcd(a, C::BM, d) * kXcds * parts)),
                     dim3(C::kWaves * kWave), 0, stream, static_cast<const uint16_t*>(x), ldx,
                     static_cast<const uint16_t*>(a.w), a.offsets, a.rows, a.groups, a.n, a.k, d,
                     static_cast<uint16_t*>(y), parts, partial);
  if (const hipError_t e = hipGetLastError()) return e;
  return SPLIT ? launch_join_rows<C>(a, a.n, d, parts, partial, y, stream) : hipSuccess;
}

template <class C, class X, bool SPLIT_DX = false, bool SPLIT_DW = false>
hipError_t launch_backward(const GroupedArgs& a, BackwardArgs b, bool f32, hipStream_t stream) {
  b.dx_deal = deal((a.k + X::BN - 1) / X::BN);
  b.dx_items = b.dx ? (int)items_per_xcd(a, X::BM, b.dx_deal) * b.dx_parts : 0;
  const long long dw_tiles = (long long)a.groups * ((a.n + C::BM - 1) / C::BM) * ((a.k + C::BN - 1) / C::BN);
  b.dw_items = b.dw ? (int)((dw_tiles * b.dw_parts + kXcds - 1) / kXcds) : 0;
  b.dw_groups = std::min(b.dw_items, kCusPerXcd * C::kPerCU);   // as many as run at once
  if (b.dx_items + b.dw_items == 0) return hipSuccess;
  // dw beyond the L2s' 32 MB leaves nothing there to read again and would
  // push dy and x out: streamed (3.76 GB: 1259 -> 1091 us)
  const size_t total = (size_t)a.groups * a.n * a.k;
  const bool stream_out = total * (f32 ? 4 : 2) > kL2Bytes;
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(b.dx_items + b.dw_groups) * kXcds), dim3(C::kWaves * kWave), 0, stream, b);
  };
  if constexpr (SPLIT_DW) run(grouped_backward<C, X, true, false, SPLIT_DX, true>);
  else if (f32)
    run(stream_out ? grouped_backward<C, X, true, true, SPLIT_DX, false>
                   : grouped_backward<C, X, true, false, SPLIT_DX, false>);
  else
    run(stream_out ? grouped_backward<C, X, false, true, SPLIT_DX, false>
                   : grouped_backward<C, X, false, false, SPLIT_DX, false>);
  if (const hipError_t e = hipGetLastError()) return e;
  if constexpr (SPLIT_DX)
    if (const hipError_t e = launch_join_rows<X>(a, a.k, b.dx_deal, b.dx_parts, b.dx_partial, b.dx, stream)) return e;
  if constexpr (SPLIT_DW) {
    const dim3 grid((unsigned)((total / 4 + 255) / 256));
    if (f32) hipLaunchKernelGGL((grouped_join_dw<true>), grid, dim3(256), 0, stream, b.dw_partial, b.dw_parts, total, b.dw);
    else hipLaunchKernelGGL((grouped_join_dw<false>), grid, dim3(256), 0, stream, b.dw_partial, b.dw_parts, total, b.dw);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t grouped_forward_workspace(const GroupedArgs& a) { return forward_parts(a).bytes(); }
size_t grouped_backward_workspace(const GroupedArgs& a, bool dx, bool dw) { return backward_parts(a, dx, dw).bytes(); }

// Tile by the rows a group has on average (64 groups, 7168 -> 4096, us with
// 64-, 128- and 256-row tiles, the first two non-temporal): few rows stream the
// weights, which two workgroups per CU, non-temporal, do best (16 rows each:
// 550, 551, 612; 224 groups of 2.7 rows, 2048 -> 7168: 927, 988, 1135), but a
// group of more rows than a tile reads them again (32 rows each 572, 578, 619,
// Zipf-skewed 741, 681, 694; 64 each 888, 632, 640, skewed 1007, 842, 705; 128
// each 1553, 1055, 691).  The 256-row tile has four waves of 128 x 128, which
// read two thirds of what eight of 128 x 64 do from LDS (eight groups of 4096
// rows, at the power limit: 1412 against 1451 us).  Grids that would leave CUs
// idle take the next smaller tile (600 rows in 8 groups, 768 -> 1024: 8.2, 9.1,
// 13.5).
hipError_t launch_grouped_forward(const GroupedArgs& a, const void* x, int64_t ldx, void* y, void* workspace,
                                  hipStream_t stream) {
  const long long rows = a.rows;
  if (workspace) {
    const int parts = forward_parts(a).dx;
    float* const partial = static_cast<float*>(workspace);
    if (parts > 1 && rows <= 16LL * a.groups) return launch_forward<Small<true>, true>(a, x, ldx, y, stream, parts, partial);
    if (parts > 1) return launch_forward<Small<false>, true>(a, x, ldx, y, stream, parts, partial);
  }
  if (rows <= 16LL * a.groups) return launch_forward<Small<true>>(a, x, ldx, y, stream);
  if (rows <= 40LL * a.groups && items<Middle<true>>(a, a.n) >= 256)
    return launch_forward<Middle<true>>(a, x, ldx, y, stream);
  if (rows > 40LL * a.groups && items<Large<2>>(a, a.n) >= 256) return launch_forward<Large<2>>(a, x, ldx, y, stream);
  if (items<Middle<false>>(a, a.n) >= 256) return launch_forward<Middle<false>>(a, x, ldx, y, stream);
  return launch_forward<Small<false>>(a, x, ldx, y, stream);
}

// 256 x 256 tiles, in eight waves (four took 2038 us where eight took 1966:
// dw's short sums and large stores leave a wave alone idle), where they fill
// the CUs (32 groups of 384 rows, 4096 x 7168: 1870 us against 2390 with
// 128 x 128), else 128 x 128 (8 groups of 75 rows, 768 x 1024: 19.1 against
// 11.7).  dx takes 64-row tiles, whose rings are deeper, where those leave CUs
// to dw or to more of them (dx alone, 8 groups of 75 rows and of 256, 768 x
// 1024: 7.6 against 9.6 us and 8.6 against 10.4; with dw 10.8 against 11.6, but
// 14.9 against 13.2).
hipError_t launch_grouped_backward(const GroupedArgs& a, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                   void* dx, bool f32, void* dw, void* workspace, hipStream_t stream) {
  const BackwardArgs b{static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(x),
                       static_cast<const uint16_t*>(a.w), lddy, ldx, a.offsets, a.rows, a.groups, a.n, a.k,
                       static_cast<uint16_t*>(dx), dw, {}, 0, 0, 0, 1, 1, nullptr, nullptr};
  const bool small = items<Small<false>>(a, a.k) <= (dw ? 256 : 512);
  if (workspace) {
    const Parts p = backward_parts(a, dx, dw);
    BackwardArgs s = b;
    s.dx_parts = p.dx;
    s.dw_parts = p.dw;
    s.dx_partial = static_cast<float*>(workspace);
    s.dw_partial = s.dx_partial + (p.dx > 1 ? p.dx * p.dx_floats : 0);
    if (p.dx > 1 && p.dw > 1) return launch_backward<Middle<false>, Small<false>, true, true>(a, s, f32, stream);
    if (p.dx > 1) return launch_backward<Middle<false>, Small<false>, true, false>(a, s, f32, stream);
    if (p.dw > 1 && small) return launch_backward<Middle<false>, Small<false>, false, true>(a, s, f32, stream);
    if (p.dw > 1) return launch_backward<Middle<false>, Middle<false>, false, true>(a, s, f32, stream);
  }
  const long long dw_tiles = (long long)a.groups * ((a.n + 255) / 256) * ((a.k + 255) / 256);
  const bool large = dw ? dw_tiles >= 256 : items<Large<4>>(a, a.k) >= 256 && a.rows > 40LL * a.groups;
  if (large) return launch_backward<Large<4>, Large<4>>(a, b, f32, stream);
  if (small) return launch_backward<Middle<false>, Small<false>>(a, b, f32, stream);
  return launch_backward<Middle<false>, Middle<false>>(a, b, f32, stream);
}

}  // namespace moe
