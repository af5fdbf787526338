// Products of ragged groups of rows with one bf16 matrix per group (a routed
// layer's unquantised experts), and their gradients.  Rows offsets[e] ..
// offsets[e+1]-1 of x [R, K] belong to group e with w_e [N, K]:
//   forward    y_r  = w_e x_r                       reduction over K
//   dx         dx_r = dy_r w_e                      reduction over N
//   dw         dw_e = sum over e's rows dy_r x_r^T  reduction over the rows
// One tile kernel on v_mfma_f32_32x32x16_bf16 serves the three: an output tile
// of BM x BN is the product of a row operand P (output rows) and a column
// operand Q (output columns) over 64 of the reduction at a time.  An operand
// lies in memory either along its reduction ("plain": x and w forward, dy for
// dx) or across it ("crossed": w for dx; dy and x for dw); a crossed operand
// is staged as it lies and read through ds_read_b64_tr_b16, which hands each
// lane one column's four consecutive reduction values, so nothing is
// transposed in memory.
//
// Staging: buffer_load ... lds copies of 1 KB per wave instruction into a ring
// of kSlots stages, loaded kSlots - 1 stages ahead.  Addresses past an edge
// (rows past the group, reduction past its length, columns past the matrix)
// get an out-of-range offset, for which the copy writes zeros: no other
// group's row, NaN or not, enters a sum.
//   plain tile: 128-byte rows of 64 reduction values whose eight 16-byte
//     chunks are permuted by chunk ^ (row & 7) ^ ((row >> 3) & 1), which
//     spreads a quarter-wave's ds_read_b128 over all 64 banks;
//   crossed tile: 64 rows (the reduction) of BM or BN columns whose 64-byte
//     units are permuted by unit ^ (row & 3): the four rows a transposed read
//     takes lie in four different units, again all 64 banks.
// Both operands number the reduction alike, so every output is one fp32 sum
// in ascending order of 16 values an MFMA, whatever the tile.
//
// Q is the instruction's first operand: a lane then ends with four
// consecutive columns of one output row, stored together.
#include <algorithm>

#include "moe_internal.h"

namespace moe {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr int kStep = 64;                      // reduction per stage
constexpr uint32_t kPastEnd = 0x80000000u;     // beyond every buffer resource below
constexpr int kMaxRange = 0x7FFFFFFF;          // bytes a resource covers

// vmcnt <= n and lgkmcnt 0
#define MOE_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (7 << 4) | ((((n) >> 4) & 3) << 14))

__device__ __forceinline__ int swz(int c, int r) { return c ^ (r & 7) ^ ((r >> 3) & 1); }

// One operand's tile of B rows (plain) or columns (crossed), `count` of them
// live, over `length` of the reduction; `base` is its first element and `ld`
// the elements from one memory row to the next.
template <bool CROSSED, int B, int WAVES>
struct Operand {
  static constexpr int kBytes = B * kStep * 2;
  static constexpr int kCopies = kBytes / 1024 / WAVES;   // copies per wave and stage
  static constexpr int kChunks = B / 8;                   // crossed: 16-byte chunks per staged row
  static_assert(!CROSSED || B >= 128, "four 64-byte units to permute");
  static_assert(kCopies * WAVES * 1024 == kBytes, "copies split evenly");

  const uint16_t* base;
  long long ld;
  int length;
  int wave;
  uint32_t off[kCopies];   // byte offset of this lane's chunk at stage 0 (kPastEnd: not live)
  int red[kCopies];        // reduction index of its first value at stage 0

  __device__ __forceinline__ Operand(const uint16_t* b, long long l, int count, int len, int w, int lane)
      : base(b), ld(l), length(len), wave(w) {
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const int i = wave + WAVES * j;
      if constexpr (!CROSSED) {
        const int r = 8 * i + (lane >> 3), c = swz(lane & 7, r);
        red[j] = 8 * c;
        off[j] = r < count ? (uint32_t)((long long)r * ld * 2) + 16 * c : kPastEnd;
      } else {
        constexpr int kRows = 64 / kChunks;   // staged rows per copy
        const int r = kRows * i + lane / kChunks, c = (lane % kChunks) ^ ((r & 3) << 2);
        red[j] = r;
        off[j] = 8 * c < count ? (uint32_t)((long long)r * ld * 2) + 16 * c : kPastEnd;
      }
    }
  }

  // copies of stage s into `buf`
  __device__ __forceinline__ void issue(uint8_t* buf, int s) const {
    const long long skip = (long long)s * kStep * (CROSSED ? ld : 1);
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base + skip), (short)0, kMaxRange, kRsrcWord3);
#pragma unroll
    for (int j = 0; j < kCopies; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(buf + (wave + WAVES * j) * 1024), 16,
                                               red[j] + s * kStep < length ? off[j] : kPastEnd, 0, 0, 0);
  }

  // MFMA operand of 32-row block b, 16-deep step k, from a staged tile
  static __device__ __forceinline__ bf16x8_t read(const uint8_t* buf, int b, int k, int lane) {
    const int h = lane >> 5;
    if constexpr (!CROSSED) {
      const int r = lane & 31;
      return *reinterpret_cast<const bf16x8_t*>(buf + (b * 32 + r) * 128 + swz(2 * k + h, r) * 16);
    } else {
      // lane i of 16 points at row i/4 and columns 4 (i%4).. of a 4 x 16 block
      const int i = lane & 15, g = (lane >> 4) & 1;
      const uint8_t* p = buf + (16 * k + 8 * h + (i >> 2)) * (B * 2) + ((b ^ (i >> 2)) * 4 + 2 * g + ((i >> 1) & 1)) * 16 +
                         (i & 1) * 8;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * (B * 2)));
      const s16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      return __builtin_bit_cast(bf16x8_t, v);
    }
  }
};

// The group and first row of row tile `tile` (tiles of BM rows, groups in
// order), or e = -1 past the last one.  Offsets are clamped to [0, rows] and
// to their predecessor, so no offset leads outside the tensors.  Every wave
// finds it by itself: a lane counts the tiles of ceil(groups / 64) groups, a
// wave scan gives each lane its first tile.
struct Tile { int e, row0, rows; };
__device__ __forceinline__ Tile find_tile(const int32_t* offsets, int groups, int rows, int bm, int tile, int lane) {
  const int per = (groups + kWave - 1) / kWave;
  const int e0 = lane * per, e1 = min(e0 + per, groups);
  int mine = 0;
  for (int e = e0; e < e1; ++e) {
    const int lo = min(max(offsets[e], 0), rows), hi = min(max(offsets[e + 1], lo), rows);
    mine += (hi - lo + bm - 1) / bm;
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int v = __shfl_up(upto, d, kWave);
    if (lane >= d) upto += v;
  }
  Tile t = {-1, 0, 0};
  int first = upto - mine;
  if (tile >= first && tile < upto) {
    for (int e = e0; e < e1; ++e) {
      const int lo = min(max(offsets[e], 0), rows), hi = min(max(offsets[e + 1], lo), rows);
      const int n = (hi - lo + bm - 1) / bm;
      if (tile < first + n) {
        t.e = e;
        t.row0 = lo + (tile - first) * bm;
        t.rows = min(bm, hi - t.row0);
        break;
      }
      first += n;
    }
  }
  const uint64_t owner = __ballot(t.e >= 0);
  if (owner == 0) return t;
  const int src = __ffsll((unsigned long long)owner) - 1;
  t.e = __builtin_amdgcn_readfirstlane(__shfl(t.e, src, kWave));
  t.row0 = __builtin_amdgcn_readfirstlane(__shfl(t.row0, src, kWave));
  t.rows = __builtin_amdgcn_readfirstlane(__shfl(t.rows, src, kWave));
  return t;
}

template <int BM_, int BN_, int WM_, int WN_, int SLOTS_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, kSlots = SLOTS_;
  static constexpr int kWaves = WM * WN;
  static constexpr int MI = BM / WM / 32, NJ = BN / WN / 32;
  static constexpr int kSlotBytes = (BM + BN) * kStep * 2;
};

// One output tile: rows 0..rows-1, columns 0..cols-1 from `out` on.
template <class C, bool PX, bool QX, bool F32>
__device__ __forceinline__ void tile_product(uint8_t* smem, const uint16_t* p, long long ldp, const uint16_t* q,
                                             long long ldq, int rows, int cols, int length, void* out, long long ldo) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  using P = Operand<PX, C::BM, C::kWaves>;
  using Q = Operand<QX, C::BN, C::kWaves>;
  const P op(p, ldp, rows, length, wave, lane);
  const Q oq(q, ldq, cols, length, wave, lane);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int stages = (length + kStep - 1) / kStep;
  constexpr int D = C::kSlots - 1, G = P::kCopies + Q::kCopies;
  f32x16_t acc[C::MI][C::NJ];
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

#pragma unroll
  for (int d = 0; d < D; ++d) {
    op.issue(smem + d * C::kSlotBytes, d);
    oq.issue(smem + d * C::kSlotBytes + P::kBytes, d);
  }
  int slot = 0;
  for (int s = 0; s < stages; ++s) {
    // this wave's copies of stage s have landed and its reads of stage s - 1
    // are done; the barrier extends both to every wave
    MOE_WAIT_VM((D - 1) * G);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const int next = slot == 0 ? C::kSlots - 1 : slot - 1;   // stage s - 1's slot
    op.issue(smem + next * C::kSlotBytes, s + D);
    oq.issue(smem + next * C::kSlotBytes + P::kBytes, s + D);
    const uint8_t* bp = smem + slot * C::kSlotBytes;
    const uint8_t* bq = bp + P::kBytes;
#pragma unroll
    for (int k = 0; k < kStep / 16; ++k) {
      bf16x8_t fp[C::MI], fq[C::NJ];
#pragma unroll
      for (int i = 0; i < C::MI; ++i) fp[i] = P::read(bp, wm * C::MI + i, k, lane);
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) fq[j] = Q::read(bq, wn * C::NJ + j, k, lane);
#pragma unroll
      for (int i = 0; i < C::MI; ++i)
#pragma unroll
        for (int j = 0; j < C::NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fq[j], fp[i], acc[i][j], 0, 0, 0);
    }
    slot = slot + 1 == C::kSlots ? 0 : slot + 1;
  }
  MOE_WAIT_VM(0);   // the copies past the end still write LDS

  // 32x32 D layout with Q first: lane holds output row l%32, columns 8(r/4) + 4(l/32) + r%4
  const int h = lane >> 5;
#pragma unroll
  for (int i = 0; i < C::MI; ++i) {
    const int row = (wm * C::MI + i) * 32 + (lane & 31);
    if (row >= rows) continue;
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int col = (wn * C::NJ + j) * 32 + 8 * t + 4 * h;
        if (col >= cols) continue;   // cols is a multiple of 8
        const f32x16_t& a = acc[i][j];
        if constexpr (F32) {
          *reinterpret_cast<float4*>(static_cast<float*>(out) + (long long)row * ldo + col) =
              make_float4(a[4 * t], a[4 * t + 1], a[4 * t + 2], a[4 * t + 3]);
        } else {
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + (long long)row * ldo + col) =
              make_uint2(f32_to_bf16_rne(a[4 * t]) | ((uint32_t)f32_to_bf16_rne(a[4 * t + 1]) << 16),
                         f32_to_bf16_rne(a[4 * t + 2]) | ((uint32_t)f32_to_bf16_rne(a[4 * t + 3]) << 16));
        }
      }
  }
}

// forward (QX false: w_e [cols, length]) and dx (QX true: w_e [length, cols]).
template <class C, bool QX>
__global__ __launch_bounds__(C::kWaves* kWave) void grouped_rows(const uint16_t* p, long long ldp, const uint16_t* w,
                                                                 const int32_t* offsets, int rows, int groups, int cols,
                                                                 int length, int slices, uint16_t* out) {
  __shared__ __align__(1024) uint8_t smem[C::kSlots * C::kSlotBytes];
  const int tile = blockIdx.x / slices, slice = blockIdx.x - tile * slices;
  const Tile t = find_tile(offsets, groups, rows, C::BM, tile, threadIdx.x & 63);
  if (t.e < 0) return;
  const int c0 = slice * C::BN;
  const uint16_t* we = w + (size_t)t.e * cols * length;
  tile_product<C, false, QX, false>(smem, p + (long long)t.row0 * ldp, ldp, QX ? we + c0 : we + (size_t)c0 * length,
                                    QX ? cols : length, t.rows, min(C::BN, cols - c0), length,
                                    out + (long long)t.row0 * cols + c0, cols);
}

// dw: [n, k] per group
template <class C, bool F32>
__global__ __launch_bounds__(C::kWaves* kWave) void grouped_dw(const uint16_t* dy, long long lddy, const uint16_t* x,
                                                               long long ldx, const int32_t* offsets, int rows, int n,
                                                               int k, int mtiles, int ntiles, void* out) {
  __shared__ __align__(1024) uint8_t smem[C::kSlots * C::kSlotBytes];
  const int per = mtiles * ntiles, e = blockIdx.x / per, i = blockIdx.x - e * per;
  const int n0 = i / ntiles * C::BM, k0 = i % ntiles * C::BN;
  const int lo = min(max(offsets[e], 0), rows), hi = min(max(offsets[e + 1], lo), rows);
  const size_t at = ((size_t)e * n + n0) * k + k0;
  void* o = F32 ? static_cast<void*>(static_cast<float*>(out) + at) : static_cast<void*>(static_cast<uint16_t*>(out) + at);
  tile_product<C, true, true, F32>(smem, dy + (long long)lo * lddy + n0, lddy, x + (long long)lo * ldx + k0, ldx,
                                   min(C::BM, n - n0), min(C::BN, k - k0), hi - lo, o, k);
}

using Tile128 = Shape<128, 128, 2, 2, 3>;

template <bool QX>
hipError_t launch_rows(const GroupedArgs& a, const void* p, int64_t ldp, int cols, int length, void* out,
                       hipStream_t stream) {
  using C = Tile128;
  const int slices = (cols + C::BN - 1) / C::BN;
  const long long tiles = a.rows / C::BM + std::min(a.groups, a.rows);
  hipLaunchKernelGGL((grouped_rows<C, QX>), dim3((unsigned)(tiles * slices)), dim3(C::kWaves * kWave), 0, stream,
                     static_cast<const uint16_t*>(p), ldp, static_cast<const uint16_t*>(a.w), a.offsets, a.rows, a.groups,
                     cols, length, slices, static_cast<uint16_t*>(out));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_forward(const GroupedArgs& a, const void* x, int64_t ldx, void* y, hipStream_t stream) {
  return launch_rows<false>(a, x, ldx, a.n, a.k, y, stream);
}

hipError_t launch_grouped_dx(const GroupedArgs& a, const void* dy, int64_t lddy, void* dx, hipStream_t stream) {
  return launch_rows<true>(a, dy, lddy, a.k, a.n, dx, stream);
}

hipError_t launch_grouped_dw(const GroupedArgs& a, const void* dy, int64_t lddy, const void* x, int64_t ldx, bool f32,
                             void* dw, hipStream_t stream) {
  using C = Tile128;
  const int mt = (a.n + C::BM - 1) / C::BM, nt = (a.k + C::BN - 1) / C::BN;
  const dim3 grid((unsigned)((long long)a.groups * mt * nt)), block(C::kWaves * kWave);
  if (f32)
    hipLaunchKernelGGL((grouped_dw<C, true>), grid, block, 0, stream, static_cast<const uint16_t*>(dy), lddy,
                       static_cast<const uint16_t*>(x), ldx, a.offsets, a.rows, a.n, a.k, mt, nt, dw);
  else
    hipLaunchKernelGGL((grouped_dw<C, false>), grid, block, 0, stream, static_cast<const uint16_t*>(dy), lddy,
                       static_cast<const uint16_t*>(x), ldx, a.offsets, a.rows, a.n, a.k, mt, nt, dw);
  return hipGetLastError();
}

}  // namespace moe
