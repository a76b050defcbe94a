// experts.hip -- the experts' products over the expert-contiguous rows that
// the dispatch makes, in e4m3 with block scales:
//   y[r, n] = sum_b sa[r, b] * sb[e, n/128, b] * sum_{k in block b} a[r, k] * w[e, n, k]
// for the rows r of expert e, b over the 128-channel blocks of the row, and
// the gated form
//   h[r, c] = silu(y[r, c]) * y[r, I + c],  quantised to e4m3 per 128 channels.
//
// One matrix instruction multiplies a whole 128-channel block (16 x 16 x
// 128, e4m3 operands, fp32 sums), so each block's partial sum starts from
// zero in the instruction and one fused multiply-add per element folds it,
// with its two scales, into the running fp32 sum.  The weights are the
// instruction's first operand: a lane then holds four consecutive output
// channels of ONE row, so the row's scale is one register per lane, the
// weights' scale is the same for the whole wave, and the output leaves in
// 8-byte stores.
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

#define MOE_INLINE __attribute__((always_inline))

constexpr int kScaleBlock = 128;  // channels per scale

// Rows of expert e that lie inside the buffer: [start, start + rows).
__device__ __forceinline__ void segment_of(const int32_t* __restrict__ counts,
                                           const int32_t* __restrict__ send, int64_t cap,
                                           int e, int32_t& start, int32_t& rows, bool& cut) {
  const int64_t s = send ? send[e] : 0, c = counts ? counts[e] : cap;
  cut = s < 0 || c < 0 || (c > 0 && s + c > cap);
  const bool none = s < 0 || c <= 0 || s >= cap;
  start = none ? 0 : (int32_t)s;
  rows = none ? 0 : (int32_t)(c < cap - s ? c : cap - s);
}

// The row tiles of all experts, from the device's counts: first[e] is the
// number of tiles before expert e, first[E] their total.  Sums saturate at
// kMostTiles, above what disjoint segments of 2^30 rows can make, so counts
// whose segments overlap cannot wrap them; such counts give no tiles at all.
constexpr int kMostTiles = 1 << 30;

template <int THREADS>
struct TileMap {
  int first[kMaxExperts + 1];
  int start[kMaxExperts];
  int rows[kMaxExperts];
  int wave_sum[THREADS / kWave];
};

template <int THREADS>
__device__ __forceinline__ void build_tile_map(TileMap<THREADS>& map,
                                               const int32_t* __restrict__ counts,
                                               const int32_t* __restrict__ send, int32_t E,
                                               int64_t cap, int tile_rows, int32_t* status) {
  constexpr int kPer = (kMaxExperts + THREADS - 1) / THREADS;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  int n[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    n[i] = 0;
    if (e < E) {
      bool cut;
      segment_of(counts, send, cap, e, map.start[e], map.rows[e], cut);
      n[i] = (map.rows[e] + tile_rows - 1) / tile_rows;
      if (cut && status && blockIdx.x == 0) atomicOr(status, (int)MOE_FLAG_GUARD);
    }
    sum = min(sum + n[i], kMostTiles);
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int up = __shfl_up(incl, d, kWave);
    if (lane >= d) incl = min(incl + up, kMostTiles);
  }
  if (lane == kWave - 1) map.wave_sum[wave] = incl;
  __syncthreads();
  int base = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / kWave; ++w) {
    if (w < wave) base = min(base + map.wave_sum[w], kMostTiles);
    total = min(total + map.wave_sum[w], kMostTiles);
  }
  const bool overlap = total > cap / tile_rows + E;
  if (overlap && status && blockIdx.x == 0 && tid == 0) atomicOr(status, (int)MOE_FLAG_GUARD);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e < E) map.first[e] = base;
    base = min(base + n[i], kMostTiles);
  }
  if (tid == 0) map.first[E] = overlap ? 0 : total;
  __syncthreads();
}

struct ProductArgs {
  const uint8_t* x;         // e4m3 rows
  int64_t xs;               // their stride in bytes
  int64_t cap;
  const float* x_scales;    // [cap, K / 128]
  const uint8_t* w;         // [E, N, K]
  const float* w_scales;    // [E, ceil(N / 128), K / 128]
  const int32_t* counts;    // [E] or null: one group of all cap rows
  const int32_t* send;      // [E + 1]
  int32_t E, K, N;          // N: weight rows of one expert
  int32_t cols;             // output channels: N, or N / 2 gated
  void* out;                // bf16 rows, or e4m3 codes (gated)
  int64_t out_stride;       // in elements
  float* out_scales;        // [cap, cols / 128] (gated)
  int32_t* status;
};

// ---- pieces of a tile ----------------------------------------------------------
// A tile's operands lie in shared memory as rows of 128 codes (one scale
// block).  The 16-byte chunks of a row are permuted by a key of the row, so
// that the 16 rows a read takes together (of neighbouring lanes) fall on all
// 64 banks once: two rows share the banks of a key.
__device__ __forceinline__ int x_key(int row) { return (row >> 1) & 7; }

// The matrix instructions' square: 16 x 16 sums of 128 e4m3 products, or
// 32 x 32 of fp16 ones (of which the 16-wide form runs at 70 % of the rate).
// A lane's place in it: one row (of either operand), and one of kGroups
// shares of a block's chunks, chunk i * kGroups + group being its i-th (both
// operands split a block alike, and the order inside a sum is free).  Of the
// sums it holds, of ONE token row, the channels (q * kGroups + group) * 4 +
// 0..3.
template <bool WIDE>
struct Unit {
  static constexpr int kSide = WIDE ? 32 : 16;
  static constexpr int kGroups = kWave / kSide;
  static constexpr int kChunks = 8 / kGroups;
  static constexpr int kQuads = kSide / (4 * kGroups);
  using Sums = std::conditional_t<WIDE, f32x16, f32x4>;
};

template <bool WIDE>
struct Codes {
  u32x4 c[Unit<WIDE>::kChunks];
};

template <bool WIDE>
__device__ __forceinline__ void read_chunk(Codes<WIDE>& f, int i, const uint8_t* tile, int row,
                                           int key, int group) {
  f.c[i] = *reinterpret_cast<const u32x4*>(
      tile + row * kScaleBlock + (((i * Unit<WIDE>::kGroups + group) ^ key) << 4));
}

template <bool WIDE>
__device__ __forceinline__ void read_codes(Codes<WIDE>& f, const uint8_t* tile, int row, int key,
                                           int group) {
#pragma unroll
  for (int i = 0; i < Unit<WIDE>::kChunks; ++i) read_chunk(f, i, tile, row, key, group);
}

// The codes as fp16 (exact): the fp16 instruction adds their products with 24
// bits throughout, for sums in full fp32.
struct Halves {
  f16x8 h[8];
};

__device__ __forceinline__ f16x8 widen8(const Codes<true>& f, int i) {
  const int lo = (int)f.c[i / 2][i % 2 * 2], hi = (int)f.c[i / 2][i % 2 * 2 + 1];
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ Halves widen(const Codes<true>& f) {
  Halves w;
#pragma unroll
  for (int i = 0; i < 8; ++i) w.h[i] = widen8(f, i);
  return w;
}

__device__ __forceinline__ i32x8 as_operand(const Codes<false>& f) {
  return i32x8{(int)f.c[0][0], (int)f.c[0][1], (int)f.c[0][2], (int)f.c[0][3],
               (int)f.c[1][0], (int)f.c[1][1], (int)f.c[1][2], (int)f.c[1][3]};
}

// The sum of a block's products from the e4m3 matrix instruction.  It adds
// groups of 8 products aligned to the largest of them, of which it keeps 13
// bits below the leading one; groups and blocks add up in fp32.
__device__ __forceinline__ f32x4 block_product(const i32x8& w, const i32x8& x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{}, 0, 0, 0, 0, 0, 0);
}

// sum += f * part, element by element.
template <class Sums>
__device__ __forceinline__ void fold(Sums& sum, const Sums& part, float f) {
  constexpr int n = sizeof(Sums) / sizeof(float);
#pragma unroll
  for (int i = 0; i < n; ++i) sum[i] = __builtin_fmaf(f, part[i], sum[i]);
}

// Two fp32 values rounded to bf16, nearest even.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// g / (1 + e^-g) * u.
__device__ __forceinline__ float gated(float g, float u) {
  const float e = __builtin_amdgcn_exp2f(g * -1.44269504088896341f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// Four e4m3 codes of h / s (s = amax / 448).  A zero scale gives zero codes;
// a block with an infinity or a NaN (its scale says so) gives NaN codes.
__device__ __forceinline__ uint32_t codes4(float h0, float h1, float h2, float h3, float s) {
  if (s == 0.0f) return 0u;
  if (!(s < __builtin_inff())) return 0x7F7F7F7Fu;
  const float q0 = __builtin_amdgcn_fmed3f(h0 / s, 448.0f, -448.0f);
  const float q1 = __builtin_amdgcn_fmed3f(h1 / s, 448.0f, -448.0f);
  const float q2 = __builtin_amdgcn_fmed3f(h2 / s, 448.0f, -448.0f);
  const float q3 = __builtin_amdgcn_fmed3f(h3 / s, 448.0f, -448.0f);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(q0, q1, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(q2, q3, w, true);
  return (uint32_t)w;
}

// f(0), f(1), .. f(N - 1), each with its number as a type.
template <int N, int I = 0, class F>
__device__ __forceinline__ void static_for(const F& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ---- asynchronous loads into shared memory ---------------------------------------
// 64 lanes' 16 (or 4) bytes go to 64 consecutive places of shared memory,
// each lane from its own address.  The loads have no destination registers;
// wait_and_meet counts them.  (As builtins the compiler would wait for the
// newest of them before every read of shared memory.)  M0 is the loads' own:
// nothing else in these kernels uses it.
// They are ordered among themselves and with the waits, not with reads of
// shared memory: a block's place is not read between the two.  The compiler
// does not look inside: the five wait states that a scalar address needs
// after a vector instruction (a readfirstlane) has written it are here.
__device__ __forceinline__ void load_lds16(uint32_t lds_base, uint32_t offset, const void* base) {
  __asm__ volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 4\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(uniform((int)lds_base)), "v"(offset), "s"(base));
}

__device__ __forceinline__ void load_lds4(uint32_t lds_base, const void* addr) {
  __asm__ volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 4\n\t"
      "global_load_lds_dword %1, off"
      :
      : "s"(uniform((int)lds_base)), "v"(addr));
}

// Waits until at most LEFT of this wave's memory operations are in flight
// and its reads of shared memory are done, then for the whole workgroup.
template <int LEFT>
__device__ __forceinline__ void wait_and_meet() {
  __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(LEFT) : "memory");
}

// The workgroup meets; only shared memory is waited for.
__device__ __forceinline__ void meet() {
  __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = (uint32_t)uniform((int)(uint32_t)v);
  const int hi = uniform((int)(v >> 32));
  return ((int64_t)hi << 32) | lo;
}

__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
  return reinterpret_cast<const uint8_t*>(uniform64(reinterpret_cast<int64_t>(p)));
}

// ---- the kernel -------------------------------------------------------------------
constexpr int kScaleSteps = 4;  // blocks whose scales are loaded together
constexpr int kRowGroup = 8;    // row tiles that walk the columns together

// Workgroups of WR x WC waves; each wave holds RT x CT squares of token rows x
// weight rows.  Gated, half of a wave's weight rows are gate rows and half
// the up rows of the same channels.  STAGES blocks have a place in shared
// memory: the one that is multiplied and those whose loads are under way.
template <bool GATED_, int RT_, int CT_, int WR_, int WC_, int STAGES_>
struct Shape {
  static constexpr bool kGated = GATED_;
  static constexpr int RT = RT_, CT = CT_, WR = WR_, WC = WC_, kStages = STAGES_;
  using U = Unit<kGated>;
  static constexpr int kSide = U::kSide;
  static constexpr int kWaves = WR * WC;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kRows = WR * RT * kSide;
  static constexpr int kWRows = WC * CT * kSide;
  static constexpr int kCols = kGated ? kWRows / 2 : kWRows;   // output channels
  static constexpr int kWBlocks = kWRows / kScaleBlock;        // weight scales a step
  static constexpr int kXLoads = kRows / 8 / kWaves;           // 16-byte loads a wave and step
  static constexpr int kWLoads = kWRows / 8 / kWaves;
  static constexpr int kLoads = kXLoads + kWLoads;
  static constexpr int kLoadsAfterMeeting = 2 * kLoads / CT;   // of a step; the others before
  static constexpr int kXBytes = kRows * kScaleBlock;
  static constexpr int kWBytes = kWRows * kScaleBlock;
  static constexpr int kStageBytes = kXBytes + kWBytes;
  // Scales come for kScaleSteps blocks at once: [rows][steps], then the
  // weights' [kWave / steps][steps], of which kWBlocks rows are used.
  static constexpr int kScaleFloats = kRows * kScaleSteps + kWave;
  // The weight rows of a wave are dealt to its squares so that a lane's sums
  // of one token row are neighbouring channels, 16 bytes of them at a time,
  // and the lanes' 16 bytes of one store lie next to each other: run i of a
  // lane's kRun channels is channel i / kPiece * kPiece * kGroups + group *
  // kPiece + i % kPiece of the wave's.  Row m of square c is run c * kPer +
  // m / (4 * kGroups) * 4 + m % 4 of group m / 4 % kGroups.
  static constexpr int kSquares = kGated ? CT / 2 : CT;        // along the channels
  static constexpr int kPer = kSide / U::kGroups;
  static constexpr int kRun = kSquares * kPer;
  static constexpr int kPiece = kGated ? 16 : 8;
  __device__ static __forceinline__ int channel(int c, int m) {
    const int i = c * kPer + m / (4 * U::kGroups) * 4 + m % 4;
    return i / kPiece * (kPiece * U::kGroups) + m / 4 % U::kGroups * kPiece + i % kPiece;
  }
  // The rows read together differ in m's low four bits.
  __device__ static __forceinline__ int w_key(int row) {
    return kGated ? (row >> 1 & 3) | (row >> 4 & 1) << 2 : (row >> 1 & 1) | (row >> 3 & 3) << 1;
  }
  static_assert(kRun % kPiece == 0, "whole stores");
  // 16-byte stores of a wave and tile.
  static constexpr int kStores = RT * kRun / kPiece;
  static constexpr int kStoredWaits = kStages - 1 - (kLoadsAfterMeeting < kLoads ? 1 : 0);
  static_assert(CT >= 2 && CT % 2 == 0 && (!kGated || RT == 1), "the order of a step");
  static_assert((kStages - 1) * kLoads + kStores < 64, "the wait counts to 63");
};

template <class S>
struct Shared {
  alignas(1024) uint8_t ring[S::kStages * S::kStageBytes];
  float scales[S::kStages][S::kScaleFloats];
  TileMap<S::kThreads> map;
  uint32_t amax[S::kGated ? S::WC : 1][S::kRows];
};

// Where a tile lies.
struct TileAt {
  int64_t row0;   // its first row
  int32_t live;   // its rows
  int32_t e, ct;  // expert, column tile
};

template <class S>
__device__ __forceinline__ TileAt locate(const ProductArgs& p, const TileMap<S::kThreads>& map,
                                         uint32_t tile, uint32_t col_tiles) {
  const int t = (int)(tile / col_tiles);
  // The number of experts whose tiles end at or before t.
  const int lane = threadIdx.x & (kWave - 1);
  int e = 0;
  for (int i = 0; i < p.E; i += kWave) {
    const bool before = i + lane < p.E && map.first[i + lane + 1] <= t;
    const int n = __popcll(__ballot(before));
    e += n;
    if (n < kWave) break;
  }
  e = uniform(e);
  const int32_t first = uniform(map.first[e]);
  const int32_t row_tiles = uniform(map.first[e + 1]) - first;
  // Groups of row tiles, inside a group column by column.
  const uint32_t in_expert = tile - (uint32_t)first * col_tiles;
  const uint32_t group = in_expert / (kRowGroup * col_tiles);
  const uint32_t in_group = in_expert - group * (kRowGroup * col_tiles);
  const uint32_t wide = (uint32_t)min(kRowGroup, row_tiles - (int)group * kRowGroup);
  const int32_t rt = (int32_t)(group * kRowGroup + in_group % wide);
  TileAt at;
  at.e = e;
  at.ct = uniform((int)(in_group / wide));
  at.row0 = uniform(map.start[e]) + (int64_t)uniform(rt) * S::kRows;
  at.live = min(S::kRows, uniform(map.rows[e]) - uniform(rt) * S::kRows);
  return at;
}

// One workgroup's loads: the blocks of its tiles, one after the other.
template <class S>
struct Loader {
  const ProductArgs& p;
  Shared<S>& sh;
  int32_t kb, nb;
  uint32_t col_tiles;
  int lane, wave;
  uint32_t tile;       // the tile the next block with b == 0 begins
  int32_t left;        // blocks not sent for yet
  int32_t b = 0;
  int scale_at = 0;
  uint32_t ring_at;    // the wave's place in a stage
  TileAt at = {};
  uint32_t x_off[S::kXLoads], w_off[S::kWLoads];
  const uint8_t *x_at = nullptr, *w_at = nullptr;

  __device__ __forceinline__ void begin_tile() {
    at = locate<S>(p, sh.map, tile, col_tiles);
    tile += gridDim.x;
#pragma unroll
    for (int i = 0; i < S::kXLoads; ++i) {
      const int row = (wave * S::kXLoads + i) * 8 + (lane >> 3);
      x_off[i] = (uint32_t)min(row, at.live - 1) * (uint32_t)p.xs +
                 ((uint32_t)((lane & 7) ^ x_key(row)) << 4);
    }
    // A wave's weight loads lie in one half of the tile (gate or up rows).
    const int w_row0 = wave * S::kWLoads * 8;
    const bool up = S::kGated && w_row0 >= S::kCols;
    const int32_t col0 = at.ct * S::kCols;
#pragma unroll
    for (int i = 0; i < S::kWLoads; ++i) {
      const int row = w_row0 + i * 8 + (lane >> 3);
      const int in_half = up ? row - S::kCols : row;
      w_off[i] = (uint32_t)min(in_half, p.cols - 1 - col0) * (uint32_t)p.K +
                 ((uint32_t)((lane & 7) ^ S::w_key(in_half)) << 4);
    }
    x_at = uniform_ptr(p.x + at.row0 * p.xs);
    w_at = uniform_ptr(p.w + ((int64_t)at.e * p.N + col0 + (up ? p.cols : 0)) * p.K);
  }

  // The next kScaleSteps blocks' scales (4 lanes a row; past the last block
  // or row, the last one's again).
  __device__ __forceinline__ void issue_scales() {
    const uint32_t to = (uint32_t)(uintptr_t)sh.scales[scale_at];
    const int32_t block = min(b + (lane & (kScaleSteps - 1)), kb - 1);
    constexpr int kPer = kWave / kScaleSteps;
    for (int i = wave; i < S::kRows / kPer; i += S::kWaves) {
      const int row = i * kPer + lane / kScaleSteps;
      load_lds4(to + i * (kWave * 4),
                p.x_scales + (at.row0 + min(row, at.live - 1)) * kb + block);
    }
    if (wave == S::kWaves - 1) {
      const int i = lane / kScaleSteps;
      const int32_t w_block = S::kGated ? at.ct + (i > 0 ? p.cols / kScaleBlock : 0)
                                        : at.ct * S::kWBlocks + i;
      load_lds4(to + S::kRows * kScaleSteps * 4,
                p.w_scales + ((int64_t)at.e * nb + min(w_block, nb - 1)) * kb + block);
    }
    scale_at = scale_at + 1 == S::kStages ? 0 : scale_at + 1;
  }

  // Turns to the next block, whose scales' loads go off first.  Past the last
  // block it stays there: its loads are sent again, into a place that nobody
  // reads, so that every step has as many loads to count.
  __device__ __forceinline__ void next_block() {
    if (left == 0) return;
    --left;
    if (b == 0) {
      begin_tile();
    } else {
      x_at += kScaleBlock;
      w_at += kScaleBlock;
    }
    if (b % kScaleSteps == 0) issue_scales();
    b = b + 1 == kb ? 0 : b + 1;
  }

  // Load i of kLoads of the block, into a stage of the ring.
  __device__ __forceinline__ void issue(int stage, int i, const uint8_t* x_from,
                                        const uint8_t* w_from) const {
    const uint32_t to = ring_at + stage * S::kStageBytes;
    if (i < S::kXLoads)
      load_lds16(to + (wave * S::kXLoads + i) * 1024, x_off[i], x_from);
    else
      load_lds16(to + S::kXBytes + (wave * S::kWLoads + i - S::kXLoads) * 1024,
                 w_off[i - S::kXLoads], w_from);
  }

  // The first n loads of the next block.
  __device__ __forceinline__ void issue_block(int stage, int n) {
    next_block();
    const uint8_t *x_from = uniform_ptr(x_at), *w_from = uniform_ptr(w_at);
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i)
      if (i < n) issue(stage, i, x_from, w_from);
  }
};

template <class S>
__global__ __launch_bounds__(S::kThreads) void product_kernel(const ProductArgs p) {
  constexpr bool kGated = S::kGated;
  constexpr int RT = S::RT, CT = S::CT, kStages = S::kStages, kSide = S::kSide;
  using U = typename S::U;
  __shared__ Shared<S> sh;

  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uniform(tid / kWave);
  const int lrow = lane % kSide, group = lane / kSide;
  const int wr = wave / S::WC, wc = wave % S::WC;
  const int32_t kb = p.K / kScaleBlock, nb = (p.N + kScaleBlock - 1) / kScaleBlock;
  const uint32_t col_tiles = (uint32_t)(p.cols + S::kCols - 1) / S::kCols;
  build_tile_map<S::kThreads>(sh.map, p.counts, p.send, p.E, p.cap, S::kRows, p.status);
  const uint32_t tiles = (uint32_t)uniform(sh.map.first[p.E]) * col_tiles;

  // Workgroups i, i + 8, ... share an XCD's L2: give each XCD neighbouring tiles.
  const uint32_t first_tile = gridDim.x % 8 == 0
                                  ? (blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8
                                  : blockIdx.x;
  if (first_tile >= tiles) return;
  const uint32_t my_tiles = (tiles - 1 - first_tile) / gridDim.x + 1;
  Loader<S> loads{p, sh, kb, nb, col_tiles, lane, wave, first_tile, (int32_t)my_tiles * kb};
  loads.ring_at = (uint32_t)(uintptr_t)sh.ring;

  // Where a wave's squares lie in the tile: token rows of square r, weight
  // rows of square c (gated: gate rows, then up rows).
  constexpr int CH = kGated ? CT / 2 : CT;
  const auto x_row = [&](int r) MOE_INLINE { return (wr * RT + r) * kSide + lrow; };
  const auto w_row = [&](int c) MOE_INLINE {
    return (c >= CH ? S::kCols : 0) + wc * CH * kSide + S::channel(c % CH, lrow);
  };
  const int x_k = x_key(lrow), w_k = S::w_key(S::channel(0, lrow));
  typename U::Sums acc[CT][RT];

  const auto clear = [&]() MOE_INLINE {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[c][r] = typename U::Sums{};
  };
  int stored = 0;  // waits to come that a tile's stores may outlast
  // The block that is read: its place in the ring, its number in its tile,
  // the place of its scales.
  int stage = 0, scale_at = 0;
  int32_t read_b = 0;
  const auto next_stage = [&]() MOE_INLINE {
    stage = stage + 1 == kStages ? 0 : stage + 1;
    ++read_b;
    if (read_b % kScaleSteps == 0 || read_b == kb)
      scale_at = scale_at + 1 == kStages ? 0 : scale_at + 1;
    if (read_b == kb) read_b = 0;
  };
  const auto read_x = [&](Codes<kGated>& f, int r) MOE_INLINE {
    read_codes(f, sh.ring + stage * S::kStageBytes, x_row(r), x_k, group);
  };
  const auto read_w = [&](Codes<kGated>& f, int c) MOE_INLINE {
    read_codes(f, sh.ring + stage * S::kStageBytes + S::kXBytes, w_row(c), w_k, group);
  };
  struct Scales {
    float x[RT], w[kGated ? 2 : 1];
  };
  const auto read_scales = [&](Scales& f) MOE_INLINE {
    const float* scales = sh.scales[scale_at] + read_b % kScaleSteps;
#pragma unroll
    for (int r = 0; r < RT; ++r) f.x[r] = scales[x_row(r) * kScaleSteps];
    f.w[0] = scales[(S::kRows + (kGated ? 0 : wc * CT * kSide / kScaleBlock)) * kScaleSteps];
    if constexpr (kGated) f.w[1] = scales[(S::kRows + 1) * kScaleSteps];
  };

  // One step multiplies one block, square column by square column.  A column's
  // weights are read (and widened) one or two columns before, the token rows
  // and the first weights of the block after it in the last two columns, so
  // the matrix unit never waits for shared memory.  In the middle, when this
  // block has been read to its end, the workgroup meets once: the next
  // block's loads have to be there, and this one's place is free for those
  // of the block kStages further on, which go off one at a time until the
  // next meeting (sent together, by all waves, they queue for 800 cycles).
  // What does not need the matrix unit is dealt out between its instructions
  // in the order written.
  Codes<kGated> wq[kGated ? 1 : 2], xq[2][RT];
  Halves wo[kGated ? 2 : 1], xo[kGated ? RT : 1];
  Scales scale[2];
  const uint8_t *x_from = nullptr, *w_from = nullptr;   // the loads being sent
  int to_stage = 0;
  const auto step = [&](auto parity) MOE_INLINE {
    constexpr int P = decltype(parity)::value;
    constexpr int kMeet = (CT - 2) * RT, n = RT * CT;   // squares
    const auto meet_before = [&](auto at) MOE_INLINE {
      if constexpr (decltype(at)::value == kMeet) {
        // In flight stay the loads of the blocks after the next one and, after
        // a whole tile's stores, those, as long as every load waited for is
        // older than they are.
        if (stored > 0) {
          --stored;
          wait_and_meet<(kStages - 2) * S::kLoads + S::kStores>();
        } else {
          wait_and_meet<(kStages - 2) * S::kLoads>();
        }
        to_stage = stage;
        next_stage();
        loads.next_block();
        x_from = uniform_ptr(loads.x_at);
        w_from = uniform_ptr(loads.w_at);
      }
    };
    // The share of the loads that goes with part `at` of `parts`.
    const auto issue_with = [&](auto at, auto parts) MOE_INLINE {
      constexpr int i = decltype(at)::value, m = decltype(parts)::value;
      constexpr int l0 = i * S::kLoads / m, l1 = (i + 1) * S::kLoads / m;
      static_for<l1 - l0>([&](auto l) MOE_INLINE {
        loads.issue(to_stage, l0 + decltype(l)::value, x_from, w_from);
      });
    };
    if constexpr (!kGated) {
      // A sum is folded in three instructions after its own, when it is done.
      f32x4 part[4];
      static_for<n + 3>([&](auto at) MOE_INLINE {
        constexpr int i = decltype(at)::value, c = i / RT, r = i % RT;
        meet_before(at);
        if constexpr (i < n) {
          part[i % 4] = block_product(as_operand(wq[c % 2]), as_operand(xq[P][r]));
          issue_with(std::integral_constant<int, (i + n - kMeet) % n>{},
                     std::integral_constant<int, n>{});
          if constexpr (c >= CT - 2) {
            if constexpr (c == CT - 2) read_x(xq[1 - P][r], r);
            if constexpr (i == n - 1) read_scales(scale[1 - P]);
          }
          if constexpr (r == RT - 1) read_w(wq[c % 2], c + 2 < CT ? c + 2 : c + 2 - CT);
        }
        if constexpr (i >= 3) {
          constexpr int pc = (i - 3) / RT, pr = (i - 3) % RT;
          fold(acc[pc][pr], part[(i - 3) % 4], scale[P].x[pr] * scale[P].w[0]);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    } else {
      static_assert(!kGated || RT == 1, "a wave's one row of squares");
      f32x16 part[2];
      xo[0] = widen(xq[0][0]);
      static_for<n>([&](auto at) MOE_INLINE {
        constexpr int c = decltype(at)::value;
        meet_before(at);
        part[c % 2] = f32x16{};
        static_for<8>([&](auto aj) MOE_INLINE {
          constexpr int j = decltype(aj)::value;
          part[c % 2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(wo[c % 2].h[j], xo[0].h[j],
                                                               part[c % 2], 0, 0, 0);
          // The next column's weights, and the codes of the one after it in
          // their place.
          wo[(c + 1) % 2].h[j] = widen8(wq[0], j);
          if constexpr (j % 2 == 1)
            read_chunk(wq[0], j / 2, sh.ring + stage * S::kStageBytes + S::kXBytes,
                       w_row(c + 2 < CT ? c + 2 : c + 2 - CT), w_k, group);
          issue_with(std::integral_constant<int, ((c + 2) % CT) * 8 + j>{},
                     std::integral_constant<int, CT * 8>{});
          if constexpr (c == CT - 1 && j == 0) {
            read_x(xq[0][0], 0);
            read_scales(scale[1]);
          }
          // The sum before is done two instructions on: 3, 3, 3, 3, 2, 2.
          if constexpr (c > 0 && j >= 2) {
            constexpr int e0 = j < 6 ? 3 * (j - 2) : 12 + 2 * (j - 6), e1 = e0 + (j < 6 ? 3 : 2);
            const float f = scale[0].x[0] * scale[0].w[c - 1 >= CH ? 1 : 0];
            static_for<e1 - e0>([&](auto e) MOE_INLINE {
              constexpr int k = e0 + decltype(e)::value;
              acc[c > 0 ? c - 1 : 0][0][k] =
                  __builtin_fmaf(f, part[(c + 1) % 2][k], acc[c > 0 ? c - 1 : 0][0][k]);
            });
          }
          __builtin_amdgcn_sched_barrier(0);
        });
      });
      fold(acc[CT - 1][0], part[(CT - 1) % 2], scale[0].x[0] * scale[0].w[kGated ? 1 : 0]);
      scale[0] = scale[1];
    }
  };

  // The sum of a lane's channel i (of kRun) and its token row r.
  const auto channel_of = [&](int r, int i) MOE_INLINE {
    return acc[i / S::kPer][r][i % S::kPer];
  };

  const auto store_product = [&](const TileAt& at) MOE_INLINE {
    const int32_t col0 = at.ct * S::kCols;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int row = x_row(r);
      if (row >= at.live) continue;
      uint16_t* dst = static_cast<uint16_t*>(p.out) + (at.row0 + row) * p.out_stride;
      // The lane's channels, eight at a time.
      const int32_t col = col0 + wc * CT * kSide + group * S::kPiece;
#pragma unroll
      for (int i = 0; i < S::kRun; i += S::kPiece) {
        const int32_t at_col = col + i * U::kGroups;
        if (at_col >= p.cols) continue;
        u32x4 o;
#pragma unroll
        for (int h = 0; h < 4; ++h)
          o[h] = bf16_pair(channel_of(r, i + 2 * h), channel_of(r, i + 2 * h + 1));
        *reinterpret_cast<u32x4*>(dst + at_col) = o;
      }
    }
  };
  // Gated: the activation in the gate's place, each row's largest, then the
  // codes.
  const auto store_gated = [&](const TileAt& at) MOE_INLINE {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 4 * U::kQuads; ++i) {
          acc[c][r][i] = gated(acc[c][r][i], acc[(kGated ? CH : 0) + c][r][i]);
          m = max(m, __float_as_uint(acc[c][r][i]) & 0x7FFFFFFFu);
        }
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
      if (group == 0) sh.amax[kGated ? wc : 0][x_row(r)] = m;
    }
    meet();
    const int32_t col0 = at.ct * S::kCols;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int row = x_row(r);
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < (kGated ? S::WC : 1); ++w) m = max(m, sh.amax[w][row]);
      const float s = __uint_as_float(m) / 448.0f;
      if (row >= at.live) continue;
      uint8_t* dst = static_cast<uint8_t*>(p.out) + (at.row0 + row) * p.out_stride + col0 +
                     wc * CH * kSide + group * S::kPiece;
#pragma unroll
      for (int i = 0; i < S::kRun; i += S::kPiece) {
        u32x4 o;
#pragma unroll
        for (int h = 0; h < 4; ++h)
          o[h] = codes4(channel_of(r, i + 4 * h), channel_of(r, i + 4 * h + 1),
                        channel_of(r, i + 4 * h + 2), channel_of(r, i + 4 * h + 3), s);
        *reinterpret_cast<u32x4*>(dst + i * U::kGroups) = o;
      }
      if (wc == 0 && group == 0)
        p.out_scales[(at.row0 + row) * (p.cols / kScaleBlock) + at.ct] = s;
    }
    meet();  // the maxima's place is free for the next tile
  };
  const auto end_tile = [&](uint32_t tile) MOE_INLINE {
    const TileAt at = locate<S>(p, sh.map, tile, col_tiles);
    keep_order();  // the stores stay behind the loads sent before
    if constexpr (kGated)
      store_gated(at);
    else
      store_product(at);
    // Every wave of a whole tile has sent kStores of them (or more).
    if (at.live == S::kRows && at.ct * S::kCols + S::kCols <= p.cols) stored = S::kStoredWaits;
    clear();
  };

  clear();
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) loads.issue_block(i, S::kLoads);
  loads.issue_block(kStages - 1, S::kLoadsAfterMeeting);
  to_stage = kStages - 1;
  x_from = uniform_ptr(loads.x_at);
  w_from = uniform_ptr(loads.w_at);
  wait_and_meet<(kStages - 2) * S::kLoads + S::kLoadsAfterMeeting>();
#pragma unroll
  for (int r = 0; r < RT; ++r) read_x(xq[0][r], r);
  read_w(wq[0], 0);
  if constexpr (kGated) {
    wo[0] = widen(wq[0]);
    read_w(wq[0], 1);
  } else {
    read_w(wq[1], 1);
  }
  read_scales(scale[0]);
  uint32_t tile = first_tile;
  int32_t b = 0;
  const auto more = [&]() MOE_INLINE {
    if (++b < kb) return true;
    b = 0;
    end_tile(tile);
    tile += gridDim.x;
    return tile < tiles;
  };
  for (;;) {
    step(std::integral_constant<int, 0>{});
    if (!more()) break;
    if constexpr (!kGated) {
      step(std::integral_constant<int, 1>{});
      if (!more()) break;
    }
  }
  // Nothing is on its way to shared memory when the workgroup ends.
  __asm__ volatile("s_waitcnt vmcnt(0)" : : : "memory");
}

constexpr int kComputeUnits = 256;

template <class S>
hipError_t launch_shape(const ProductArgs& p, int64_t expected_rows, hipStream_t stream) {
  const int64_t col_tiles = (p.cols + S::kCols - 1) / S::kCols;
  const int64_t row_tiles =
      expected_rows / S::kRows + (p.counts ? (expected_rows < p.E ? expected_rows : p.E) : 1);
  constexpr int kPerUnit = 160 * 1024 / sizeof(Shared<S>);
  const int64_t most = kComputeUnits * (kPerUnit < 1 ? 1 : kPerUnit);
  const int64_t want = row_tiles * col_tiles;
  const dim3 grid((uint32_t)(want < 1 ? 1 : want < most ? want : most));
  launch_kernel(product_kernel<S>, grid, S::kThreads, stream, p);
  return hipGetLastError();
}

template <bool GATED>
hipError_t launch_product(const ProductArgs& p, int64_t expected_rows, hipStream_t stream) {
  const int64_t per_expert = expected_rows / p.E;
  if constexpr (GATED) {
    if (per_expert <= 32) return launch_shape<Shape<true, 1, 2, 1, 4, 4>>(p, expected_rows, stream);
    return launch_shape<Shape<true, 1, 4, 4, 2, 3>>(p, expected_rows, stream);
  } else {
    if (per_expert <= 32) return launch_shape<Shape<false, 2, 2, 1, 4, 3>>(p, expected_rows, stream);
    return launch_shape<Shape<false, 4, 4, 2, 4, 3>>(p, expected_rows, stream);
  }
}

}  // namespace

hipError_t launch_grouped_gemm(const GroupedGemm& g, hipStream_t stream) {
  ProductArgs p;
  p.x = static_cast<const uint8_t*>(g.x);
  p.xs = g.x_stride;
  p.cap = g.capacity_rows;
  p.x_scales = g.x_scales;
  p.w = static_cast<const uint8_t*>(g.w);
  p.w_scales = g.w_scales;
  p.counts = g.counts;
  p.send = g.send;
  p.E = g.num_experts;
  p.K = g.in_features;
  p.N = g.gated ? 2 * g.out_features : g.out_features;
  p.cols = g.out_features;
  p.out = g.out;
  p.out_stride = g.out_stride;
  p.out_scales = g.out_scales;
  p.status = g.status;
  return g.gated ? launch_product<true>(p, g.expected_rows, stream)
                 : launch_product<false>(p, g.expected_rows, stream);
}

}  // namespace moe
