// experts.hip -- the experts' products over the expert-contiguous rows that
// the dispatch makes, in e4m3 with block scales:
//   y[r, n] = sum_b sa[r, b] * sb[e, n/128, b] * sum_{k in block b} a[r, k] * w[e, n, k]
// for the rows r of expert e, b over the 128-channel blocks of the row, and
// the gated form
//   h[r, c] = silu(y[r, c]) * y[r, I + c],  quantised to e4m3 per 128 channels.
//
// A block's partial sum starts from zero in the matrix unit, and one fused
// multiply-add per element folds it, with its two scales, into the running
// fp32 sum.  The weights are the instruction's first operand: a lane then
// holds output channels of ONE row, so the row's scale is one register per
// lane, the weights' scale is the same for the whole wave, and a lane's
// output is 16 neighbouring bytes.
//
// The plain product multiplies e4m3 in the matrix unit (16 x 16 x 128, a
// block an instruction).  Its sums keep 13 bits below the largest of 8
// products, which moves 2 % of the bf16 outputs by one step and leaves their
// error against 64 bits as it is; the gated form's fp32 scales would show it
// (1.3e-5 off), so there the codes are widened, exactly, to fp16 (32 x 32 x 16;
// 1e-7) at 40 % of the rate.
//
// One workgroup a compute unit stays for the whole launch and walks tiles, so
// that a tile's first loads are under way while the one before is finished.
// Operands go from memory to a ring of stages in shared memory without
// passing registers.  Few rows an expert: the weights' bytes bound it
// (128 tokens on 256 experts, 2048 -> 7168: 573 - 587 us, 6.4 TB/s; gated 7168 ->
// 2 * 2048: 1070 - 1131 us, 6.5 - 6.9 TB/s; without the non-temporal mark 620
// and 1214 - 1267).
// Many: the matrix unit's power does, which lowers the clock to 1.9 - 2.1 GHz,
// and what moving the operands adds to it (32 experts of 1024 rows, gated:
// 1.81 - 2.01 ms, 960 - 1060 TFLOP/s; with operands from the first cache 1.60 ms
// at 2.3 GHz; plain 2048 -> 7168: 505 - 542 us, 1775 - 1905 TFLOP/s).  Between the two,
// 128 rows an expert on average, 0.94 - 1.0 ms is what 0.86 ms of loads and 0.74 ms
// of products take together.
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
// whose segments overlap cannot wrap them; such counts give no tiles at all,
// since two workgroups would write the same rows.
constexpr int kMostTiles = 1 << 30;

template <int THREADS>
struct TileMap {
  static constexpr int kWaves = THREADS / kWave;
  int first[kMaxExperts + 1];
  int start[kMaxExperts];
  int rows[kMaxExperts];
  int wave_sum[kWaves];
  int wave_end[kWaves];
  int wave_says[kWaves];
};

// Whether any thread of the workgroup says so.  Two calls need a barrier
// between them.
template <int THREADS>
__device__ __forceinline__ bool anyone(TileMap<THREADS>& map, bool says) {
  const bool wave_says = __ballot(says) != 0;
  if ((threadIdx.x & (kWave - 1)) == 0) map.wave_says[threadIdx.x / kWave] = wave_says;
  __syncthreads();
  int any = 0;
#pragma unroll
  for (int w = 0; w < THREADS / kWave; ++w) any |= map.wave_says[w];
  return any != 0;
}

template <int THREADS>
__device__ __forceinline__ void build_tile_map(TileMap<THREADS>& map,
                                               const int32_t* __restrict__ counts,
                                               const int32_t* __restrict__ send, int32_t E,
                                               int64_t cap, int tile_rows, int32_t* status) {
  constexpr int kPer = (kMaxExperts + THREADS - 1) / THREADS;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  int start[kPer], rows[kPer], n[kPer], sum = 0, end = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    start[i] = rows[i] = n[i] = 0;
    if (e < E) {
      bool cut;
      segment_of(counts, send, cap, e, start[i], rows[i], cut);
      map.start[e] = start[i];
      map.rows[e] = rows[i];
      n[i] = (rows[i] + tile_rows - 1) / tile_rows;
      if (cut && status && blockIdx.x == 0) atomicOr(status, (int)MOE_FLAG_GUARD);
    }
    sum = min(sum + n[i], kMostTiles);
    end = max(end, start[i] + rows[i]);
  }
  int incl = sum, high = end;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int up = __shfl_up(incl, d, kWave), up_end = __shfl_up(high, d, kWave);
    if (lane >= d) {
      incl = min(incl + up, kMostTiles);
      high = max(high, up_end);
    }
  }
  int before = __shfl_up(high, 1, kWave);
  if (lane == 0) before = 0;
  if (lane == kWave - 1) {
    map.wave_sum[wave] = incl;
    map.wave_end[wave] = high;
  }
  __syncthreads();
  int base = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / kWave; ++w) {
    if (w < wave) {
      base = min(base + map.wave_sum[w], kMostTiles);
      before = max(before, map.wave_end[w]);
    }
    total = min(total + map.wave_sum[w], kMostTiles);
  }
  // Segments that each start behind all earlier ones, as a layout's do, are
  // disjoint.
  bool early = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e < E) map.first[e] = base;
    base = min(base + n[i], kMostTiles);
    early |= rows[i] > 0 && start[i] < before;
    before = max(before, start[i] + rows[i]);
  }
  if (tid == 0) map.first[E] = total;
  if (!anyone(map, early)) return;
  // Others are compared, each with each.
  bool overlap = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    for (int f = 0; f < E; ++f)
      overlap |= rows[i] > 0 && map.rows[f] > 0 && f != tid * kPer + i &&
                 start[i] < map.start[f] + map.rows[f] && map.start[f] < start[i] + rows[i];
  __syncthreads();
  if (!anyone(map, overlap)) return;
  if (tid == 0) {
    map.first[E] = 0;
    if (status && blockIdx.x == 0) atomicOr(status, (int)MOE_FLAG_GUARD);
  }
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
__device__ __forceinline__ void read_codes(Codes<WIDE>& f, const uint8_t* tile, int row, int key,
                                           int group) {
#pragma unroll
  for (int i = 0; i < Unit<WIDE>::kChunks; ++i)
    f.c[i] = *reinterpret_cast<const u32x4*>(
        tile + row * kScaleBlock + (((i * Unit<WIDE>::kGroups + group) ^ key) << 4));
}

// The codes as fp16 (exact), for sums in full fp32.
struct Halves {
  f16x8 h[8];
};

__device__ __forceinline__ f16x8 widen8(uint32_t lo, uint32_t hi) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, false);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, true);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ Halves as_operand(const Codes<true>& f) {
  Halves w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w.h[2 * i] = widen8(f.c[i][0], f.c[i][1]);
    w.h[2 * i + 1] = widen8(f.c[i][2], f.c[i][3]);
  }
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

// The same sum with 24 bits throughout: the codes widened to fp16.
__device__ __forceinline__ f32x16 block_product(const Halves& w, const Halves& x) {
  f32x16 c = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(w.h[i], x.h[i], c, 0, 0, 0);
  return c;
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

// The lane, counted again where it is asked for.  What is made of it is made
// where it is needed, once a tile or a few blocks, and neither is kept in
// registers through the products, which have none left (kept values were
// spilled, and each wait for one drained the loads under way; the gated 32- and
// 64-row tiles still spill up to 5 scalar ones, to lanes of a vector register).
__device__ __forceinline__ int lane_again() {
  int none = 0;
  __asm__ volatile("" : "+v"(none));  // new to the compiler
  return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, none));
}

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ---- asynchronous loads into shared memory ---------------------------------------
// 64 lanes' 16 (or 4) bytes go to 64 consecutive places from lds_base on,
// each lane from its own address.  The loads have no destination registers;
// wait_and_meet counts them.  (As builtins the compiler would wait for the
// newest of them before every read of shared memory.)  The compiler does not
// look inside: the five wait states that a scalar address needs after a
// vector instruction (a readfirstlane) has written it are here.  M0 is the
// loads' own: nothing else in these kernels uses it.  Reads of shared memory
// may move across a load: it writes to a stage that is read only behind the
// next wait_and_meet, which nothing passes.
// ONCE: bytes that no other workgroup will ask for, marked non-temporal.
template <bool ONCE>
__device__ __forceinline__ void load_lds16(uint32_t lds_base, uint32_t offset, const void* base) {
  if constexpr (ONCE)
    __asm__ volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 4\n\t"
        "global_load_lds_dwordx4 %1, %2 nt"
        :
        : "s"(uniform((int)lds_base)), "v"(offset), "s"(base));
  else
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
      : "s"(uniform((int)lds_base)), "v"(addr)
      : "memory");
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
// Row tiles that walk the columns together, so that an XCD's 32 workgroups
// share rows and weights in its L2 (4 and 16 measure the same, 2 costs 2 %).
constexpr int kRowGroup = 8;
constexpr int kTurnStride = 4096;
constexpr int kTurnCols = 256;  // channels whose sums begin at the same block
constexpr int kTurnBlocks = 7;  // and how much further on the next ones do

// Workgroups of WR x WC waves; each wave holds RT x CT squares of token rows x
// weight rows.  Gated, half of a wave's weight rows are gate rows and half
// the up rows of the same channels.  STAGES blocks have a place in shared
// memory: the one that is multiplied and those whose loads are under way.
// ONCE: so few rows an expert that one row tile has them all on average, and
// most weights are read once.  (An expert with more reads its own again, from
// beyond the caches that the mark passes by.)
template <bool GATED_, int RT_, int CT_, int WR_, int WC_, int STAGES_, bool ONCE_>
struct Shape {
  static constexpr bool kGated = GATED_, kOnce = ONCE_;
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
  static_assert(kTurnCols % kCols == 0, "a tile's sums begin at one block");
  static_assert(kXLoads * 8 * kWaves == kRows && kWLoads * 8 * kWaves == kWRows, "whole loads");
  static_assert(kRows % (kWave / kScaleSteps) == 0, "whole scale loads");
  static_assert(!kGated || (kCols == kScaleBlock && CT % 2 == 0), "one scale block a tile");
  static_assert(kScaleBlock % ((kGated ? CT / 2 : CT) * kSide) == 0,
                "a wave's channels share a scale");
  static_assert((kStages - 1) * kLoads < 64, "the wait counts to 63");
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
  const int lane = lane_again();
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

// One workgroup's loads: a tile and a block in it, and what they have in
// shared memory.
template <class S>
struct Loader {
  const ProductArgs& p;
  Shared<S>& sh;
  int32_t kb, nb;
  uint32_t tiles, col_tiles;
  int wave;
  uint32_t tile;
  int32_t b = 0;
  int stage = 0, scale_at = 0;
  uint32_t to = 0;
  const uint8_t *x_from = nullptr, *w_from = nullptr;
  TileAt at = {};
  uint32_t x_off[S::kXLoads], w_off[S::kWLoads];
  const uint8_t *x_at = nullptr, *w_at = nullptr;
  int32_t turn = 0;    // the block a tile begins with

  __device__ __forceinline__ bool more() const { return tile < tiles; }

  __device__ __forceinline__ void begin_tile() {
    at = locate<S>(p, sh.map, tile, col_tiles);
    const int lane = lane_again();
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
    // Weight rows a multiple of 4096 bytes apart share memory channels, and
    // tiles that run together would all ask the same few: there column tiles
    // begin at different blocks and go round (64 experts of 8 rows, 4096 ->
    // 1536 gated 169 -> 131 us, 4096 -> 4096 plain 204 -> 169; of 64 rows 191 ->
    // 158 and 249 -> 205; of 256 within 3 % either way; at other channel counts
    // it costs up to 4 %, tiles side by side no longer sharing the rows they read).
    // The start depends on the output channel alone, so the sums of a row do
    // not depend on the tile's shape or the rows with it.
    turn = p.K % kTurnStride == 0 ? col0 / kTurnCols * kTurnBlocks % kb : 0;
    x_at = p.x + at.row0 * p.xs + turn * kScaleBlock;
    w_at = p.w + ((int64_t)at.e * p.N + col0 + (up ? p.cols : 0)) * p.K + turn * kScaleBlock;
  }

  // The next kScaleSteps blocks' scales (4 lanes a row; past the last block
  // or row, the last one's again).
  __device__ __forceinline__ void issue_scales() {
    const int lane = lane_again();
    const uint32_t to = (uint32_t)(uintptr_t)sh.scales[scale_at];
    int32_t block = min(b + (lane & (kScaleSteps - 1)), kb - 1) + turn;
    if (block >= kb) block -= kb;
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

  // Turns to the next block and sends off its scales' loads.  Behind the last
  // block the last one's loads are repeated, into stages nobody reads: every
  // wave then has the same number in flight at every wait.
  __device__ __forceinline__ void next() {
    if (more()) {
      if (b == 0) {
        begin_tile();
      } else {
        const int32_t by = b + turn == kb ? kScaleBlock - p.K : kScaleBlock;
        x_at += by;
        w_at += by;
      }
      if (b % kScaleSteps == 0) issue_scales();
      if (++b == kb) {
        b = 0;
        tile += gridDim.x;
      }
    }
    to = (uint32_t)(uintptr_t)sh.ring + stage * S::kStageBytes;
    x_from = uniform_ptr(x_at);
    w_from = uniform_ptr(w_at);
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
  }

  // Sends off load i of that block's S::kLoads.
  __device__ __forceinline__ void load(int i) const {
    if (i < S::kXLoads)
      load_lds16<false>(to + (wave * S::kXLoads + i) * 1024, x_off[i], x_from);
    else
      load_lds16<S::kOnce>(to + S::kXBytes + (wave * S::kWLoads + i - S::kXLoads) * 1024,
                           w_off[i - S::kXLoads], w_from);
  }
};

// A block's operands in registers, with their scales.
template <class S>
struct Block {
  Codes<S::kGated> x[S::RT], w[S::CT];
  float sx[S::RT], sw[S::kGated ? 2 : 1];
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
  Loader<S> loads{p, sh, kb, nb, tiles, col_tiles, wave, first_tile};

  // Where a wave's squares lie in the tile: token rows of square r, weight
  // rows of square c (gated: gate rows, then up rows).
  constexpr int CH = kGated ? CT / 2 : CT;
  const auto x_row = [&](int r) { return (wr * RT + r) * kSide + lrow; };
  const auto w_row = [&](int c) {
    return (c >= CH ? S::kCols : 0) + wc * CH * kSide + S::channel(c % CH, lrow);
  };
  const int x_k = x_key(lrow), w_k = S::w_key(S::channel(0, lrow));
  int stage = 0, scale_at = 0;
  int32_t read_b = 0;
  typename U::Sums acc[CT][RT];

  const auto clear = [&]() {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[c][r] = typename U::Sums{};
  };
  const auto x_stage = [&]() { return sh.ring + stage * S::kStageBytes; };
  const auto w_stage = [&]() { return sh.ring + stage * S::kStageBytes + S::kXBytes; };
  const auto read_scales = [&](Block<S>& blk) {
    const float* scales = sh.scales[scale_at] + read_b % kScaleSteps;
#pragma unroll
    for (int r = 0; r < RT; ++r) blk.sx[r] = scales[x_row(r) * kScaleSteps];
    blk.sw[0] = scales[(S::kRows + (kGated ? 0 : wc * CT * kSide / kScaleBlock)) * kScaleSteps];
    if constexpr (kGated) blk.sw[1] = scales[(S::kRows + 1) * kScaleSteps];
  };
  const auto block_read = [&]() {
    stage = stage + 1 == kStages ? 0 : stage + 1;
    ++read_b;
    if (read_b % kScaleSteps == 0 || read_b == kb)
      scale_at = scale_at + 1 == S::kStages ? 0 : scale_at + 1;
    if (read_b == kb) read_b = 0;
  };
  // Reads a block's operands and multiplies them.  Turning to the next loads
  // (some 400 cycles) hides behind the first reads as far as registers allow:
  // plain behind the operands', gated behind the scales' (odd batch 57 us
  // behind the operands', 54 so), gated with four squares a wave before them
  // (32 experts of 1024 rows 1888, 1874 and 1844).  The loads go in between the products: each takes
  // the address unit 16 cycles, and a wave that sends all of its own at once
  // waits there for everyone's.
  const auto multiply = [&]() {
    const uint8_t *xs = x_stage(), *ws = w_stage();
    Block<S> blk;
    if constexpr (kGated && RT > 1) loads.next();
    read_scales(blk);
    if constexpr (kGated && RT == 1) loads.next();
    decltype(as_operand(blk.x[0])) xo[RT];
    read_codes(blk.w[0], ws, w_row(0), w_k, group);
#pragma unroll
    for (int r = 0; r < RT; ++r) read_codes(blk.x[r], xs, x_row(r), x_k, group);
    if constexpr (!kGated) loads.next();
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (c > 0) read_codes(blk.w[c], ws, w_row(c), w_k, group);
      const auto wo = as_operand(blk.w[c]);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (c == 0) xo[r] = as_operand(blk.x[r]);
        fold(acc[c][r], block_product(wo, xo[r]), blk.sx[r] * blk.sw[c >= CH ? 1 : 0]);
        // With two stages the block is awaited next: its loads go in the
        // first half (shared expert's product 74 -> 70 us; with three stages
        // that costs 2 %).
        constexpr int kAmong = kStages == 2 ? RT * CT / 2 : RT * CT;
        const int sq = c * RT + r;
#pragma unroll
        for (int i = sq * S::kLoads / kAmong;
             i < (sq + 1) * S::kLoads / kAmong && i < S::kLoads; ++i)
          loads.load(i);
      }
    }
    block_read();
  };

  // The sum of a lane's channel i (of kRun) and its token row r.
  const auto channel_of = [&](int r, int i) {
    return acc[i / S::kPer][r][i % S::kPer];
  };

  const auto store_product = [&](const TileAt& at) {
    const int lane_ = lane_again(), lrow = lane_ % kSide, group = lane_ / kSide;
    const int32_t col0 = at.ct * S::kCols;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int row = (wr * RT + r) * kSide + lrow;
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
  const auto store_gated = [&](const TileAt& at) {
    const int lane_ = lane_again(), lrow = lane_ % kSide, group = lane_ / kSide;
    const auto x_row = [&](int r) { return (wr * RT + r) * kSide + lrow; };
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
  const auto end_tile = [&](const TileAt& at) {
    if constexpr (kGated)
      store_gated(at);
    else
      store_product(at);
    clear();
  };

  clear();
  // With fewer blocks than stages to come all of them are waited for here,
  // and none is repeated yet (16 tokens of 128 channels 7.7 -> 7.2 us).
  int ahead = 0;
#pragma unroll 1
  for (; ahead < kStages - 1 && loads.more(); ++ahead) {
    loads.next();
#pragma unroll
    for (int l = 0; l < S::kLoads; ++l) loads.load(l);
  }
  if (ahead < kStages - 1) wait_and_meet<0>();
  for (uint32_t tile = first_tile; tile < tiles; tile += gridDim.x) {
    const TileAt at = locate<S>(p, sh.map, tile, col_tiles);
    // Gated, where tiles are often half empty, waves without rows only load:
    // 256 experts of 20 to 32 rows, 7168 -> 2048, 8 to 14 % quicker (32 each:
    // 1288 -> 1118 us), of 40 to 48 equal ones within 1 % and skewed ones 5 to
    // 8 %; 64 experts, 4096 -> 1536, of 24 3 %, of 40 to 48 1 to 2 % slower.
    // The plain product measures the same either way.
    const bool any = !(kGated && S::kOnce && S::WR > 1) || wr * RT * kSide < at.live;
    for (int32_t b = 0; b < kb; ++b) {
      // This block's loads are done, everyone's (scale loads between them
      // only make the wait stricter), and the block before it is read: its
      // place takes the next loads.
      wait_and_meet<(kStages - 2) * S::kLoads>();
      if (any) {
        multiply();
      } else {
        loads.next();
#pragma unroll
        for (int l = 0; l < S::kLoads; ++l) loads.load(l);
        block_read();
      }
    }
    end_tile(at);
  }
  wait_and_meet<0>();  // shared memory is given back with no load under way
}

constexpr int kComputeUnits = 256;

// Tiles to expect when each expert's last one is half full on average.
template <class S>
int64_t tiles_to_expect(const ProductArgs& p, int64_t expected_rows) {
  const int64_t experts = p.counts ? (expected_rows < p.E ? expected_rows : p.E) : 1;
  const int64_t row_tiles = (expected_rows + experts * (S::kRows / 2)) / S::kRows;
  return row_tiles * ((p.cols + S::kCols - 1) / S::kCols);
}

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

// Rows to expect of an expert choose the tile: few rows leave the weights'
// bytes to count, many the squares.  Times in us of 64 experts by rows an
// expert on average and tile, for equal counts and (below) for counts that
// fall with the expert's rank to the power -0.6:
//   gated, 4096 -> 1536     8   16   24   32   44   64   96  128  187  256
//          32 rows, once  126  127  128  130  203  203  291  374  537  705
//                         145  141  140  165  194  252  343  441  599  786
//                32 rows  142  143  144  144  214  214  306  400  564  717
//                         160  156  150  171  196  261  367  461  629  826
//          64 rows, once  126  128  129  130  148  153  275  275  374  492
//                         128  145  153  162  175  212  275  357  467  599
//                64 rows  145  146  146  147  150  153  267  282  386  502
//                         146  176  168  166  168  207  267  336  451  563
//               128 rows  206  202  200  200  208  210  212  220  405  415
//                         204  190  223  230  243  257  270  316  399  506
//   plain, 1536 -> 4096     8   16   24   32   44   64   96  128  187  256
//          32 rows, once   65   68   72   75  130  110  171  191  302  393
//                          68   75   90   91  119  150  192  236  338  451
//                32 rows   77   78   78   79   97  103  127  163  218  294
//                          77   82   86   88   98  110  140  169  230  297
//          64 rows, once   67   70   72   75   78   82  135  113  162  193
//                          67   74   78   83   86   98  127  163  188  227
//                64 rows   76   78   77   79   84   89  106  113  154  196
//                          76   80   82   85   87   96  109  132  167  209
//               128 rows   77   78   78   81   86   90   97  102  131  145
//                          77   77   86   88   93   95  100  113  134  165
// The mean alone decides: a batch's skew is not known on the host.  At 96 equal
// rows the gated 128-row tile would be the quicker, at 96 skewed ones the same.
// Where the small tiles all run at once they are the quickest whatever the rows
// (4 experts of 225 rows, gated 2048 -> 1024: 21.6 us, 64-row tiles 24.9, 128-row
// 34.5; one of 1024, plain 2048 -> 2048: 15.1, 16.6 and 21.3), then those of 64.
template <class Use>
auto with_gated_shape(const ProductArgs& p, int64_t expected_rows, Use use) {
  using Large = Shape<true, 2, 2, 2, 4, 3, false>;
  using Middle = Shape<true, 1, 2, 2, 4, 3, false>;
  using MiddleOnce = Shape<true, 1, 2, 2, 4, 3, true>;
  using Small = Shape<true, 1, 2, 1, 4, 4, false>;
  using SmallOnce = Shape<true, 1, 2, 1, 4, 4, true>;
  const int64_t rows = expected_rows / p.E;
  if (rows <= 20) return use(SmallOnce{});
  if (tiles_to_expect<Small>(p, expected_rows) <= kComputeUnits) return use(Small{});
  if (rows <= 44) return use(MiddleOnce{});
  if (rows <= 96 || tiles_to_expect<Middle>(p, expected_rows) <= kComputeUnits)
    return use(Middle{});
  return use(Large{});
}

template <class Use>
auto with_plain_shape(const ProductArgs& p, int64_t expected_rows, Use use) {
  using Full = Shape<false, 4, 8, 4, 2, 2, false>;   // 256 x 256
  using Half = Shape<false, 4, 4, 2, 4, 3, false>;   // 128 x 256
  using Middle = Shape<false, 2, 4, 2, 4, 3, false>;
  using MiddleOnce = Shape<false, 2, 4, 2, 4, 3, true>;
  using Small = Shape<false, 2, 2, 1, 4, 3, false>;  // two of them a compute unit
  using SmallOnce = Shape<false, 2, 2, 1, 4, 3, true>;
  const int64_t rows = expected_rows / p.E;
  if (rows <= 16) return use(SmallOnce{});
  if (tiles_to_expect<Small>(p, expected_rows) <= 2 * kComputeUnits)
    return use(Small{});
  if (rows <= 48) return use(MiddleOnce{});
  if (tiles_to_expect<Middle>(p, expected_rows) <= kComputeUnits)
    return use(Middle{});
  // A full tile takes 1.6 times a half one's time (its operands move less)
  // but leaves more of the last round idle: whichever's rounds are shorter.
  // 2048 -> 7168, half and full: 32 experts of 1024 rows 599 and 505 us, of 256
  // 168 and 167; one of 8192 148 and 137, of 4096 84 and 70; 1408 -> 4224, one of
  // 5000 47 and 51.
  const auto rounds = [](int64_t tiles) { return (tiles + kComputeUnits - 1) / kComputeUnits; };
  if (rounds(tiles_to_expect<Full>(p, expected_rows)) * 8 <
      rounds(tiles_to_expect<Half>(p, expected_rows)) * 5)
    return use(Full{});
  return use(Half{});
}

template <class Use>
auto with_shape(const GroupedGemm& g, const ProductArgs& p, Use use) {
  return g.gated ? with_gated_shape(p, g.expected_rows, use)
                 : with_plain_shape(p, g.expected_rows, use);
}

ProductArgs args_of(const GroupedGemm& g) {
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
  return p;
}

}  // namespace

hipError_t launch_grouped_gemm(const GroupedGemm& g, hipStream_t stream) {
  const ProductArgs p = args_of(g);
  return with_shape(g, p, [&](auto shape) {
    return launch_shape<decltype(shape)>(p, g.expected_rows, stream);
  });
}

ProductTile grouped_gemm_tile(const GroupedGemm& g) {
  return with_shape(g, args_of(g), [](auto shape) {
    using S = decltype(shape);
    return ProductTile{S::kRows, S::kCols, S::kOnce};
  });
}

}  // namespace moe
