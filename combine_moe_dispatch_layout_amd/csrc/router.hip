// router.hip -- the router's product and its gradient:
//   logits[t, e] = sum_h x[t, h] * w[e, h]                   (fp32)
//   dx[t, h] = sum_e dl[t, e] * w[e, h] + add[t, h]          (rounded once to bf16)
//   dw[e, h] = sum_t dl[t, e] * x[t, h]                      (fp32)
//
// All three are products in the bf16 matrix instruction with fp32 sums.  x and
// w are bf16, so the forward's products are exact.  dl is fp32: it is split
// once into three bf16 parts that add up to it exactly (8 + 8 + 8 bits), and
// the gradients add the parts' products: two for dx, which is rounded to 8 bits
// itself, all three for dw.  What dx leaves out is at most 2^-16 of a term (the
// first part leaves less than 2^-7 of it, of which the second's rounding leaves
// 2^-9).  With the third 4 in 10000 of its values come out a step of bf16 apart, the
// error against 64 bits stays the same to four digits, and dx of 4096 tokens of 7168
// channels takes on 64, 128, 256 and 512 experts 28, 34, 89 and 99 us in place of 27,
// 31, 42 and 75.
//
// router_kernel is a product of tiles, D[j, i] = sum_p sum_k J_p[j, k] * I[i, k].  An
// operand lies in memory either by rows (k neighbouring) or by columns (i or j
// neighbouring, x and dl in dw); the latter is turned by the transposing read of
// shared memory, so nothing is transposed in memory.  It makes the logits of many
// tokens (16384 of 7168 channels on 512 experts 130 us, 925 TFLOP/s: products alone
// take 80, with the reads of shared memory 100, with the loads 114, and loads alone
// 105; other tiles, reads a step ahead, loads through registers and rows fetched
// ahead into L2 by a wave of their own measure the same or worse) and dw of many
// (4096 of 7168 on 256 51 us and 7 for the sum of its shares, 880 TFLOP/s of the
// three parts).
// The other kernels are for what that one does badly: one_token_kernel and
// shared_k_kernel for few tokens or experts, few_grad_w for their dw,
// small_grad_x_kernel for their dx (128 of 7168 on 256 7 us) and grad_x_kernel for
// dx of many, whose k is short (4096 of 7168 on 256 42 us, 45 to 49 beside the
// parts of dl: the start with dl 9, products 28, the memory of add and dx the rest).
#include "lds_loads.h"
#include "moe_internal.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));  // at any float
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kDepth = 64;      // k of a stage: rows of 128 bytes in shared memory
constexpr int kSide = 32;       // the matrix instruction's square (32 x 32 x 16)
constexpr int kSteps = kDepth / 16;
constexpr int kRowBytes = 2 * kDepth;
constexpr int kUnits = 256;     // compute units

// An operand: element (n, k) at n * stride + k by rows, at k * stride + n by
// columns.
struct Operand {
  const uint16_t* base;
  int64_t stride;   // elements
  int64_t plane;    // elements from one part to the next
  int32_t count;    // of n (a multiple of 8 by columns)
  int32_t depth;    // of k
};

struct Product {
  Operand i, j;
  int32_t tiles_i, tiles_j, splits, blocks;  // blocks: of kDepth
  int32_t jobs;
  bool i_first;      // neighbouring jobs are neighbouring tiles of i, else of j
  float* out;        // [j, i], one after the other for each split
  int64_t out_stride, split_stride;  // elements
  int32_t cols, rows;  // i's and j's that are written
  bool vectors;      // four i's at a time
};

// WI x WJ waves with RI x RJ squares each.  The 16-byte chunks of a row in
// shared memory are permuted by a key of the row: by rows, so that the 16 rows
// a read takes together fall on all 64 banks once; by columns, so that the four
// rows a transposing read takes together do.
template <bool I_COLS_, bool J_COLS_, int PARTS_, int RI_, int RJ_, int WI_, int WJ_,
          int STAGES_>
struct Shape {
  static constexpr bool kICols = I_COLS_, kJCols = J_COLS_;
  static constexpr int P = PARTS_, RI = RI_, RJ = RJ_, WI = WI_, WJ = WJ_, kStages = STAGES_;
  static constexpr int kWaves = WI * WJ;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kTileI = WI * RI * kSide, kTileJ = WJ * RJ * kSide;
  static constexpr int kILoads = kTileI / 8 / kWaves;      // a wave and stage
  static constexpr int kJLoads = P * kTileJ / 8 / kWaves;
  static constexpr int kLoads = kILoads + kJLoads;
  static constexpr int kIBytes = kTileI * kRowBytes, kJBytes = kTileJ * kRowBytes;
  static constexpr int kStageBytes = kIBytes + P * kJBytes;
  static_assert(kILoads * 8 * kWaves == kTileI && kJLoads * 8 * kWaves == P * kTileJ, "loads");
  static_assert((kStages - 2) * kLoads <= 63, "loads that one wait can leave");
  static_assert(kStages * kStageBytes <= 160 * 1024, "shared memory");
};

__device__ __forceinline__ int row_key(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int col_key(int k) { return (k >> 1 & 1) * 4; }

// The place in an operand of the 16 bytes that a lane puts into row `row` of
// the tile in shared memory.  Rows or columns past the end are given their
// last neighbours: they reach only sums that are not written.
template <bool COLS>
__device__ __forceinline__ int64_t chunk_at(const Operand& o, int32_t n0, int32_t k0, int row,
                                            int lane) {
  const int slot = lane % 8;
  if (COLS) {  // rows of k, panels of 64 n
    const int32_t n = n0 + row / kDepth * kDepth + (slot ^ col_key(row)) * 8;
    return (int64_t)(k0 + row % kDepth) * o.stride + min(n, o.count - 8);
  }
  return (int64_t)min(n0 + row, o.count - 1) * o.stride + k0 + (slot ^ row_key(row)) * 8;
}

// Whether that chunk lies behind the last k.
template <bool COLS>
__device__ __forceinline__ bool behind(const Operand& o, int32_t k0, int row, int lane) {
  const int k = COLS ? row % kDepth : (lane % 8 ^ row_key(row)) * 8;
  return k0 + k >= o.depth;
}

typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// A square's operand: the lane's 8 k (16 * step + 8 * (lane / 32) on) of row
// lane % 32 of the square that begins at row `n` of the tile.
template <bool COLS, bool SPREAD>
__device__ __forceinline__ bf16x8 read_square(const uint8_t* tile, int n, int step, int lane) {
  if (!COLS) {
    const int row = n + lane % kSide, chunk = 2 * step + lane / kSide;
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(
                                          tile + row * kRowBytes + ((chunk ^ row_key(row)) << 4)));
  }
  // 16 lanes give the addresses of a block of 4 k x 16 n, four n each, and get
  // a column of it each.  Which four n stand at places 4m .. 4m + 3 is free:
  // SPREAD takes the order that leaves a lane's sums in runs of 8 neighbours.
  const int s = lane % 16, g = lane / 16;
  const int m = 4 * (g % 2) + s % 4;  // of the square's 8 groups of four
  const int four = SPREAD ? (m >> 2) * 4 + (m & 1) * 2 + (m >> 1 & 1) : m;
  const int col = n + 4 * four;
  const int k = 16 * step + 8 * (g / 2) + s / 4;
  const int chunk = col % kDepth / 8;
  const uint8_t* at = tile + col / kDepth * (kDepth * kRowBytes) + (col & 4) * 2;
  s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_s16x4*)(at + k * kRowBytes + ((chunk ^ col_key(k)) << 4)));
  s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_s16x4*)(at + (k + 4) * kRowBytes + ((chunk ^ col_key(k + 4)) << 4)));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Workgroups b, b + 8, ... share an XCD's L2: each XCD takes a run of jobs.  The
// first job of workgroup b; where there are fewer workgroups than jobs, it goes
// on with every step-th up to `last`.
__device__ __forceinline__ int32_t first_of_xcd(int32_t jobs, int32_t xcd) {
  return xcd * (jobs / 8) + min(xcd, jobs % 8);
}
__device__ __forceinline__ int32_t own_job(int32_t jobs, int32_t b) {
  return first_of_xcd(jobs, b % 8) + b / 8;
}
__device__ __forceinline__ void own_jobs(int32_t jobs, int32_t& job, int32_t& step,
                                         int32_t& last) {
  const int32_t xcd = blockIdx.x % 8;
  job = own_job(jobs, blockIdx.x);
  step = ((int32_t)gridDim.x - xcd + 7) / 8;
  last = first_of_xcd(jobs, xcd + 1);
}

// A workgroup's walk through its jobs' blocks.
struct Walk {
  int32_t job, step, last;   // this job, and the next one's distance and the end
  int32_t i0, j0, split, block, end;
  __device__ __forceinline__ bool more() const { return job < last; }
  template <class S>
  __device__ __forceinline__ void enter(const Product& p) {
    if (!more()) return;
    const int32_t tiles = p.tiles_i * p.tiles_j, tile = job % tiles;
    split = job / tiles;
    i0 = (p.i_first ? tile % p.tiles_i : tile / p.tiles_j) * S::kTileI;
    j0 = (p.i_first ? tile / p.tiles_i : tile % p.tiles_j) * S::kTileJ;
    block = (int32_t)((int64_t)p.blocks * split / p.splits);
    end = (int32_t)((int64_t)p.blocks * (split + 1) / p.splits);
  }
  template <class S>
  __device__ __forceinline__ void next(const Product& p) {
    if (++block < end) return;
    job += step;
    enter<S>(p);
  }
};

// The addresses of a wave's loads, kept from one block of a tile to the next.
// Only a depth that does not fill its last block is looked at again there: what
// lies behind it reads as zeros (an infinity would otherwise spoil a sum).
template <class S>
struct Loads {
  const uint16_t* i[S::kILoads];
  const uint16_t* j[S::kJLoads];

  __device__ __forceinline__ static int i_row(int wave, int lane, int n) {
    return (wave * S::kILoads + n) * 8 + lane / 8;
  }
  __device__ __forceinline__ static int j_row(int wave, int lane, int n) {
    return (wave * S::kJLoads + n) % (S::kTileJ / 8) * 8 + lane / 8;
  }
  __device__ __forceinline__ void enter(const Product& p, const Walk& at, int wave, int lane) {
    const int32_t k0 = at.block * kDepth;
#pragma unroll
    for (int n = 0; n < S::kILoads; ++n)
      i[n] = p.i.base + chunk_at<S::kICols>(p.i, at.i0, k0, i_row(wave, lane, n), lane);
#pragma unroll
    for (int n = 0; n < S::kJLoads; ++n)
      j[n] = p.j.base + (wave * S::kJLoads + n) / (S::kTileJ / 8) * p.j.plane +
             chunk_at<S::kJCols>(p.j, at.j0, k0, j_row(wave, lane, n), lane);
  }
  __device__ __forceinline__ void step(const Product& p) {
    const int64_t di = S::kICols ? kDepth * p.i.stride : kDepth;
    const int64_t dj = S::kJCols ? kDepth * p.j.stride : kDepth;
#pragma unroll
    for (int n = 0; n < S::kILoads; ++n) i[n] += di;
#pragma unroll
    for (int n = 0; n < S::kJLoads; ++n) j[n] += dj;
  }
  // Sends off a block's loads and turns to the next block.
  __device__ __forceinline__ void send(const Product& p, Walk& at, uint32_t to, int wave,
                                       int lane) {
    const int32_t k0 = at.block * kDepth;
    const uint32_t i_to = to + wave * S::kILoads * 1024;
    const uint32_t j_to = to + S::kIBytes + wave * S::kJLoads * 1024;
    if (k0 + kDepth <= p.i.depth) {
#pragma unroll
      for (int n = 0; n < S::kILoads; ++n) load_lds16_from(i_to + n * 1024, i[n]);
    } else {
#pragma unroll
      for (int n = 0; n < S::kILoads; ++n)
        load_lds16_from(i_to + n * 1024, behind<S::kICols>(p.i, k0, i_row(wave, lane, n), lane)
                                             ? static_cast<const void*>(&kZeroVec)
                                             : i[n]);
    }
    if (k0 + kDepth <= p.j.depth) {
#pragma unroll
      for (int n = 0; n < S::kJLoads; ++n) load_lds16_from(j_to + n * 1024, j[n]);
    } else {
#pragma unroll
      for (int n = 0; n < S::kJLoads; ++n)
        load_lds16_from(j_to + n * 1024, behind<S::kJCols>(p.j, k0, j_row(wave, lane, n), lane)
                                             ? static_cast<const void*>(&kZeroVec)
                                             : j[n]);
    }
    const int32_t job = at.job;
    at.next<S>(p);
    if (at.job == job)
      step(p);
    else if (at.more())
      enter(p, at, wave, lane);
  }
};

template <class S>
__device__ __forceinline__ void write_tile(const Product& p, const Walk& at,
                                           const f32x16 (&sum)[S::RI][S::RJ], int wi, int wj,
                                           int lane) {
#pragma unroll
  for (int b = 0; b < S::RJ; ++b) {
    const int32_t j = at.j0 + (wj * S::RJ + b) * kSide + lane % kSide;
    if (j >= p.rows) continue;
    float* to = p.out + at.split * p.split_stride + j * p.out_stride;
#pragma unroll
    for (int a = 0; a < S::RI; ++a)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int32_t i =
            at.i0 + (wi * S::RI + a) * kSide + 8 * q + 4 * (lane / kSide);
        const f32x4 v = {sum[a][b][4 * q], sum[a][b][4 * q + 1], sum[a][b][4 * q + 2],
                         sum[a][b][4 * q + 3]};
        if (p.vectors) {
          if (i < p.cols) *reinterpret_cast<f32x4*>(to + i) = v;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (i + c < p.cols) to[i + c] = v[c];
        }
      }
  }
}

// Workgroups stay and walk jobs (a tile, and a share of k where there are few
// tiles), so that a job's first loads are under way while the one before is
// finished.
// (Asked for two waves a SIMD, the compiler keeps the sums in ordinary
// registers; else it moves them to accumulation registers and back at every
// block.)
template <class S>
__global__ __launch_bounds__(S::kThreads, 2) void router_kernel(const Product p) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[S::kStages * S::kStageBytes];
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int wi = wave % S::WI, wj = wave / S::WI;
  const uint32_t base = (uint32_t)(uintptr_t)ring;

  Walk at;
  own_jobs(p.jobs, at.job, at.step, at.last);
  at.enter<S>(p);
  Walk ahead = at;
  Loads<S> loads;
  if (ahead.more()) loads.enter(p, ahead, wave, lane);
  int stage = 0, fill = 0;
#pragma unroll
  for (int n = 0; n < S::kStages - 1; ++n) {
    if (ahead.more()) loads.send(p, ahead, base + fill * S::kStageBytes, wave, lane);
    fill = fill + 1 == S::kStages ? 0 : fill + 1;
  }
  while (at.more()) {
    f32x16 sum[S::RI][S::RJ] = {};
    for (int32_t block = at.block; block < at.end; ++block) {
      // The stage's loads are the oldest under way.  Behind the last block's
      // there are fewer than the wait would leave.
      if (ahead.more()) {
        wait_and_meet<(S::kStages - 2) * S::kLoads>();
        loads.send(p, ahead, base + fill * S::kStageBytes, wave, lane);
      } else {
        wait_and_meet<0>();
      }
      fill = fill + 1 == S::kStages ? 0 : fill + 1;
      const uint8_t* tile = ring + stage * S::kStageBytes;
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        bf16x8 i[S::RI];
#pragma unroll
        for (int a = 0; a < S::RI; ++a)
          i[a] = read_square<S::kICols, false>(tile, (wi * S::RI + a) * kSide, s, lane);
#pragma unroll
        for (int b = 0; b < S::RJ; ++b)
#pragma unroll
          for (int part = 0; part < S::P; ++part) {
            const bf16x8 j = read_square<S::kJCols, false>(
                tile + S::kIBytes + part * S::kJBytes, (wj * S::RJ + b) * kSide, s, lane);
#pragma unroll
            for (int a = 0; a < S::RI; ++a)
              sum[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(i[a], j, sum[a][b], 0, 0, 0);
          }
      }
    }
    write_tile<S>(p, at, sum, wi, wj, lane);
    at.block = at.end - 1;
    at.next<S>(p);
  }
}

// ---- logits of one token --------------------------------------------------------------
// A wave an expert: its weight is read once, and the token's row, which all
// waves share, comes from the caches.  (7168 channels, 256 experts: 5.3 us, 6.1 by
// the next kernel, which takes over at two tokens, where this way is level.)
__global__ __launch_bounds__(256) void one_token_kernel(const u32x4* __restrict__ x,
                                                        const u32x4* __restrict__ w, int32_t nvec,
                                                        int32_t experts,
                                                        float* __restrict__ logits) {
  const int lane = threadIdx.x & (kWave - 1);
  const int32_t e = blockIdx.x * 4 + threadIdx.x / kWave;
  if (e >= experts) return;
  const u32x4* we = w + (int64_t)e * nvec;
  float sum = 0.0f;
  constexpr int kUnroll = 4;
  for (int32_t v0 = lane; v0 < nvec; v0 += kWave * kUnroll) {
    u32x4 wv[kUnroll], xv[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t v = min(v0 + u * kWave, nvec - 1);
      wv[u] = we[v];
      xv[u] = x[v];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (v0 + u * kWave >= nvec) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        sum = __builtin_fmaf(bf16lo_to_f32(wv[u][c]), bf16lo_to_f32(xv[u][c]), sum);
        sum = __builtin_fmaf(bf16hi_to_f32(wv[u][c]), bf16hi_to_f32(xv[u][c]), sum);
      }
    }
  }
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d, kWave);
  if (lane == 0) logits[e] = sum;
}

// ---- logits of small batches ----------------------------------------------------------
// These have too few tiles to fill the card, and shares of k that a second launch
// joins cost as much as the product: here a workgroup's waves share the k of a
// small tile, every WAVES-th block of 64 each, in stages of their own, where no
// wave waits for another, and their sums meet in shared memory at the end.  It is
// bound by the tiles' rows coming from the caches (128 tokens of 7168 channels on
// 256 experts: 58 MB, 6.4 us, 512: 235 MB, 12.7 us, 18 TB/s).
struct SharedK {
  Operand i, j;      // w, x: by rows
  int32_t tiles_i, tiles_j, blocks, jobs;
  int32_t band;      // token tiles that neighbouring jobs take of an expert tile
  float* out;
  int64_t out_stride;
  int32_t experts, bs;
};

template <int SIDE, int WAVES, int STAGES>
__global__ __launch_bounds__(WAVES* kWave) void shared_k_kernel(const SharedK p) {
  typedef float Sum __attribute__((ext_vector_type(SIDE * SIDE / kWave)));
  constexpr int kLoads = 2 * SIDE / 8;
  constexpr int kBytes = 2 * SIDE * kRowBytes;
  constexpr int kGroups = kWave / SIDE;           // lanes of a row
  constexpr int kShareSteps = kDepth / (8 * kGroups);
  constexpr int kOut = (SIDE * SIDE + WAVES * kWave - 1) / (WAVES * kWave);
  static_assert((STAGES - 1) * kLoads <= 63, "loads that one wait can leave");
  static_assert(SIDE * SIDE * 4 <= STAGES * kBytes, "the sums take the stages' place");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[WAVES * STAGES * kBytes];
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int32_t job = own_job(p.jobs, blockIdx.x), full = p.band * p.tiles_i;
  const int32_t j_first = job / full * p.band, width = min(p.band, p.tiles_j - j_first);
  const int32_t i0 = job % full / width * SIDE;
  const int32_t j0 = (j_first + job % full % width) * SIDE;
  uint8_t* mine = lds + wave * STAGES * kBytes;

  const uint16_t* from[kLoads];
#pragma unroll
  for (int n = 0; n < kLoads; ++n) {
    const int row = n * 8 + lane / 8, chunk = lane % 8 ^ row_key(row);
    const Operand& o = n < kLoads / 2 ? p.i : p.j;
    const int32_t at = n < kLoads / 2 ? i0 + row : j0 + row - SIDE;
    from[n] = o.base + (int64_t)min(at, o.count - 1) * o.stride + chunk * 8;
  }
  const auto send = [&](int32_t block, int stage) {
    const uint32_t to = (uint32_t)(uintptr_t)mine + stage * kBytes;
    const int32_t k0 = block * kDepth;
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int chunk = lane % 8 ^ row_key(n * 8 + lane / 8);
      load_lds16_from(to + n * 1024, k0 + chunk * 8 < p.i.depth
                                         ? static_cast<const void*>(from[n] + k0)
                                         : &kZeroVec);
    }
  };
#pragma unroll
  for (int s = 0; s < STAGES; ++s)
    if (wave + s * WAVES < p.blocks) send(wave + s * WAVES, s);
  Sum sum = {};
  int stage = 0;
  for (int32_t block = wave; block < p.blocks; block += WAVES) {
    const int32_t ahead = block + STAGES * WAVES;
    if (ahead - WAVES < p.blocks)
      wait_own<(STAGES - 1) * kLoads>();
    else
      wait_own<0>();
    const uint8_t* tile = mine + stage * kBytes;
    bf16x8 i[kShareSteps], j[kShareSteps];
#pragma unroll
    for (int s = 0; s < kShareSteps; ++s) {
      const int row = lane % SIDE, chunk = s * kGroups + lane / SIDE;
      i[s] = __builtin_bit_cast(
          bf16x8, *reinterpret_cast<const u32x4*>(tile + row * kRowBytes +
                                                  ((chunk ^ row_key(row)) << 4)));
      j[s] = __builtin_bit_cast(
          bf16x8, *reinterpret_cast<const u32x4*>(tile + (SIDE + row) * kRowBytes +
                                                  ((chunk ^ row_key(SIDE + row)) << 4)));
    }
    if (ahead < p.blocks) {
      wait_reads();
      send(ahead, stage);
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
#pragma unroll
    for (int s = 0; s < kShareSteps; ++s) {
      if constexpr (SIDE == 16)
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(i[s], j[s], sum, 0, 0, 0);
      else
        sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(i[s], j[s], sum, 0, 0, 0);
    }
  }
  // [token][expert] of each wave, in its stages' place; experts permuted by the
  // token so that all banks are used.
  wait_own<0>();
  float* sums = reinterpret_cast<float*>(mine);
  const int t = lane % SIDE;
#pragma unroll
  for (int q = 0; q < SIDE * SIDE / kWave / 4; ++q) {
    const int four = (SIDE == 16 ? 0 : 2 * q) + lane / SIDE;
    *reinterpret_cast<f32x4*>(sums + t * SIDE + ((four ^ (t * SIDE / 32)) & (SIDE / 4 - 1)) * 4) =
        f32x4{sum[4 * q], sum[4 * q + 1], sum[4 * q + 2], sum[4 * q + 3]};
  }
  meet();
#pragma unroll
  for (int n = 0; n < kOut; ++n) {
    const int at = threadIdx.x + n * WAVES * kWave;
    if (at >= SIDE * SIDE) return;
    const int token = at / SIDE, expert = at % SIDE;
    const int place =
        token * SIDE + ((expert / 4 ^ (token * SIDE / 32)) & (SIDE / 4 - 1)) * 4 + expert % 4;
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
      total += reinterpret_cast<const float*>(lds + w * STAGES * kBytes)[place];
    if (j0 + token < p.bs && i0 + expert < p.experts)
      p.out[(int64_t)(j0 + token) * p.out_stride + i0 + expert] = total;
  }
}

// ---- the parts of dl -----------------------------------------------------------------
// Two values' three bf16 parts, that of the second in the upper half.  The first
// is the value cut to 8 bits (so that none rounds up to infinity), the second
// what is left rounded to 8, the third the rest, which has no more than 8.  (Of
// values below 2^-110 that rest ends below 2^-133, bf16's smallest step, and is
// rounded to it.)  An infinity is all in the first; a NaN, whose mark the cut may
// lose, is in the others too.
__device__ __forceinline__ void pair_parts(float a, float b, uint32_t& hi, uint32_t& mid,
                                           uint32_t& lo) {
  const uint32_t up = __float_as_uint(a), vp = __float_as_uint(b);
  hi = up >> 16 | (vp & 0xFFFF0000u);
  float ra = a - __uint_as_float(up & 0xFFFF0000u), rb = b - __uint_as_float(vp & 0xFFFF0000u);
  ra = __builtin_isinf(a) ? 0.0f : ra;
  rb = __builtin_isinf(b) ? 0.0f : rb;
  mid = bf16_pair(ra, rb);
  lo = bf16_pair(ra - bf16lo_to_f32(mid), rb - bf16hi_to_f32(mid));
}

struct Parts {
  const float* dl;
  int64_t dl_stride;
  int32_t bs, experts;
  int32_t rows, cols;   // padded with zeros to whole stages
  uint16_t* parts;      // [3][rows][cols]
};

// The three parts of dl.  Done by `blocks` workgroups of 256 threads.
__device__ __forceinline__ void split_parts(const Parts& p, int32_t block, int32_t blocks) {
  const int64_t all = (int64_t)p.rows * p.cols;
  for (int64_t n = ((int64_t)block * 256 + threadIdx.x) * 4; n < all; n += (int64_t)blocks * 1024) {
    const int64_t r = n / p.cols;
    const int32_t c = (int32_t)(n - r * p.cols);
    float f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      f[u] = r < p.bs && c + u < p.experts ? p.dl[r * p.dl_stride + c + u] : 0.0f;
    uint32_t v[3][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) pair_parts(f[2 * u], f[2 * u + 1], v[0][u], v[1][u], v[2][u]);
#pragma unroll
    for (int part = 0; part < 3; ++part)
      *reinterpret_cast<u32x2*>(p.parts + part * all + n) = u32x2{v[part][0], v[part][1]};
  }
}

__global__ __launch_bounds__(256) void split_kernel(const Parts p) {
  split_parts(p, blockIdx.x, gridDim.x);
}

int32_t split_blocks(const Parts& p) {
  const int64_t want = ((int64_t)p.rows * p.cols / 4 + 255) / 256;
  return (int32_t)(want < 2 * kUnits ? want : 2 * kUnits);
}

// ---- dw of a few tokens ----------------------------------------------------------------
// Made of dl as it is, which is split into its three parts in registers: no
// launch for those, and the workgroups run beside those of dx.  A workgroup has
// kFewCols channels of kFewExperts experts and a range of tokens, a wave 64
// channels of 32 experts.
constexpr int kFewCols = 128;
constexpr int kFewExperts = 64;
constexpr int kFewThreads = 256;
constexpr int kFewXBytes = kDepth * kFewCols * 2;
constexpr int kFewStage = kFewXBytes + kDepth * kFewExperts * 4;
constexpr int kFewBytes = 2 * kFewStage;

struct FewGradW {
  const float* dl;
  int64_t dl_stride;
  const uint16_t* x;
  int64_t x_stride;
  int32_t bs, hidden, experts;
  int32_t ranges;   // of tokens
  bool vectors;     // dl's rows are of whole 16 bytes and begin there
  float* dw;        // [ranges][experts][hidden]
};

// All three parts of 8 values.
__device__ __forceinline__ void three_parts(const float (&f)[8], bf16x8 (&parts)[3]) {
  u32x4 h, m, l;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t hi, mid, lo;
    pair_parts(f[2 * c], f[2 * c + 1], hi, mid, lo);
    h[c] = hi;
    m[c] = mid;
    l[c] = lo;
  }
  parts[0] = __builtin_bit_cast(bf16x8, h);
  parts[1] = __builtin_bit_cast(bf16x8, m);
  parts[2] = __builtin_bit_cast(bf16x8, l);
}

// Rows of dl in shared memory: 64 experts of a token, the two halves swapped in
// every other 8 tokens, so that the two half waves, which read 8 tokens apart,
// fall on different banks.
__device__ __forceinline__ int few_key(int t) { return t >> 3 & 1; }

__device__ __forceinline__ void few_grad_w(const FewGradW& p, int32_t block, uint8_t* lds) {
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int32_t col_tiles = (p.hidden + kFewCols - 1) / kFewCols;
  const int32_t range = block % p.ranges, tile = block / p.ranges;
  const int32_t e0 = tile / col_tiles * kFewExperts, h0 = tile % col_tiles * kFewCols;
  const int32_t stages = (p.bs + kDepth - 1) / kDepth;
  const int32_t first = (int32_t)((int64_t)stages * range / p.ranges);
  const int32_t end = (int32_t)((int64_t)stages * (range + 1) / p.ranges);

  const auto send = [&](int32_t stage) {
    const uint32_t to = (uint32_t)(uintptr_t)lds + (stage & 1) * kFewStage;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int row = (wave * 4 + n) * 8 + lane / 8, k = row % kDepth;
      const int32_t t = stage * kDepth + k;
      const int32_t h = h0 + row / kDepth * 64 + (lane % 8 ^ col_key(k)) * 8;
      load_lds16_from(to + (wave * 4 + n) * 1024,
                      t < p.bs ? static_cast<const void*>(p.x + t * p.x_stride +
                                                          min(h, p.hidden - 8))
                               : &kZeroVec);
    }
    if (p.vectors) {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int k = (wave * 4 + n) * 4 + lane / 16;
        const int32_t t = stage * kDepth + k, e = e0 + (lane % 16 ^ 8 * few_key(k)) * 4;
        load_lds16_from(to + kFewXBytes + (wave * 4 + n) * 1024,
                        t < p.bs && e < p.experts
                            ? static_cast<const void*>(p.dl + t * p.dl_stride + e)
                            : &kZeroVec);
      }
    } else {
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const int k = wave * 16 + n;
        const int32_t t = stage * kDepth + k, e = e0 + (lane ^ 32 * few_key(k));
        load_lds4(to + kFewXBytes + k * 256, t < p.bs && e < p.experts
                                                 ? static_cast<const void*>(
                                                       p.dl + t * p.dl_stride + e)
                                                 : &kZeroVec);
      }
    }
  };
  send(first);

  const int wj = wave % 2, wi = wave / 2;
  f32x16 sum[2] = {};
  for (int32_t stage = first; stage < end; ++stage) {
    wait_and_meet<0>();
    if (stage + 1 < end) send(stage + 1);
    const uint8_t* x = lds + (stage & 1) * kFewStage;
    const float* dl = reinterpret_cast<const float*>(x + kFewXBytes);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      float f[8];
      const int k = 16 * s + 8 * (lane / kSide);
      const int e = wj * kSide + lane % kSide ^ 32 * few_key(k);
#pragma unroll
      for (int u = 0; u < 8; ++u) f[u] = dl[(k + u) * kFewExperts + e];
      bf16x8 i[2], parts[3];
#pragma unroll
      for (int a = 0; a < 2; ++a)
        i[a] = read_square<true, false>(x, wi * 64 + a * kSide, s, lane);
      three_parts(f, parts);
#pragma unroll
      for (int part = 2; part >= 0; --part)
#pragma unroll
        for (int a = 0; a < 2; ++a)
          sum[a] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(i[a], parts[part], sum[a], 0, 0, 0);
    }
  }
  const int32_t e = e0 + wj * kSide + lane % kSide;
  if (e >= p.experts) return;
  float* out = p.dw + ((int64_t)range * p.experts + e) * p.hidden;
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int32_t h = h0 + wi * 64 + a * kSide + 8 * q + 4 * (lane / kSide);
      if (h < p.hidden)
        *reinterpret_cast<f32x4*>(out + h) =
            f32x4{sum[a][4 * q], sum[a][4 * q + 1], sum[a][4 * q + 2], sum[a][4 * q + 3]};
    }
}

__global__ __launch_bounds__(kFewThreads) void few_grad_w_kernel(const FewGradW p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kFewBytes];
  few_grad_w(p, blockIdx.x, lds);
}

int32_t ceil_to(int32_t n, int32_t of) { return (n + of - 1) / of * of; }
int32_t ceil_div(int32_t n, int32_t by) { return (n + by - 1) / by; }

int32_t few_grad_w_tiles(int32_t hidden, int32_t experts) {
  return ceil_div(hidden, kFewCols) * ceil_div(experts, kFewExperts);
}

// ---- dx --------------------------------------------------------------------------
// k is short here (the experts), so a wave keeps its 32 rows of dl in registers,
// all k of them, split into two bf16 parts as they are read; only w passes
// shared memory, a stage holding all k of 64 channels.  KB blocks of 64 k: each
// count has a kernel of its own (4096 tokens of 7168 channels on 300 experts by five
// 49 us, by eight, as 512 take, 70).
constexpr int kGradCols = 64;    // channels of a stage
constexpr int kGradRows = 128;   // tokens of a workgroup
constexpr int kGradThreads = 256;

// Before the workgroups of dx come those of something else that dw needs of dl:
// its parts, or with few tokens dw itself.  (Each would take a launch of its own.)
struct Beside {
  int32_t split_blocks, few_blocks, blocks;  // the sum, a multiple of 8
  Parts parts;
  FewGradW few;
};

struct GradX {
  const float* dl;
  int64_t dl_stride;
  const uint16_t* w;   // [experts, hidden]
  const uint16_t* add; // bf16 [bs, hidden], or null
  int64_t add_stride;
  uint16_t* dx;
  int64_t dx_stride;
  int32_t bs, hidden, experts;
  int32_t row_tiles, ranges, jobs;  // jobs: a row tile and a range of channels
};

// The first two parts of 8 values.
__device__ __forceinline__ void two_parts(const float (&f)[8], bf16x8& hi, bf16x8& mid) {
  u32x4 h, m;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t first, second, third;
    pair_parts(f[2 * c], f[2 * c + 1], first, second, third);
    h[c] = first;
    m[c] = second;
  }
  __asm__ volatile("" : "+v"(h), "+v"(m));  // made here, not where they are used
  hi = __builtin_bit_cast(bf16x8, h);
  mid = __builtin_bit_cast(bf16x8, m);
}

// Whether this workgroup was one of those, and its work with it.
__device__ __forceinline__ bool done_beside(const Beside& beside, uint8_t* lds) {
  const int32_t block = blockIdx.x;
  if (block >= beside.blocks) return false;
  if (block < beside.split_blocks)
    split_parts(beside.parts, block, beside.split_blocks);
  else if (block - beside.split_blocks < beside.few_blocks)
    few_grad_w(beside.few, block - beside.split_blocks, lds);
  return true;
}

template <int KB>
__global__ __launch_bounds__(kGradThreads, KB > 4 ? 1 : 2) void grad_x_kernel(
    const GradX p, const Beside beside) {
  constexpr int kLoads = 2 * KB;  // a wave and stage
  constexpr int kBytes = KB * kDepth * kRowBytes;
  constexpr int kTurned = 4096;  // bytes of a wave
  __shared__ __attribute__((aligned(1024))) uint8_t lds[
      2 * kBytes + kGradThreads / kWave * kTurned > kFewBytes
          ? 2 * kBytes + kGradThreads / kWave * kTurned
          : kFewBytes];
  uint8_t* ring = lds;
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  const int half = lane / kSide;
  if (done_beside(beside, lds)) return;
  const int32_t job = own_job(p.jobs, blockIdx.x - beside.blocks);
  const int32_t range = job / p.row_tiles;
  const int32_t row0 = (job % p.row_tiles) * kGradRows + wave * kSide;  // the wave's 32
  const int32_t tiles = (p.hidden + kGradCols - 1) / kGradCols;
  const int32_t first = (int32_t)((int64_t)tiles * range / p.ranges);
  const int32_t end = (int32_t)((int64_t)tiles * (range + 1) / p.ranges);

  const auto send = [&](int32_t tile) {
    const uint32_t to = (uint32_t)(uintptr_t)ring + (tile & 1) * kBytes + wave * kLoads * 1024;
    const int slot = lane % 8;
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int k = (wave * kLoads + n) * 8 + lane / 8;
      const int32_t col = min(tile * kGradCols + (slot ^ col_key(k)) * 8, p.hidden - 8);
      const uint16_t* from = p.w + (int64_t)k * p.hidden + col;
      load_lds16_from(to + n * 1024,
                      k < p.experts ? static_cast<const void*>(from) : &kZeroVec);
    }
  };
  send(first);

  // dl comes and dx goes by whole rows, eight lanes a row, and is turned to a
  // row a lane in 4 KB of shared memory of the wave's own, 16-byte chunks
  // permuted so that all banks are used.  (Each lane on its own row: dx of 4096
  // tokens 54 us.)
  uint8_t* mine = lds + 2 * kBytes + wave * kTurned;
  bf16x8 hi[KB * kSteps], mid[KB * kSteps];
  constexpr int kPasses = 2 * KB;       // of 32 k
  f32x4 v[4];
  const auto read_dl = [&](int pass) {  // (more than one ahead measures the same)
    const int k = 32 * pass + lane % 8 * 4;
    const float* from[4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
      from[n] = p.dl + (int64_t)min(row0 + 8 * n + lane / 8, p.bs - 1) * p.dl_stride;
    if (32 * pass + 32 <= p.experts) {
#pragma unroll
      for (int n = 0; n < 4; ++n) v[n] = *reinterpret_cast<const f32x4_any*>(from[n] + k);
    } else if (p.experts >= 4) {
      // Where a row ends among these, its last four.
      const int at = min(k, p.experts - 4);
#pragma unroll
      for (int n = 0; n < 4; ++n) v[n] = *reinterpret_cast<const f32x4_any*>(from[n] + at);
    } else {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[n][c] = from[n][min(k + c, p.experts - 1)];
    }
  };
  // What read_dl brought, with zeros behind the last expert.
  const auto dl_of = [&](int pass, int n) {
    const int k = 32 * pass + lane % 8 * 4;
    f32x4 dl = v[n];
    if (32 * pass + 32 <= p.experts) return dl;
    if (p.experts >= 4) {
      const int by = k - min(k, p.experts - 4);
      if (by & 1) dl = f32x4{dl[1], dl[2], dl[3], 0.0f};
      if (by & 2) dl = f32x4{dl[2], dl[3], 0.0f, 0.0f};
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (k + c >= p.experts) dl[c] = 0.0f;
    return dl;
  };
  read_dl(0);
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int r = 8 * n + lane / 8;
      *reinterpret_cast<f32x4*>(mine + r * 128 + ((lane % 8 ^ row_key(r)) << 4)) = dl_of(pass, n);
    }
    keep_order();
    if (pass + 1 < kPasses) read_dl(pass + 1);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int r = lane % kSide, chunk = 4 * s + 2 * half;
      float f[8];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(
            mine + r * 128 + ((chunk + n ^ row_key(r)) << 4));
#pragma unroll
        for (int c = 0; c < 4; ++c) f[4 * n + c] = v[c];
      }
      two_parts(f, hi[2 * pass + s], mid[2 * pass + s]);
    }
    keep_order();
  }

  for (int32_t tile = first; tile < end; ++tile) {
    wait_and_meet<0>();
    const int32_t col = tile * kGradCols + lane % 8 * 8;
    u32x4 add[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int32_t row = row0 + 8 * n + lane / 8;
      add[n] = u32x4{0u, 0u, 0u, 0u};
      if (p.add && row < p.bs && col < p.hidden)
        add[n] = load_stream(reinterpret_cast<const u32x4*>(p.add + row * p.add_stride + col));
    }
    if (tile + 1 < end) send(tile + 1);
    const uint8_t* w = ring + (tile & 1) * kBytes;
    f32x16 sum[2] = {};
    bf16x8 next[2] = {read_square<true, true>(w, 0, 0, lane),
                      read_square<true, true>(w, kSide, 0, lane)};
#pragma unroll
    for (int s = 0; s < KB * kSteps; ++s) {
      const bf16x8 i[2] = {next[0], next[1]};
      if (s + 1 < KB * kSteps) {
#pragma unroll
        for (int a = 0; a < 2; ++a) next[a] = read_square<true, true>(w, a * kSide, s + 1, lane);
      }
      keep_order();  // reads one step ahead, not more
#pragma unroll
      for (int a = 0; a < 2; ++a)
        sum[a] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(i[a], mid[s], sum[a], 0, 0, 0);
#pragma unroll
      for (int a = 0; a < 2; ++a)
        sum[a] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(i[a], hi[s], sum[a], 0, 0, 0);
    }
    // 16 rows of 64 channels at a time.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (lane % kSide / 16 == h) {
        const int r = lane % 16;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int chunk = 8 * a + 4 * (q / 2) + 2 * half + q % 2;
            *reinterpret_cast<f32x4*>(mine + r * 256 + ((chunk ^ r) << 4)) =
                f32x4{sum[a][4 * q], sum[a][4 * q + 1], sum[a][4 * q + 2], sum[a][4 * q + 3]};
          }
      }
      keep_order();
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int r = 8 * n + lane / 8;
        const int32_t row = row0 + 16 * h + r;
        u32x4 o;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(
              mine + r * 256 + ((2 * (lane % 8) + m ^ r) << 4));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float lo = v[2 * c], up = v[2 * c + 1];
            if (p.add) {
              lo += bf16lo_to_f32(add[2 * h + n][2 * m + c]);
              up += bf16hi_to_f32(add[2 * h + n][2 * m + c]);
            }
            o[2 * m + c] = bf16_pair(lo, up);
          }
        }
        if (row < p.bs && col < p.hidden)
          store_stream(o, reinterpret_cast<u32x4*>(p.dx + row * p.dx_stride + col));
      }
      keep_order();
    }
  }
}

// ---- dx of small batches ---------------------------------------------------------------
// A workgroup has 32 tokens and 64 channels, and its four waves share the experts:
// a wave reads its 16 * KB of each row of dl and of w, and the waves' sums meet in
// shared memory.
constexpr int kSmallRows = 32;

// Four floats from `from` + k of a row that ends at `end`, zeros behind it.
__device__ __forceinline__ f32x4 four_of_row(const float* from, int k, int end) {
  f32x4 v;
  if (end >= 4) {
    const int at = min(k, end - 4), by = k - at;
    v = *reinterpret_cast<const f32x4_any*>(from + at);
    if (by & 1) v = f32x4{v[1], v[2], v[3], 0.0f};
    if (by & 2) v = f32x4{v[2], v[3], 0.0f, 0.0f};
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = from[min(k + c, end - 1)];
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (k + c >= end) v[c] = 0.0f;
  return v;
}

constexpr int kSmallSums = kSmallRows * kGradCols * 4;  // of a wave
constexpr int small_grad_x_bytes(int kb) {
  const int own = kGradThreads / kWave * (16 * kb * kRowBytes + kSmallSums);
  return own > kFewBytes ? own : kFewBytes;
}

template <int KB>
__global__ __launch_bounds__(kGradThreads) void small_grad_x_kernel(const GradX p,
                                                                    const Beside beside) {
  constexpr int kDepthOf = 16 * KB;                 // experts of a wave
  constexpr int kWaveBytes = kDepthOf * kRowBytes;  // w's rows
  constexpr int kSums = kSmallSums;
  constexpr int kWaves = kGradThreads / kWave;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[small_grad_x_bytes(KB)];
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x / kWave);
  if (done_beside(beside, lds)) return;
  const int32_t job = own_job(p.jobs, blockIdx.x - beside.blocks);
  const int32_t row0 = job % p.row_tiles * kSmallRows, col0 = job / p.row_tiles * kGradCols;
  const int k0 = wave * kDepthOf;
  uint8_t* w = lds + wave * kWaveBytes;
#pragma unroll
  for (int n = 0; n < 2 * KB; ++n) {
    const int k = n * 8 + lane / 8;
    const int32_t col = min(col0 + (lane % 8 ^ col_key(k)) * 8, p.hidden - 8);
    load_lds16_from((uint32_t)(uintptr_t)w + n * 1024,
                    k0 + k < p.experts
                        ? static_cast<const void*>(p.w + (int64_t)(k0 + k) * p.hidden + col)
                        : &kZeroVec);
  }
  // A thread's eight channels of a row at the end.
  const int32_t row = row0 + threadIdx.x / 8, col = col0 + threadIdx.x % 8 * 8;
  const bool real = row < p.bs && col < p.hidden;
  u32x4 add = {0u, 0u, 0u, 0u};
  if (p.add && real)
    add = load_stream(reinterpret_cast<const u32x4*>(p.add + row * p.add_stride + col));
  const float* dl = p.dl + (int64_t)min(row0 + lane % kSide, p.bs - 1) * p.dl_stride;
  f32x4 f[2 * KB];
#pragma unroll
  for (int s = 0; s < KB; ++s)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      f[2 * s + c] = four_of_row(dl, k0 + 16 * s + 8 * (lane / kSide) + 4 * c, p.experts);
  bf16x8 hi[KB], mid[KB];
#pragma unroll
  for (int s = 0; s < KB; ++s) {
    const float v[8] = {f[2 * s][0],     f[2 * s][1],     f[2 * s][2],     f[2 * s][3],
                        f[2 * s + 1][0], f[2 * s + 1][1], f[2 * s + 1][2], f[2 * s + 1][3]};
    two_parts(v, hi[s], mid[s]);
  }
  wait_own<0>();
  f32x16 sum[2] = {};
#pragma unroll
  for (int s = 0; s < KB; ++s)
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const bf16x8 i = read_square<true, true>(w, a * kSide, s, lane);
      sum[a] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(i, mid[s], sum[a], 0, 0, 0);
      sum[a] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(i, hi[s], sum[a], 0, 0, 0);
    }
  uint8_t* sums = lds + kWaves * kWaveBytes;
  const int r = lane % kSide;
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int chunk = 8 * a + 4 * (q / 2) + 2 * (lane / kSide) + q % 2;
      *reinterpret_cast<f32x4*>(sums + wave * kSums + r * 256 + ((chunk ^ r % 16) << 4)) =
          f32x4{sum[a][4 * q], sum[a][4 * q + 1], sum[a][4 * q + 2], sum[a][4 * q + 3]};
    }
  meet();
  if (!real) return;
  const int t = threadIdx.x / 8;
  u32x4 o;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    f32x4 v = {};
#pragma unroll
    for (int k = 0; k < kWaves; ++k)
      v += *reinterpret_cast<const f32x4*>(sums + k * kSums + t * 256 +
                                           ((2 * (threadIdx.x % 8) + m ^ t % 16) << 4));
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float lo = v[2 * c], up = v[2 * c + 1];
      if (p.add) {
        lo += bf16lo_to_f32(add[2 * m + c]);
        up += bf16hi_to_f32(add[2 * m + c]);
      }
      o[2 * m + c] = bf16_pair(lo, up);
    }
  }
  store_stream(o, reinterpret_cast<u32x4*>(p.dx + row * p.dx_stride + col));
}

hipError_t launch_grad_x(GradX p, Beside beside, hipStream_t stream) {
  beside.blocks = (beside.split_blocks + beside.few_blocks + 7) / 8 * 8;
  const int32_t tiles = (p.hidden + kGradCols - 1) / kGradCols;
  // As long as the small ones run all at once.  (us, small and not: 14 tokens of 2816
  // channels on 262 experts 6.1, 10.7; 128 of 7168 on 256 7.1, 12.1, on 64 4.8, 7.3; 330 of
  // 2752 on 383 10.0, 12.4; 777 of 1408 on 60, more of them, 6.4, 6.0.)
  const int32_t block_count = ceil_div(p.experts, kDepth);
  const int32_t small_bytes = small_grad_x_bytes(block_count);
  const bool small =
      (int64_t)ceil_div(p.bs, kSmallRows) * tiles <= kUnits * (160 * 1024 / small_bytes);
  p.row_tiles = ceil_div(p.bs, small ? kSmallRows : kGradRows);
  const int32_t resident = (p.experts > 256 ? 1 : 2) * kUnits;
  // Ranges of channels: the fewest rounds of workgroups, whose start takes about
  // as long as three tiles.
  int64_t best = INT64_MAX;
  for (int32_t r = 1; r <= tiles && r <= 64; ++r) {
    const int64_t jobs = (int64_t)p.row_tiles * r;
    const int64_t cost = (jobs + resident - 1) / resident * (3 + (tiles + r - 1) / r);
    if (cost < best) {
      best = cost;
      p.ranges = r;
    }
  }
  if (small) p.ranges = tiles;
  p.jobs = p.row_tiles * p.ranges;
  const dim3 grid((uint32_t)(beside.blocks + p.jobs));
#define MOE_GRAD_X(KB)                                                                \
  case KB:                                                                             \
    if (small)                                                                         \
      launch_kernel(small_grad_x_kernel<KB>, grid, kGradThreads, stream, p, beside);   \
    else                                                                               \
      launch_kernel(grad_x_kernel<KB>, grid, kGradThreads, stream, p, beside);         \
    break
  switch (block_count) {
    MOE_GRAD_X(1);
    MOE_GRAD_X(2);
    MOE_GRAD_X(3);
    MOE_GRAD_X(4);
    MOE_GRAD_X(5);
    MOE_GRAD_X(6);
    MOE_GRAD_X(7);
    MOE_GRAD_X(8);
  }
#undef MOE_GRAD_X
  return hipGetLastError();
}

// out[r, c] = sum over the splits of parts[s, r, c], `cols` padded to four in
// the parts: SLICES threads add every SLICES-th split of four columns, then
// their sums in turn.
template <int SLICES>
__global__ __launch_bounds__(256) void sum_splits_kernel(const float* __restrict__ parts,
                                                         int32_t splits, int64_t rows,
                                                         int32_t quads, int32_t cols,
                                                         float* __restrict__ out,
                                                         int64_t out_stride, bool vectors) {
  constexpr int kOut = 256 / SLICES;
  constexpr int kAtOnce = 4;   // loads under way, the last ones too
  __shared__ f32x4 sums[SLICES][kOut];
  const int slice = threadIdx.x / kOut, at = threadIdx.x % kOut;
  const int64_t all = rows * quads, n = (int64_t)blockIdx.x * kOut + at;
  f32x4 s = {};
  if (n < all) {
    const f32x4* from = reinterpret_cast<const f32x4*>(parts) + n;
    for (int32_t k0 = slice; k0 < splits; k0 += kAtOnce * SLICES) {
      f32x4 v[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        v[k] = load_stream(from + min(k0 + k * SLICES, splits - 1) * all);
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (k0 + k * SLICES < splits) s += v[k];
    }
  }
  if (SLICES > 1) {
    sums[slice][at] = s;
    __syncthreads();
    if (slice > 0) return;
#pragma unroll
    for (int k = 1; k < SLICES; ++k) s += sums[k][at];
  }
  if (n >= all) return;
  const int64_t r = n / quads;
  const int32_t c = (int32_t)(n - r * quads) * 4;
  float* to = out + r * out_stride + c;
  if (vectors) {
    *reinterpret_cast<f32x4*>(to) = s;
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (c + u < cols) to[u] = s[u];
  }
}

hipError_t launch_sum_splits(const float* parts, int32_t splits, int64_t rows, int32_t cols,
                             float* out, int64_t out_stride, bool vectors, hipStream_t stream) {
  const int32_t quads = (cols + 3) / 4;
  const int64_t all = rows * quads;
  // So many slices that the card is full; more than two splits one after the
  // other would each wait for memory (7 of 60 x 1408: 1.5 us more).
#define MOE_SUM(SLICES)                                                                       \
  launch_kernel(sum_splits_kernel<SLICES>,                                                    \
                dim3((uint32_t)((all + 256 / SLICES - 1) / (256 / SLICES))), 256, stream, parts, \
                splits, rows, quads, cols, out, out_stride, vectors)
  if (all >= (1 << 17) || splits < 3)
    MOE_SUM(1);
  else
    MOE_SUM(8);
#undef MOE_SUM
  return hipGetLastError();
}

__global__ __launch_bounds__(256) void fill_zero_kernel(float* to, int64_t count) {
  for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < count;
       n += (int64_t)gridDim.x * 256)
    to[n] = 0.0f;
}

// What a workgroup of a shape costs, in us: from its start to its first block's
// products and from its last one's to its end, and a block; the latter with one
// workgroup a unit and, of shapes whose stages fit twice, with two.
struct Cost {
  int tile_i, tile_j, a_unit;
  float ends, block, block_of_two;
};

struct Plan {
  int shape;
  int32_t tiles_i, tiles_j, splits, blocks;
  float time;   // us
};

// The shape and the number of shares of the depth that take the least time.
// Shares have their sums written and read again (some 8 TB/s, as the caches
// hold them) in a launch of its own.
template <int SHAPES>
Plan plan_product(const Cost (&costs)[SHAPES], int32_t n_i, int32_t n_j, int32_t depth) {
  constexpr int32_t kMostSplits = 32;
  Plan best = {};
  best.time = 3.0e38f;
  for (int s = 0; s < SHAPES; ++s) {
    const Cost& c = costs[s];
    Plan p;
    p.shape = s;
    p.tiles_i = ceil_div(n_i, c.tile_i);
    p.tiles_j = ceil_div(n_j, c.tile_j);
    p.blocks = ceil_div(depth, kDepth);
    const int64_t tiles = (int64_t)p.tiles_i * p.tiles_j;
    for (p.splits = 1; p.splits <= kMostSplits && p.splits <= p.blocks; ++p.splits) {
      const int64_t jobs = tiles * p.splits, places = (int64_t)c.a_unit * kUnits;
      if (p.splits > 1 && jobs > 2 * places) break;
      const float rounds = (float)((jobs + places - 1) / places);
      const float block = jobs > kUnits ? c.block_of_two : c.block;
      p.time = rounds * (c.ends + block * (float)ceil_div(p.blocks, p.splits));
      if (p.splits > 1) p.time += 2.0f + (float)p.splits * (float)n_i * (float)n_j * 1.0e-6f;
      if (p.time < best.time) best = p;
    }
  }
  return best;
}

// 64 x 64 for short sums and few tokens, 128 x 128 and 128 x 256 for ever more
// (us, each at its best number of shares: 128 tokens of 7168 channels on 256
// experts 9.0, 11.1, 12.2; 2048 21.2, 21.4, 25.3; 4096 33.7, 29.6, 33.7; 8192 66.4,
// 48.5, 48.4; 16384 on 512 254, 161, 138; 16384 of 1024 on 128 12.0, 14.9, 21.2).
using ForwardSmall = Shape<false, false, 1, 1, 1, 2, 2, 4>;
using ForwardMiddle = Shape<false, false, 1, 2, 1, 2, 4, 3>;
using ForwardLarge = Shape<false, false, 1, 2, 2, 2, 4, 3>;
constexpr Cost kForward[] = {{64, 64, 2, 2.0f, 0.36f, 0.56f},
                             {128, 128, 1, 3.0f, 0.68f, 0.68f},
                             {128, 256, 1, 3.0f, 1.14f, 1.14f}};
// 16 x 16 and 32 x 32 tiles whose k eight and four waves share, against those: (us,
// 128 tokens of 7168 channels on 256 experts 6.4, 12.6, 9.5; 512 12.7, 12.8, 13.9; 512
// of 2048 on 500 9.1, 6.2, 10.8; 777 of 1408 on 60 4.2, 5.3, 8.3; 8192 of 2048 on 64
// 15.7, 9.9, 13.7; 16384 of 512 on 60 15.1, 8.1, 7.6; 4096 of 1024 on 512 32.1, 17.4,
// 12.2.  64 x 64 tiles so: 14.4 where 32 x 32 take 16.0, 1094 of 3008 on 494, but level
// or worse elsewhere.)  What they cost besides the launch: rounds of workgroups,
// two a unit, each a start and a wave's blocks, `block` us where no two share a
// unit.
struct SharedCost {
  int side, waves;
  float block, block_of_two;
};
constexpr SharedCost kSharedK[] = {{16, 8, 0.32f, 0.70f}, {32, 4, 0.36f, 0.85f}};
constexpr int kSharedShapes = 3;   // Plan::shape of the first of them

Plan forward_plan(int32_t bs, int32_t hidden, int32_t experts) {
  Plan best = plan_product(kForward, experts, bs, hidden);
  best.time += best.splits > 1 ? 3.0f : 2.0f;
  for (int s = 0; s < 2; ++s) {
    const SharedCost& c = kSharedK[s];
    Plan p = {kSharedShapes + s, ceil_div(experts, c.side), ceil_div(bs, c.side), 1,
              ceil_div(hidden, kDepth), 0.0f};
    const int32_t jobs = p.tiles_i * p.tiles_j;
    if (jobs > most_items(c.waves * kWave)) continue;  // a workgroup each, in one launch
    const float rounds = fmaxf(1.0f, (float)jobs / (2 * kUnits));  // the last one fills up
    p.time = 2.3f + rounds * (0.5f + (jobs > kUnits ? c.block_of_two : c.block) *
                                         (float)ceil_div(p.blocks, c.waves));
    if (p.time < best.time) best = p;
  }
  return best;
}

using GradWSmall = Shape<true, true, 3, 1, 1, 2, 2, 2>;
using GradWLarge = Shape<true, true, 3, 2, 2, 4, 2, 2>;
constexpr Cost kGradW[] = {{64, 64, 2, 3.0f, 0.75f, 0.85f}, {256, 128, 1, 4.0f, 2.4f, 2.4f}};
Plan grad_w_plan(int32_t bs, int32_t hidden, int32_t experts) {
  return plan_product(kGradW, hidden, experts, bs);
}

// In how many ranges of tokens few_grad_w makes dw, 0 where the products of parts
// made beforehand are to be taken.  Those need two launches more, kFewGain us, but
// split dl once, not once for every 128 channels.  More workgroups than half the
// card's are in the way of dx's.  (us, dx and dw, in ranges and by parts: 128
// tokens of 7168 channels on 64 experts 7.6, 11.6, on 256 14.9, 18.4; 777 of 1408 on
// 60 10.5, 14.9; 512 of 7168 on 256 19.3, 25.5; 8192 of 2048 on 64 33.7, 36.9; 4096 of
// 7168 on 64 51.0, 52.7, 2048 on 256 62.2, 59.1.  dw alone, 512 of 7168 on 256 17.7,
// 16.4, 8192 of 2048 on 64 21.3, 20.4: it goes by the same rule, so that its bits do
// not depend on what else is asked.)
// (Ranges, dw alone: 10165 tokens of 64 channels on 14 experts in 32 15.6, in 96 10.5, in
// 128 10.9; 16384 of 512 on 8 18.3, 13.3, 12.1.)
constexpr float kFewGain = 9.0f;
constexpr int32_t kMostRanges = 96;

int32_t few_grad_w_ranges(int32_t bs, int32_t hidden, int32_t experts) {
  const int32_t stages = ceil_div(bs, kDepth), tiles = few_grad_w_tiles(hidden, experts);
  int32_t best = 0;
  float least = grad_w_plan(bs, hidden, experts).time + kFewGain;
  for (int32_t r = 1; r <= stages && r <= kMostRanges; ++r) {
    const int32_t jobs = tiles * r;
    float time = (float)ceil_div(jobs, kUnits) * (2.0f + 1.6f * (float)ceil_div(stages, r));
    if (jobs > kUnits / 2) time += 2.5f;
    if (r > 1) time += 2.5f + (float)r * (0.03f + (float)experts * (float)hidden * 1.0e-6f);
    if (time < least) {
      least = time;
      best = r;
    }
  }
  return best;
}

template <class S>
hipError_t launch_product(Product p, const Plan& plan, hipStream_t stream) {
  p.tiles_i = plan.tiles_i;
  p.tiles_j = plan.tiles_j;
  p.splits = plan.splits;
  p.blocks = plan.blocks;
  p.jobs = plan.tiles_i * plan.tiles_j * plan.splits;
  const int32_t resident = kUnits * (160 * 1024 / (S::kStages * S::kStageBytes));
  launch_kernel(router_kernel<S>, dim3((uint32_t)(p.jobs < resident ? p.jobs : resident)),
                S::kThreads, stream, p);
  return hipGetLastError();
}

template <int SIDE, int WAVES, int STAGES>
hipError_t launch_shared_k(const RouterArgs& a, const Plan& plan, hipStream_t stream) {
  SharedK p = {};
  p.i = {static_cast<const uint16_t*>(a.weight), a.hidden, 0, a.num_experts, a.hidden};
  p.j = {static_cast<const uint16_t*>(a.x), a.x_stride, 0, a.bs, a.hidden};
  p.tiles_i = plan.tiles_i;
  p.tiles_j = plan.tiles_j;
  p.blocks = plan.blocks;
  p.jobs = plan.tiles_i * plan.tiles_j;
  // An XCD's run of jobs is about as many tokens wide as experts.
  p.band = 1;
  while (32 * (int64_t)p.band * p.band <= p.jobs && 2 * p.band <= p.tiles_j) p.band *= 2;
  p.out = a.logits;
  p.out_stride = a.logits_stride;
  p.experts = a.num_experts;
  p.bs = a.bs;
  launch_kernel(shared_k_kernel<SIDE, WAVES, STAGES>, dim3((uint32_t)p.jobs), WAVES * kWave,
                stream, p);
  return hipGetLastError();
}

hipError_t launch_one_token(const RouterArgs& a, hipStream_t stream) {
  launch_kernel(one_token_kernel, dim3((uint32_t)ceil_div(a.num_experts, 4)), 256, stream,
                static_cast<const u32x4*>(a.x), static_cast<const u32x4*>(a.weight), a.hidden / 8,
                a.num_experts, a.logits);
  return hipGetLastError();
}

size_t parts_bytes(int32_t bs, int32_t experts) {
  return (size_t)3 * ceil_to(bs, kDepth) * ceil_to(experts, kDepth) * sizeof(uint16_t);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

hipError_t launch_fill_zero(float* to, int64_t count, hipStream_t stream) {
  const int64_t want = (count + 255) / 256;
  launch_kernel(fill_zero_kernel, dim3((uint32_t)(want < 65536 ? want : 65536)), 256, stream, to,
                count);
  return hipGetLastError();
}

size_t router_workspace_bytes(int32_t bs, int32_t hidden, int32_t num_experts) {
  if (bs <= 1) return 0;
  const Plan plan = forward_plan(bs, hidden, num_experts);
  return plan.splits == 1
             ? 0
             : (size_t)plan.splits * bs * ceil_to(num_experts, 4) * sizeof(float);
}

size_t router_backward_workspace_bytes(int32_t bs, int32_t hidden, int32_t num_experts) {
  const int32_t ranges = few_grad_w_ranges(bs, hidden, num_experts);
  if (ranges) return ranges == 1 ? 0 : (size_t)ranges * num_experts * hidden * sizeof(float);
  const Plan plan = grad_w_plan(bs, hidden, num_experts);
  return parts_bytes(bs, num_experts) +
         (plan.splits == 1 ? 0 : (size_t)plan.splits * num_experts * hidden * sizeof(float));
}

hipError_t launch_router(const RouterArgs& a, void* workspace, hipStream_t stream) {
  if (a.bs == 1) return launch_one_token(a, stream);
  const Plan plan = forward_plan(a.bs, a.hidden, a.num_experts);
  if (plan.shape == kSharedShapes) return launch_shared_k<16, 8, 2>(a, plan, stream);
  if (plan.shape == kSharedShapes + 1) return launch_shared_k<32, 4, 2>(a, plan, stream);
  Product p = {};
  p.i = {static_cast<const uint16_t*>(a.weight), a.hidden, 0, a.num_experts, a.hidden};
  p.j = {static_cast<const uint16_t*>(a.x), a.x_stride, 0, a.bs, a.hidden};
  p.i_first = true;
  p.rows = a.bs;
  const int32_t padded = ceil_to(a.num_experts, 4);
  const bool vectors = a.num_experts % 4 == 0 && a.logits_stride % 4 == 0 && aligned16(a.logits);
  if (plan.splits == 1) {
    p.out = a.logits;
    p.out_stride = a.logits_stride;
    p.cols = a.num_experts;
    p.vectors = vectors;
  } else {
    p.out = static_cast<float*>(workspace);
    p.out_stride = p.cols = padded;
    p.split_stride = (int64_t)a.bs * padded;
    p.vectors = true;
  }
  const hipError_t err = plan.shape == 0   ? launch_product<ForwardSmall>(p, plan, stream)
                         : plan.shape == 1 ? launch_product<ForwardMiddle>(p, plan, stream)
                                           : launch_product<ForwardLarge>(p, plan, stream);
  if (err != hipSuccess || plan.splits == 1) return err;
  return launch_sum_splits(static_cast<const float*>(workspace), plan.splits, a.bs,
                           a.num_experts, a.logits, a.logits_stride, vectors, stream);
}

hipError_t launch_router_backward(const RouterArgs& a, void* workspace, hipStream_t stream) {
  if (a.bs == 0) {
    if (a.grad_weight == nullptr) return hipSuccess;
    return launch_fill_zero(a.grad_weight, (int64_t)a.num_experts * a.hidden, stream);
  }
  Beside beside = {};
  const int32_t few = few_grad_w_ranges(a.bs, a.hidden, a.num_experts);
  if (a.grad_weight && few) {
    beside.few = {a.grad_logits, a.grad_logits_stride, static_cast<const uint16_t*>(a.x),
                  a.x_stride, a.bs, a.hidden, a.num_experts, few,
                  a.num_experts % 4 == 0 && a.grad_logits_stride % 4 == 0 &&
                      aligned16(a.grad_logits),
                  few == 1 ? a.grad_weight : static_cast<float*>(workspace)};
    beside.few_blocks = few * few_grad_w_tiles(a.hidden, a.num_experts);
  } else if (a.grad_weight) {
    beside.parts = {a.grad_logits, a.grad_logits_stride, a.bs, a.num_experts,
                    ceil_to(a.bs, kDepth), ceil_to(a.num_experts, kDepth),
                    static_cast<uint16_t*>(workspace)};
    beside.split_blocks = split_blocks(beside.parts);
  }
  if (a.grad_x) {
    GradX p = {};
    p.dl = a.grad_logits;
    p.dl_stride = a.grad_logits_stride;
    p.w = static_cast<const uint16_t*>(a.weight);
    p.add = static_cast<const uint16_t*>(a.grad_x_add);
    p.add_stride = a.grad_x_add_stride;
    p.dx = static_cast<uint16_t*>(a.grad_x);
    p.dx_stride = a.grad_x_stride;
    p.bs = a.bs;
    p.hidden = a.hidden;
    p.experts = a.num_experts;
    const hipError_t err = launch_grad_x(p, beside, stream);
    if (err != hipSuccess) return err;
  } else if (few) {
    launch_kernel(few_grad_w_kernel, dim3((uint32_t)beside.few_blocks), 256, stream, beside.few);
  } else {
    launch_kernel(split_kernel, dim3((uint32_t)beside.split_blocks), 256, stream, beside.parts);
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.grad_weight == nullptr || few == 1) return err;
  if (few)
    return launch_sum_splits(static_cast<const float*>(workspace), few, a.num_experts, a.hidden,
                             a.grad_weight, a.hidden, true, stream);
  const int32_t rows = beside.parts.rows, cols = beside.parts.cols;
  uint16_t* parts = beside.parts.parts;
  const int64_t plane = (int64_t)rows * cols;
  const Plan plan = grad_w_plan(a.bs, a.hidden, a.num_experts);
  float* shares = reinterpret_cast<float*>(parts + 3 * plane);
  Product p = {};
  p.i = {static_cast<const uint16_t*>(a.x), a.x_stride, 0, a.hidden, a.bs};
  p.j = {parts, cols, plane, cols, rows};
  p.i_first = false;
  p.out = plan.splits == 1 ? a.grad_weight : shares;
  p.out_stride = p.cols = a.hidden;
  p.rows = a.num_experts;
  p.split_stride = (int64_t)a.num_experts * a.hidden;
  p.vectors = true;
  err = plan.shape == 0 ? launch_product<GradWSmall>(p, plan, stream)
                        : launch_product<GradWLarge>(p, plan, stream);
  if (err != hipSuccess || plan.splits == 1) return err;
  return launch_sum_splits(shares, plan.splits, a.num_experts, a.hidden, a.grad_weight, a.hidden,
                           true, stream);
}

}  // namespace moe
