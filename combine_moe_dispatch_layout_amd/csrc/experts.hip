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
#include "moe_internal.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kScaleBlock = 128;  // channels per scale
constexpr int kTileThreads = 256;
constexpr int kTileRows = 64;
constexpr int kTileCols = 128;    // output channels per workgroup

// The row tiles of all experts, from the device's counts: first[e] is the
// number of tiles before expert e, first[E] their total.  Sums saturate at
// kMostTiles, above what disjoint segments of 2^30 rows can make, so counts
// whose segments overlap cannot wrap them; such counts give no tiles at all.
constexpr int kMostTiles = 1 << 30;

struct TileMap {
  int first[kMaxExperts + 1];
  int wave_sum[kTileThreads / kWave];
};

// Rows of expert e that lie inside the buffer: [start, start + rows).
__device__ __forceinline__ void segment_of(const int32_t* __restrict__ counts,
                                           const int32_t* __restrict__ send, int64_t cap,
                                           int e, int64_t& start, int64_t& rows, bool& cut) {
  if (counts == nullptr) {
    start = 0;
    rows = cap;
    cut = false;
    return;
  }
  const int64_t s = send[e], c = counts[e];
  cut = s < 0 || c < 0 || (c > 0 && s + c > cap);
  start = s < 0 ? 0 : s;
  rows = (s < 0 || c <= 0 || s >= cap) ? 0 : (c < cap - s ? c : cap - s);
}

__device__ __forceinline__ void build_tile_map(TileMap& map, const int32_t* __restrict__ counts,
                                               const int32_t* __restrict__ send, int32_t E,
                                               int64_t cap, int tile_rows, int32_t* status) {
  constexpr int kPer = kMaxExperts / kTileThreads;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  int n[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    n[i] = 0;
    if (e < E) {
      int64_t start, rows;
      bool cut;
      segment_of(counts, send, cap, e, start, rows, cut);
      n[i] = (int)((rows + tile_rows - 1) / tile_rows);
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
  for (int w = 0; w < kTileThreads / kWave; ++w) {
    if (w < wave) base = min(base + map.wave_sum[w], kMostTiles);
    total = min(total + map.wave_sum[w], kMostTiles);
  }
  const bool overlap = total > cap / tile_rows + E;
  if (overlap && status && blockIdx.x == 0 && tid == 0) atomicOr(status, (int)MOE_FLAG_GUARD);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e < E) map.first[e] = base;
    base += n[i];
  }
  if (tid == 0) map.first[E] = overlap ? 0 : total;
  __syncthreads();
}

// The expert whose tiles hold tile t (first[e] <= t < first[e + 1]).
__device__ __forceinline__ int expert_of(const TileMap& map, int32_t E, int t) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (map.first[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
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

// Element offset in a 128-byte-row LDS tile, 16-byte chunks permuted by row
// so that the 16 rows a fragment read touches fall on different banks.
__device__ __forceinline__ int lds_chunk(int row, int chunk) {
  return row * kScaleBlock + ((chunk ^ (row & 7)) << 4);
}

__device__ __forceinline__ i32x8 read_fragment(const uint8_t* tile, int row, int quarter) {
  const u32x4 lo = *reinterpret_cast<const u32x4*>(tile + lds_chunk(row, quarter));
  const u32x4 hi = *reinterpret_cast<const u32x4*>(tile + lds_chunk(row, quarter + 4));
  i32x8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = (int)lo[i];
    f[4 + i] = (int)hi[i];
  }
  return f;
}

// The sum of a block's products from the e4m3 matrix instruction.  It adds
// groups of 8 products aligned to the largest of them, of which it keeps 13
// bits below the leading one; groups and blocks add up in fp32.
__device__ __forceinline__ f32x4 block_product(const i32x8& w, const i32x8& x) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, 0, 0, 0, 0, 0, 0);
}

// Eight codes as fp16 (exact).
__device__ __forceinline__ f16x8 widen8(int lo, int hi) {
  f16x8 f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(i ? hi : lo, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(i ? hi : lo, 1.0f, true);
    f[4 * i] = a[0];
    f[4 * i + 1] = a[1];
    f[4 * i + 2] = b[0];
    f[4 * i + 3] = b[1];
  }
  return f;
}

// The same sum in full fp32: the codes widened to fp16, whose products the
// matrix unit adds with 24 bits.
__device__ __forceinline__ f32x4 block_product_fp32(const i32x8& w, const i32x8& x) {
  f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(w[i], w[i + 1]), widen8(x[i], x[i + 1]), c,
                                               0, 0, 0);
  return c;
}

// g / (1 + e^-g) * u.
__device__ __forceinline__ float gated(float g, float u) {
  const float e = __builtin_amdgcn_exp2f(g * -1.44269504088896341f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// Four e4m3 codes of h / s (s = amax / 448).  A zero scale gives zero codes;
// a block with an infinity or a NaN (its scale says so) gives NaN codes.
__device__ __forceinline__ uint32_t codes4(const float (&h)[4], float s) {
  if (s == 0.0f) return 0u;
  if (!(s < __builtin_inff())) return 0x7F7F7F7Fu;
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = __builtin_amdgcn_fmed3f(h[i] / s, 448.0f, -448.0f);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
  return (uint32_t)w;
}

template <bool GATED>
__global__ __launch_bounds__(kTileThreads) void product_kernel(const ProductArgs p) {
  constexpr int kSub = GATED ? 4 : 2;       // 16-channel weight tiles per wave
  constexpr int kWRows = GATED ? 2 * kTileCols : kTileCols;
  constexpr int kRowSub = kTileRows / 16;
  constexpr int kXLoads = kTileRows * kScaleBlock / 16 / kTileThreads;
  constexpr int kWLoads = kWRows * kScaleBlock / 16 / kTileThreads;
  __shared__ TileMap map;
  __shared__ alignas(16) uint8_t x_lds[kTileRows * kScaleBlock];
  __shared__ alignas(16) uint8_t w_lds[kWRows * kScaleBlock];
  __shared__ uint32_t amax_lds[kTileThreads / kWave][kTileRows];

  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int l16 = lane & 15, quarter = lane >> 4;
  const int32_t kb = p.K / kScaleBlock, nb = (p.N + kScaleBlock - 1) / kScaleBlock;
  const int32_t col_tiles = (p.cols + kTileCols - 1) / kTileCols;
  build_tile_map(map, p.counts, p.send, p.E, p.cap, kTileRows, p.status);
  const int64_t tiles = (int64_t)map.first[p.E] * col_tiles;

  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int e = expert_of(map, p.E, (int)(tile / col_tiles));
    const int32_t row_tiles = map.first[e + 1] - map.first[e];
    const int64_t in_expert = tile - (int64_t)map.first[e] * col_tiles;
    const int32_t ct = (int32_t)(in_expert / row_tiles), rt = (int32_t)(in_expert % row_tiles);
    int64_t start, rows;
    bool cut;
    segment_of(p.counts, p.send, p.cap, e, start, rows, cut);
    const int64_t row0 = start + (int64_t)rt * kTileRows;
    const int32_t live = (int32_t)min((int64_t)kTileRows, start + rows - row0);
    const int32_t col0 = ct * kTileCols;
    const uint8_t* we = p.w + (int64_t)e * p.N * p.K;
    const float* wse = p.w_scales + (int64_t)e * nb * kb;

    const uint8_t* x_src[kXLoads];
    const uint8_t* w_src[kWLoads];
    int x_dst[kXLoads], w_dst[kWLoads];
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
      const int c = i * kTileThreads + tid, row = c >> 3;
      x_src[i] = p.x + (row0 + min(row, live - 1)) * p.xs + (c & 7) * 16;
      x_dst[i] = lds_chunk(row, c & 7);
    }
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) {
      const int c = i * kTileThreads + tid, row = c >> 3;
      const int in_half = row & (kTileCols - 1);
      const int64_t n = min(col0 + in_half, p.cols - 1) + (row >= kTileCols ? p.cols : 0);
      w_src[i] = we + n * p.K + (c & 7) * 16;
      w_dst[i] = lds_chunk(row, c & 7);
    }
    const float* xs_src[kRowSub];
#pragma unroll
    for (int r = 0; r < kRowSub; ++r)
      xs_src[r] = p.x_scales + (row0 + min(r * 16 + l16, live - 1)) * kb;
    const float* ws_src[GATED ? 2 : 1];
    ws_src[0] = wse + (int64_t)(col0 / kScaleBlock) * kb;
    if (GATED) ws_src[GATED ? 1 : 0] = wse + (int64_t)((p.cols + col0) / kScaleBlock) * kb;

    f32x4 acc[kSub][kRowSub];
#pragma unroll
    for (int s = 0; s < kSub; ++s)
#pragma unroll
      for (int r = 0; r < kRowSub; ++r) acc[s][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int32_t b = 0; b < kb; ++b) {
      u32x4 xv[kXLoads], wv[kWLoads];
#pragma unroll
      for (int i = 0; i < kXLoads; ++i)
        xv[i] = *reinterpret_cast<const u32x4*>(x_src[i] + (int64_t)b * kScaleBlock);
#pragma unroll
      for (int i = 0; i < kWLoads; ++i)
        wv[i] = *reinterpret_cast<const u32x4*>(w_src[i] + (int64_t)b * kScaleBlock);
      float sx[kRowSub];
#pragma unroll
      for (int r = 0; r < kRowSub; ++r) sx[r] = xs_src[r][b];
      __syncthreads();  // the previous block's fragments are read
#pragma unroll
      for (int i = 0; i < kXLoads; ++i) *reinterpret_cast<u32x4*>(x_lds + x_dst[i]) = xv[i];
#pragma unroll
      for (int i = 0; i < kWLoads; ++i) *reinterpret_cast<u32x4*>(w_lds + w_dst[i]) = wv[i];
      __syncthreads();
      i32x8 xf[kRowSub];
#pragma unroll
      for (int r = 0; r < kRowSub; ++r) xf[r] = read_fragment(x_lds, r * 16 + l16, quarter);
#pragma unroll
      for (int s = 0; s < kSub; ++s) {
        const int row = (s >> 1) * kTileCols + wave * 32 + (s & 1) * 16 + l16;
        const i32x8 wf = read_fragment(w_lds, row, quarter);
        const float sw = ws_src[GATED ? s >> 1 : 0][b];
#pragma unroll
        for (int r = 0; r < kRowSub; ++r) {
          const f32x4 part = GATED ? block_product_fp32(wf, xf[r]) : block_product(wf, xf[r]);
          const float f = sx[r] * sw;
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[s][r][i] = __builtin_fmaf(f, part[i], acc[s][r][i]);
        }
      }
    }

    if constexpr (!GATED) {
#pragma unroll
      for (int r = 0; r < kRowSub; ++r) {
        const int row = r * 16 + l16;
        if (row >= live) continue;
#pragma unroll
        for (int s = 0; s < kSub; ++s) {
          const int32_t col = col0 + wave * 32 + s * 16 + quarter * 4;
          if (col >= p.cols) continue;
          const f32x4 v = acc[s][r];
          const u32x2 o = {f32_to_bf16_rne(v[0]) | (f32_to_bf16_rne(v[1]) << 16),
                           f32_to_bf16_rne(v[2]) | (f32_to_bf16_rne(v[3]) << 16)};
          *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + (row0 + row) * p.out_stride +
                                    col) = o;
        }
      }
    } else {
      float h[2][kRowSub][4];
#pragma unroll
      for (int r = 0; r < kRowSub; ++r) {
        uint32_t m = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[s][r][i] = gated(acc[s][r][i], acc[(GATED ? 2 : 0) + s][r][i]);
            m = max(m, __float_as_uint(h[s][r][i]) & 0x7FFFFFFFu);
          }
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
        if (quarter == 0) amax_lds[wave][r * 16 + l16] = m;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kRowSub; ++r) {
        const int row = r * 16 + l16;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < kTileThreads / kWave; ++w) m = max(m, amax_lds[w][row]);
        const float s = __uint_as_float(m) / 448.0f;
        if (row < live) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) +
                                         (row0 + row) * p.out_stride + col0 + wave * 32 +
                                         i * 16 + quarter * 4) = codes4(h[i][r], s);
          if (wave == 0 && quarter == 0)
            p.out_scales[(row0 + row) * (p.cols / kScaleBlock) + ct] = s;
        }
      }
      __syncthreads();  // amax_lds is free for the next tile
    }
  }
}

template <bool GATED>
hipError_t launch_product(const ProductArgs& p, int64_t expected_rows, hipStream_t stream) {
  const int64_t col_tiles = (p.cols + kTileCols - 1) / kTileCols;
  const int64_t row_tiles =
      expected_rows / kTileRows + (p.counts ? (expected_rows < p.E ? expected_rows : p.E) : 1);
  const int64_t want = row_tiles * col_tiles;
  const dim3 grid((uint32_t)(want < 1 ? 1 : want < 65536 ? want : 65536));
  launch_kernel(product_kernel<GATED>, grid, kTileThreads, stream, p);
  return hipGetLastError();
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
