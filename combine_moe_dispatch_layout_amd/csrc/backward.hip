// backward.hip -- the gradient of the combine.  With
//   out[t] = sum_j w[t, j] * y[slot(t, j)] + shared[t]   and   g = dL/dout:
//   dy[slot(t, j)] = w[t, j] * g[t]        (rounded once to bf16)
//   dw[t, j]       = <g[t], y[slot(t, j)]> (fp32)
// and the shared row's gradient is g itself.  The scatter's gradient is the
// combine's gather-sum with unit weights (combine.hip).
//
// Each row of y is read once and each row of dy written once; a token's pairs
// run on one XCD, whose L2 gives them g.  Long rows have a workgroup a pair,
// short ones (up to 1024 channels, or 2048 where the pairs are many) a group
// of lanes.  Memory bounds both: 4096 tokens of 7168 channels, K = 8, take 182
// to 192 us (1.0 GB at 5.2 to 5.5 TB/s; a copy of 2 GiB reaches 4.8 to 5.0), 128
// tokens 8.9 to 9.3; 16384 tokens of 512 channels 54 to 59 us (0.285 GB at 4.8
// to 5.3 TB/s).
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kShortThreads = 256;
// Up to this many pairs every pair has a group of lanes (or a workgroup) of its
// own; beyond, groups take two of rows of 264 to 2048 channels (shorter rows
// keep a group a pair, longer ones a workgroup).
constexpr int64_t kFewPairs = 4096;
// Pairs of one launch (2^24), of at most a workgroup each: larger batches take
// several.
constexpr int32_t kMostPairs = most_items(kThreads);

// Eight channels of w * g, rounded to bf16.
__device__ __forceinline__ u32x4 scaled(const u32x4& g, float w) {
  u32x4 o;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    o[c] = f32_to_bf16_rne(w * bf16lo_to_f32(g[c])) |
           (f32_to_bf16_rne(w * bf16hi_to_f32(g[c])) << 16);
  return o;
}

__device__ __forceinline__ void add_products(const u32x4& g, const u32x4& y, float& dot) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    dot = __builtin_fmaf(bf16lo_to_f32(g[c]), bf16lo_to_f32(y[c]), dot);
    dot = __builtin_fmaf(bf16hi_to_f32(g[c]), bf16hi_to_f32(y[c]), dot);
  }
}

// dy does not need y: its stores go out while y's loads are under way (128
// tokens 10.2 -> 9.6 us).  Where dy is y itself, a thread stores only what
// its own earlier load has asked for.
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const u32x4* __restrict__ g, int64_t gs, const u32x4* y, int64_t ys, int64_t cap,
    const int32_t* __restrict__ ids, const int32_t* __restrict__ idx,
    const int32_t* __restrict__ send, const float* scales, int32_t nvec, int32_t k,
    int32_t E, u32x4* dy, int64_t dys, float* dw, int32_t* status) {
  constexpr int UNROLL = 4;
  __shared__ int send_lds[StagedSend<kThreads>::kSlots];
  __shared__ float sum_lds[kThreads / kWave];
  // Workgroups i, i + 8, ... share an XCD's L2: the pairs of a token go to
  // one of them, which then fetches g's row once.
  int32_t pair = blockIdx.x;
  const int32_t set = 8 * k, first = pair / set * set, in_set = pair - first;
  if (first + set <= (int32_t)gridDim.x) pair = first + in_set % 8 * k + in_set / 8;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  PairMeta meta;
  fetch_pair_meta(meta, pair, 1, ids, idx, scales);
  StagedSend<kThreads> staged;
  staged.load(send, E + 1);
  // The first of g does not depend on the route.
  const u32x4* gt = g + (int64_t)(pair / k) * gs;
  u32x4 gv[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) gv[u] = gt[min((int)threadIdx.x + u * kThreads, nvec - 1)];
  keep_order();
  staged.store(send_lds);
  __syncthreads();
  int64_t slot[1];
  float w[1];
  resolve_routes<1>(meta, send_lds, nullptr, 1, E, cap, slot, w, status, threadIdx.x < kWave);

  float dot = 0.0f;
  for (int32_t v0 = threadIdx.x; slot[0] >= 0 && v0 < nvec; v0 += kThreads * UNROLL) {
    u32x4 yv[UNROLL];
    if (dw) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int32_t v = v0 + u * kThreads;
        if (v < nvec) yv[u] = load_stream(y + slot[0] * ys + v);
      }
    }
    if (dy) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int32_t v = v0 + u * kThreads;
        if (v < nvec) store_stream(scaled(gv[u], w[0]), dy + slot[0] * dys + v);
      }
    }
    if (dw) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u)
        if (v0 + u * kThreads < nvec) add_products(gv[u], yv[u], dot);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      gv[u] = gt[min(v0 + (UNROLL + u) * kThreads, nvec - 1)];
  }
  if (!dw) return;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) dot += __shfl_xor(dot, d, kWave);
  if (lane == 0) sum_lds[wave] = dot;
  __syncthreads();
  if (threadIdx.x == 0) dw[pair] = sum_lds[0] + sum_lds[1];
}

// Short rows: GROUP lanes take a pair, VECS 16-byte vectors a lane, and each
// of them PAIRS pairs, so that a wave has many rows in flight.  (Here stores
// before the products measure the same or slower.)
template <int GROUP, int VECS, int PAIRS>
__global__ __launch_bounds__(kShortThreads) void combine_backward_short_kernel(
    const u32x4* __restrict__ g, int64_t gs, const u32x4* y, int64_t ys, int64_t cap,
    const int32_t* __restrict__ ids, const int32_t* __restrict__ idx,
    const int32_t* __restrict__ send, const float* scales, int32_t nvec, int32_t k,
    int32_t pairs, int32_t E, u32x4* dy, int64_t dys, float* dw, int32_t* status) {
  constexpr int kGroups = kShortThreads / GROUP;
  const int lane = threadIdx.x % GROUP;
  const int32_t first = blockIdx.x * (kGroups * PAIRS) + threadIdx.x / GROUP;
  int32_t e[PAIRS], r[PAIRS];
  float w[PAIRS];
#pragma unroll
  for (int u = 0; u < PAIRS; ++u) {
    const int32_t at = min(first + u * kGroups, pairs - 1);
    e[u] = ids[at];
    r[u] = idx[at];
    w[u] = dy ? scales[at] : 0.0f;
  }
  int64_t slot[PAIRS];
#pragma unroll
  for (int u = 0; u < PAIRS; ++u) {
    slot[u] = -1;
    if (first + u * kGroups < pairs && e[u] >= 0 && e[u] < E && r[u] >= 0) {
      const int64_t to = (int64_t)send[e[u]] + r[u];
      if (to >= 0 && to < cap)
        slot[u] = to;
      else if (status && lane == 0)
        atomicOr(status, (int)MOE_FLAG_GUARD);
    }
  }
  u32x4 gv[PAIRS][VECS], yv[PAIRS][VECS];
#pragma unroll
  for (int u = 0; u < PAIRS; ++u) {
    if (slot[u] < 0) continue;
    const u32x4* gt = g + (int64_t)((first + u * kGroups) / k) * gs;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int v = lane + i * GROUP;
      if (v >= nvec) continue;
      gv[u][i] = gt[v];
      if (dw) yv[u][i] = load_stream(y + slot[u] * ys + v);
    }
  }
#pragma unroll
  for (int u = 0; u < PAIRS; ++u) {
    float dot = 0.0f;
    if (slot[u] >= 0) {
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        const int v = lane + i * GROUP;
        if (v >= nvec) continue;
        if (dw) add_products(gv[u][i], yv[u][i], dot);
        if (dy) store_stream(scaled(gv[u][i], w[u]), dy + slot[u] * dys + v);
      }
    }
    if (!dw) continue;
#pragma unroll
    for (int d = 1; d < GROUP; d <<= 1) dot += __shfl_xor(dot, d, kWave);
    if (lane == 0 && first + u * kGroups < pairs) dw[first + u * kGroups] = dot;
  }
}

}  // namespace

hipError_t launch_combine_backward(const void* grad_out, int64_t grad_stride, const void* y,
                                   int64_t y_stride, int64_t capacity_rows, const int32_t* ids,
                                   const int32_t* expand_idx, const int32_t* send,
                                   const float* scales, int32_t bs, int32_t hidden, int32_t k,
                                   int32_t num_experts, void* grad_y, int64_t grad_y_stride,
                                   float* grad_scales, int32_t* status, hipStream_t stream) {
  const int32_t most = kMostPairs / k;  // tokens a launch
  if (bs > most) {
    for (int32_t t = 0; t < bs; t += most) {
      const int64_t p = (int64_t)t * k;
      const hipError_t err = launch_combine_backward(
          static_cast<const uint16_t*>(grad_out) + t * grad_stride, grad_stride, y, y_stride,
          capacity_rows, ids + p, expand_idx + p, send, scales ? scales + p : nullptr,
          bs - t < most ? bs - t : most, hidden, k, num_experts, grad_y, grad_y_stride,
          grad_scales ? grad_scales + p : nullptr, status, stream);
      if (err != hipSuccess) return err;
    }
    return hipSuccess;
  }
  const u32x4* gv = static_cast<const u32x4*>(grad_out);
  const u32x4* yv = static_cast<const u32x4*>(y);
  u32x4* dv = static_cast<u32x4*>(grad_y);
  const int32_t nvec = hidden / 8, pairs = bs * k;
  const bool few = pairs <= kFewPairs;
#define MOE_SHORT(GROUP, VECS, PAIRS)                                                         \
  launch_kernel(combine_backward_short_kernel<GROUP, VECS, PAIRS>,                            \
                dim3((uint32_t)(((int64_t)pairs * GROUP + kShortThreads * PAIRS - 1) /         \
                                (kShortThreads * PAIRS))),                                    \
                kShortThreads, stream, gv, grad_stride / 8, yv, y_stride / 8, capacity_rows,  \
                ids, expand_idx, send, scales, nvec, k, pairs, num_experts, dv,               \
                grad_y_stride / 8, grad_scales, status)
  // Times in us, a workgroup a pair against groups of lanes: 3200 pairs of 64
  // channels 5.3 and 3.6, of 512 6.2 and 4.6, of 1024 7.2 and 6.0, of 2048 9.8
  // and 10.4; 32768 pairs of 64 27 and 5.0, of 512 33 and 16.5, of 1024 43 and
  // 31.5, of 2048 60 and 58, of 4096 109 and 115.  Two pairs a group against
  // one: 32768 pairs of 512 16.5 and 21, of 1024 31.5 and 33.5; 3200 pairs 6.2
  // and 4.6, 6.9 and 6.0.
  if (nvec <= 8)
    MOE_SHORT(8, 1, 1);
  else if (nvec <= 16)
    MOE_SHORT(16, 1, 1);
  else if (nvec <= 32)
    MOE_SHORT(32, 1, 1);
  else if (nvec <= 64 && few)
    MOE_SHORT(64, 1, 1);
  else if (nvec <= 64)
    MOE_SHORT(32, 2, 2);
  else if (nvec <= 128 && few)
    MOE_SHORT(64, 2, 1);
  else if (nvec <= 128)
    MOE_SHORT(64, 2, 2);
  else if (nvec <= 256 && !few)
    MOE_SHORT(64, 4, 2);
  else
    launch_kernel(combine_backward_kernel, dim3((uint32_t)pairs), kThreads, stream, gv,
                  grad_stride / 8, yv, y_stride / 8, capacity_rows, ids, expand_idx, send,
                  scales, nvec, k, num_experts, dv, grad_y_stride / 8, grad_scales, status);
#undef MOE_SHORT
  return hipGetLastError();
}

}  // namespace moe
