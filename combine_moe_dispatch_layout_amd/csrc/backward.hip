// backward.hip -- the gradient of the combine.  With
//   out[t] = sum_j w[t, j] * y[slot(t, j)] + shared[t]   and   g = dL/dout:
//   dy[slot(t, j)] = w[t, j] * g[t]        (rounded once to bf16)
//   dw[t, j]       = <g[t], y[slot(t, j)]> (fp32)
// and the shared row's gradient is g itself.  The scatter's gradient is the
// combine's gather-sum with unit weights (combine.hip).
//
// A workgroup takes one pair (KMAX 1, `share` = K) or one token: each row of
// y is read once and each row of dy written once.  Per pair each workgroup
// has one row in and one row out, and a token's pairs run on one XCD, whose
// L2 gives them g; per token g is read once and the route's set-up is paid
// once for K rows.  HBM bounds both: 4096 tokens of 7168 channels, K = 8, take
// 180 us per pair (1.0 GB at 5.6 TB/s; a copy of 2 GiB reaches 5.0) and 205
// per token, 128 tokens 9.9 and 27 us; at 1024 channels 4096 tokens take 43
// and 31 us, 512 tokens 7.3 and 8.5.
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
// Rows of at least this many 16-byte vectors, and batches of at most this
// many pairs, go pair by pair (2048 channels: 17.4 against 20.6 us at 1024
// tokens, 215 against 226 at 16384).
constexpr int32_t kPerPairVecs = 256;
constexpr int64_t kPerPairMost = 4096;

// g's rows are read once per token, or K times per pair (then worth caching).
template <bool SHARED>
__device__ __forceinline__ u32x4 load_grad(const u32x4* p) {
  if constexpr (SHARED)
    return *p;
  else
    return load_stream(p);
}

template <int KMAX, int UNROLL>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const u32x4* __restrict__ g, int64_t gs, int32_t share, const u32x4* y, int64_t ys,
    int64_t cap, const int32_t* __restrict__ ids, const int32_t* __restrict__ idx,
    const int32_t* __restrict__ send, const float* __restrict__ scales, int32_t nvec, int32_t k,
    int32_t E, u32x4* dy, int64_t dys, float* __restrict__ dw, int32_t* status) {
  __shared__ int send_lds[StagedSend<kThreads>::kSlots];
  __shared__ float sum_lds[kThreads / kWave][KMAX];
  int32_t t = blockIdx.x;
  if constexpr (KMAX == 1) {
    // Workgroups i, i + 8, ... share an XCD's L2: the pairs of a token go
    // to one of them, which then fetches g's row once.
    const int32_t set = 8 * share, first = t / set * set, in_set = t - first;
    if (first + set <= (int32_t)gridDim.x) t = first + in_set % 8 * share + in_set / 8;
  }
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  PairMeta meta;
  fetch_pair_meta(meta, t, k, ids, idx, scales);
  StagedSend<kThreads> staged;
  staged.load(send, E + 1);
  // The first of g does not depend on the route.
  const u32x4* gt = g + (int64_t)(t / share) * gs;
  u32x4 gv[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const int32_t v = threadIdx.x + u * kThreads;
    gv[u] = load_grad<KMAX == 1>(gt + min(v, nvec - 1));
  }
  keep_order();
  staged.store(send_lds);
  __syncthreads();
  int64_t slot[KMAX];
  float w[KMAX];
  resolve_routes<KMAX>(meta, send_lds, nullptr, k, E, cap, slot, w, status, threadIdx.x < kWave);

  float dot[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) dot[j] = 0.0f;
  for (int32_t v0 = threadIdx.x; v0 < nvec; v0 += kThreads * UNROLL) {
    u32x4 yv[UNROLL][KMAX];
    if (dw) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int32_t v = v0 + u * kThreads;
#pragma unroll
        for (int j = 0; j < KMAX; ++j)
          if (slot[j] >= 0 && v < nvec) yv[u][j] = load_stream(y + slot[j] * ys + v);
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int32_t v = v0 + u * kThreads;
      if (v >= nvec) continue;
      float gf[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        gf[2 * c] = bf16lo_to_f32(gv[u][c]);
        gf[2 * c + 1] = bf16hi_to_f32(gv[u][c]);
      }
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        if (slot[j] < 0) continue;
        if (dw) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            dot[j] = __builtin_fmaf(gf[2 * c], bf16lo_to_f32(yv[u][j][c]), dot[j]);
            dot[j] = __builtin_fmaf(gf[2 * c + 1], bf16hi_to_f32(yv[u][j][c]), dot[j]);
          }
        }
        if (dy) {
          u32x4 o;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            o[c] = f32_to_bf16_rne(w[j] * gf[2 * c]) |
                   (f32_to_bf16_rne(w[j] * gf[2 * c + 1]) << 16);
          store_stream(o, dy + slot[j] * dys + v);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int32_t v = v0 + (UNROLL + u) * kThreads;
      gv[u] = load_grad<KMAX == 1>(gt + min(v, nvec - 1));
    }
  }
  if (!dw) return;
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) dot[j] += __shfl_xor(dot[j], d, kWave);
    if (lane == 0) sum_lds[wave][j] = dot[j];
  }
  __syncthreads();
  if ((int)threadIdx.x < k) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / kWave; ++i) s += sum_lds[i][threadIdx.x];
    dw[(int64_t)t * k + threadIdx.x] = s;
  }
}

}  // namespace

hipError_t launch_combine_backward(const void* grad_out, int64_t grad_stride, const void* y,
                                   int64_t y_stride, int64_t capacity_rows, const int32_t* ids,
                                   const int32_t* expand_idx, const int32_t* send,
                                   const float* scales, int32_t bs, int32_t hidden, int32_t k,
                                   int32_t num_experts, void* grad_y, int64_t grad_y_stride,
                                   float* grad_scales, int32_t* status, hipStream_t stream) {
  const u32x4* gv = static_cast<const u32x4*>(grad_out);
  const u32x4* yv = static_cast<const u32x4*>(y);
  u32x4* dv = static_cast<u32x4*>(grad_y);
  const int32_t nvec = hidden / 8;
#define MOE_COMBINE_BACKWARD(KM, UN, ITEMS, SHARE, KK)                                          \
  launch_kernel(combine_backward_kernel<KM, UN>, dim3((uint32_t)(ITEMS)), kThreads, stream, gv, \
                grad_stride / 8, SHARE, yv, y_stride / 8, capacity_rows, ids, expand_idx, send,  \
                scales, nvec, KK, num_experts, dv, grad_y_stride / 8, grad_scales, status)
  if (nvec >= kPerPairVecs || (int64_t)bs * k <= kPerPairMost)
    MOE_COMBINE_BACKWARD(1, 4, bs * k, k, 1);
  else if (k <= 2)
    MOE_COMBINE_BACKWARD(2, 2, bs, 1, k);
  else if (k <= 4)
    MOE_COMBINE_BACKWARD(4, 1, bs, 1, k);
  else if (k <= 8)
    MOE_COMBINE_BACKWARD(8, 1, bs, 1, k);
  else
    MOE_COMBINE_BACKWARD(16, 1, bs, 1, k);
#undef MOE_COMBINE_BACKWARD
  return hipGetLastError();
}

}  // namespace moe
