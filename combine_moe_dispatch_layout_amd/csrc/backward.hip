// backward.hip -- the gradient of the combine.  With
//   out[t] = sum_j w[t, j] * y[slot(t, j)] + shared[t]   and   g = dL/dout:
//   dy[slot(t, j)] = w[t, j] * g[t]        (rounded once to bf16)
//   dw[t, j]       = <g[t], y[slot(t, j)]> (fp32)
// and the shared row's gradient is g itself.  The scatter's gradient is the
// combine's gather-sum with unit weights (combine.hip).
//
// One workgroup per token: each row of y is read once and each row of dy
// written once, g once for all K pairs.
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 128;

template <int KMAX>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const u32x4* __restrict__ g, int64_t gs, const u32x4* y, int64_t ys, int64_t cap,
    const int32_t* __restrict__ ids, const int32_t* __restrict__ idx,
    const int32_t* __restrict__ send, const float* __restrict__ scales, int32_t nvec, int32_t k,
    int32_t E, u32x4* dy, int64_t dys, float* __restrict__ dw, int32_t* status) {
  __shared__ int send_lds[StagedSend<kThreads>::kSlots];
  __shared__ float sum_lds[kThreads / kWave][KMAX];
  const int32_t t = blockIdx.x;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  PairMeta meta;
  fetch_pair_meta(meta, t, k, ids, idx, scales);
  StagedSend<kThreads> staged;
  staged.load(send, E + 1);
  staged.store(send_lds);
  __syncthreads();
  int64_t slot[KMAX];
  float w[KMAX];
  resolve_routes<KMAX>(meta, send_lds, nullptr, k, E, cap, slot, w, status, threadIdx.x < kWave);

  float dot[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) dot[j] = 0.0f;
  for (int32_t v = threadIdx.x; v < nvec; v += kThreads) {
    const u32x4 gv = load_stream(g + (int64_t)t * gs + v);
    u32x4 yv[KMAX];
    if (dw) {
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (slot[j] >= 0) yv[j] = load_stream(y + slot[j] * ys + v);
    }
    float gf[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      gf[2 * c] = bf16lo_to_f32(gv[c]);
      gf[2 * c + 1] = bf16hi_to_f32(gv[c]);
    }
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      if (slot[j] < 0) continue;
      if (dw) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          dot[j] = __builtin_fmaf(gf[2 * c], bf16lo_to_f32(yv[j][c]), dot[j]);
          dot[j] = __builtin_fmaf(gf[2 * c + 1], bf16hi_to_f32(yv[j][c]), dot[j]);
        }
      }
      if (dy) {
        u32x4 o;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          o[c] = f32_to_bf16_rne(w[j] * gf[2 * c]) | (f32_to_bf16_rne(w[j] * gf[2 * c + 1]) << 16);
        store_stream(o, dy + slot[j] * dys + v);
      }
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
  const dim3 grid((uint32_t)bs);
#define MOE_COMBINE_BACKWARD(KM)                                                             \
  launch_kernel(combine_backward_kernel<KM>, grid, kThreads, stream, gv, grad_stride / 8, yv, \
                y_stride / 8, capacity_rows, ids, expand_idx, send, scales, hidden / 8, k,    \
                num_experts, dv, grad_y_stride / 8, grad_scales, status)
  if (k <= 2)
    MOE_COMBINE_BACKWARD(2);
  else if (k <= 4)
    MOE_COMBINE_BACKWARD(4);
  else if (k <= 8)
    MOE_COMBINE_BACKWARD(8);
  else
    MOE_COMBINE_BACKWARD(16);
#undef MOE_COMBINE_BACKWARD
  return hipGetLastError();
}

}  // namespace moe
