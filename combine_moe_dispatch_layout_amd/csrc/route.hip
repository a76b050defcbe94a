// route.hip -- routing of tokens to experts, and its gradient.  From a row of
// logits l over E experts, with scores s (softmax(l), or 1 / (1 + e^-l)):
//   key_e = l_e, or s_e + bias_e with a bias
//   of `groups` groups of neighbouring experts the best `top_groups` stay
//     (by their largest key, or by the sum of their two largest s + bias)
//   ids   = the k largest keys, ties to the lowest expert
//   w_j   = scale * s_j, or scale * s_j / sum of the chosen s
// The gradient of the weights with respect to the logits, q = w / scale and
// G = sum_j g_j q_j (the choice itself has none):
//   softmax:                 scale * p_e (g_e - G) over all experts
//   softmax, renormalised:   scale * q_j (g_j - G) at the chosen
//   sigmoid:                 scale * s_j (1 - s_j) g_j at the chosen
//   sigmoid, renormalised:   scale * q_j (1 - s_j) (g_j - G) at the chosen
//
// A row of E <= 512 values is a few instructions a lane; what counts is how few.
// LANES lanes take a row (16 in large batches, so that a wave has four rows and
// an exchange between lanes is one instruction; the whole wave in small ones).
// An expert's key becomes its distance below the row's largest key in 23 bits,
// with its index in the 9 bits below: one number whose minimum is the best
// expert, the lowest index among equals.  Each lane sorts its 4 best, and k
// rounds take the minimum over the lanes' first ones.
//
// Measured: 16384 rows of 512 logits, softmax, best 8, 9.1 us in a graph (33 MB, 3.6
// TB/s).  Instructions bound it: a wave's four rows take 829 vector ones, which of 4
// waves a SIMD at 4 cycles each are 5.5 us, beside a launch's 2.2 and the loads that
// come first.  128 rows of 256 with a bias and 8 groups 5.1; the gradient of 16384 rows
// of 512 13.6 (5.0 TB/s), of 777 of 60 3.3.
//
// Where neighbours in that order are nearer to each other than the numbers can
// tell (23 bits, and the rounding of fp32 scores), the candidates are compared
// in 64 bits; where that does not settle it, or groups are too near, the row is
// done again in 64 bits by the whole wave (15183 rows of 25, softmax with a bias,
// 12.1 us with all of those by the whole wave, 9.5 so).
#include "lanes.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kIndexBits = 9;                 // kMaxExperts
constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr int kFirst = 4;                     // best experts a lane keeps in order
constexpr float kFltMax = 3.40282347e38f;
// By how much two keys have to differ for their order to be sure: twice the
// error of one.  A sigmoid's is the exponential's (2e-7 of it), an addition's
// and a reciprocal's: 3.8e-7 at most.  A softmax's score is off by 1.4e-6 of
// itself (13 additions of the sum, two exponentials, a division and a product), so
// by that share of the largest score.  An addition of the bias rounds once more.
constexpr float kSigmoidError = 8e-7f;
constexpr float kSoftmaxError = 2.8e-6f;
constexpr float kSumError = 1.3e-7f;
// A group's score of two keys is off by both's errors, and by roundings at the
// size of the keys, not of their sum, which may cancel: 2^-24 of |one| + |two| for
// the keys', the sum's, and that of taking this error off.
constexpr float kGroupError = 2e-7f;
// A sum of such exponentials: their 2.4e-7, and the rounding of each argument, whose
// size is at most log E = 6.3 where averaged by the terms' shares.
constexpr double kShareError = 7e-7;

// e^x to about 2 ulp for any x that is not NaN.
__device__ __forceinline__ float exp_f32(float x) {
  x = __builtin_amdgcn_fmed3f(x, -1000.0f, 1000.0f);
  const float n = __builtin_rintf(x * 1.44269504088896341f);
  const float f =
      __builtin_fmaf(x, 1.9259629911e-8f, __builtin_fmaf(x, 1.44269502162933349609f, -n));
  return __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}

// The k chosen experts' scores are made in 64 bits, and weights and gradients
// rounded once: one value a lane, little beside the choice (us, in 32 bits and so:
// 16384 x 512 softmax 9.1, 9.1, its gradient with sigmoid 13.4, 13.6; 777 x 60's
// gradient 3.2, 3.3; weights' error 5.5e-8, 2.5e-8).  A sum over all experts is one
// of fp32 exponentials: the gradient through it takes 18.4 for 16384 x 512 as it is.
//
// e^x to 2^-32 of itself: x = n log 2 + r, and r's Taylor series to its 8th power
// (|r| <= 0.347, so what is left out is below 0.347^9 / 9! = 2e-10).
__device__ __forceinline__ double exp_f64(double x) {
  x = fmin(fmax(x, -700.0), 700.0);  // past what an fp32 result can tell
  const double n = __builtin_rint(x * 1.4426950408889634074);
  const double r = __builtin_fma(n, -0.69314718055994530942, x);
  double e = 1.0 / 40320;
  e = __builtin_fma(e, r, 1.0 / 5040);
  e = __builtin_fma(e, r, 1.0 / 720);
  e = __builtin_fma(e, r, 1.0 / 120);
  e = __builtin_fma(e, r, 1.0 / 24);
  e = __builtin_fma(e, r, 1.0 / 6);
  e = __builtin_fma(e, r, 0.5);
  e = __builtin_fma(e, r, 1.0);
  e = __builtin_fma(e, r, 1.0);
  return __builtin_ldexp(e, (int)n);
}

// 1 / x, x a normal number: the reciprocal instruction's (off by 2^-24 of itself,
// measured), whose error a step of Newton's squares.
__device__ __forceinline__ double inverse(double x) {
  const double y = __builtin_amdgcn_rcp(x);
  return __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
}

// A logit as it counts: a NaN or -inf masks the expert, +inf is the largest
// finite value.
__device__ __forceinline__ float counted(float l) {
  return fminf(fmaxf(l, -__builtin_inff()), kFltMax);
}

template <bool BF16>
__device__ __forceinline__ float read_logit(const RouteArgs& a, int64_t at) {
  return BF16 ? bf16lo_to_f32(static_cast<const uint16_t*>(a.logits)[at])
              : static_cast<const float*>(a.logits)[at];
}

template <bool BF16>
__device__ __forceinline__ float logit_at(const RouteArgs& a, int64_t row, int e) {
  return counted(read_logit<BF16>(a, row * a.logits_stride + e));
}

// A row's logits, expert lane + i * LANES at i; -inf past the last.  No load
// waits for a condition.
template <int LANES, int PER, bool BF16>
__device__ __forceinline__ void read_row(const RouteArgs& a, int64_t row, int lane,
                                         float (&l)[PER]) {
  const int64_t at = row * a.logits_stride;
  if (a.num_experts == LANES * PER) {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = read_logit<BF16>(a, at + lane + i * LANES);
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = counted(l[i]);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      l[i] = read_logit<BF16>(a, at + min(lane + i * LANES, a.num_experts - 1));
#pragma unroll
    for (int i = 0; i < PER; ++i)
      l[i] = lane + i * LANES < a.num_experts ? counted(l[i]) : -__builtin_inff();
  }
}

// The experts' bias, laid out alike; 0 without one.
template <int LANES, int PER>
__device__ __forceinline__ void read_bias(const RouteArgs& a, int lane, float (&b)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) b[i] = 0.0f;
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < PER; ++i) b[i] = a.bias[min(lane + i * LANES, a.num_experts - 1)];
  }
}

// A row's sum: few additions in turn round in 32 bits (kSoftmaxError), and
// independently in each of four parts of a lane; the parts are added in 64.
template <int LANES, int PER>
__device__ __forceinline__ double row_sum(const float (&v)[PER]) {
  float four[4] = {};
#pragma unroll
  for (int i = 0; i < PER; ++i) four[i % 4] += v[i];
  return over_row<LANES, Sum>(((double)four[0] + four[1]) + ((double)four[2] + four[3]));
}

__device__ __forceinline__ bool masked(float l) { return l == -__builtin_inff(); }

// The chosen experts' weights (before the scaling): lane j of the row holds the
// logit of the j-th (k <= 16: in the row's first 16 lanes).  Softmax without
// renormalisation needs the row's largest logit and the sum of its exponentials.
__device__ __forceinline__ double weight_of(const RouteArgs& a, float l, bool real, float top,
                                            double sum) {
  if (!a.renormalize) {
    if (!real) return 0.0;
    return a.sigmoid ? inverse(1.0 + exp_f64(-(double)l))
                     : exp_f64((double)l - top) * inverse(sum);
  }
  const float most = over_row<16, Max>(real ? l : -__builtin_inff());
  double t = 0.0;
  if (real) {
    if (a.sigmoid) {
      // Scores times e^-c, so that the largest is at least 1/2.
      const double c = fminf(most, 0.0f);
      t = inverse(exp_f64(c) + exp_f64(c - l));
    } else {
      t = exp_f64((double)l - most);
    }
  }
  const double total = over_row<16, Sum>(t);
  return real ? t * inverse(total) : 0.0;
}

template <int LANES>
__device__ __forceinline__ void write_choice(const RouteArgs& a, int64_t row, int lane, int id,
                                             float l, float top, double sum) {
  const double w = a.scale * weight_of(a, l, id >= 0, top, sum);
  if (lane < a.k) {
    a.ids[row * a.k + lane] = id;
    a.scales[row * a.k + lane] = (float)w;
  }
}

// ---- a row in 64 bits, by the whole wave --------------------------------------------
// Rarely run, so what it takes is mostly the fetching of its code: short loops
// over keys in shared memory (unrolled, it took 5 us more).
constexpr int kWavePer = kMaxExperts / kWave;

template <bool BF16>
__device__ __forceinline__ void route_exactly(const RouteArgs& a, int64_t row, double* keys) {
  const int lane = threadIdx.x & (kWave - 1);
  const double inf = __builtin_inf();
  const int rounds = (a.num_experts + kWave - 1) / kWave;
  const bool by_score = a.bias || (a.groups > 1 && a.by_two);
  float l[kWavePer], bias[kWavePer], top = -__builtin_inff();
  read_row<kWave, kWavePer, BF16>(a, row, lane, l);
  read_bias<kWave, kWavePer>(a, lane, bias);
#pragma unroll
  for (int i = 0; i < kWavePer; ++i) top = fmaxf(top, l[i]);
  top = over_row<kWave, Max>(top);
  // A lane's own places of `keys`, until the groups are looked at.
  if (by_score) {
#pragma unroll
    for (int i = 0; i < kWavePer; ++i) keys[lane + i * kWave] = l[i];
    const double shift = a.sigmoid || masked(top) ? 0.0 : (double)top;
    const double sign = a.sigmoid ? -1.0 : 1.0;
    double total = 0.0;
#pragma unroll 1
    for (int i = 0; i < rounds; ++i) {
      const double v = exp(sign * (keys[lane + i * kWave] - shift));
      keys[lane + i * kWave] = v;
      total += v;
    }
    total = over_row<kWave, Sum>(total);
#pragma unroll 1
    for (int i = 0; i < rounds; ++i) {
      const double v = keys[lane + i * kWave];
      keys[lane + i * kWave] = a.sigmoid ? 1.0 / (1.0 + v) : v / total;
    }
  }
  double key[kWavePer];
#pragma unroll
  for (int i = 0; i < kWavePer; ++i) {
    const double v = by_score ? keys[lane + i * kWave] + bias[i] : l[i];
    key[i] = masked(l[i]) || !(v > -inf) ? -inf : v;
  }
  if (a.groups > 1) {
#pragma unroll
    for (int i = 0; i < kWavePer; ++i) keys[lane + i * kWave] = key[i];
    __builtin_amdgcn_wave_barrier();
    keep_order();
    const int size = a.num_experts / a.groups;
    double of = -inf;
    if (lane < a.groups) {
      double one = -inf, two = -inf;
#pragma unroll 4
      for (int i = 0; i < size; ++i) {
        const double v = keys[lane * size + i];
        two = v > one ? one : (v > two ? v : two);
        one = v > one ? v : one;
      }
      of = a.by_two && two > -inf ? one + two : one;
    }
    uint64_t kept = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      const double best = over_row<kWave, Max>(of);
      if (!(best > -inf)) break;
      const int g = __builtin_ctzll(__ballot(of == best));
      kept |= uint64_t(1) << g;
      if (lane == g) of = -inf;
    }
#pragma unroll
    for (int i = 0; i < kWavePer; ++i) {
      const int e = lane + i * kWave;
      if (e >= a.num_experts || !(kept >> (e / size) & 1))
        key[i] = -inf;
      else if (by_score && !a.bias && key[i] > -inf)
        key[i] = l[i];
    }
    keep_order();
  }
  int id = -1;
  float chosen = 0.0f;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    double best = -inf;
#pragma unroll
    for (int i = 0; i < kWavePer; ++i) best = key[i] > best ? key[i] : best;
    best = over_row<kWave, Max>(best);
    if (!(best > -inf)) break;
    int e = kMaxExperts;  // the lowest that has it
    float of = 0.0f;
#pragma unroll
    for (int i = kWavePer - 1; i >= 0; --i) {
      const uint64_t has = __ballot(key[i] == best);
      if (has) {
        e = __builtin_ctzll(has) + i * kWave;
        of = of_lane(l[i], e & (kWave - 1));
      }
    }
#pragma unroll
    for (int i = 0; i < kWavePer; ++i)
      if (lane + i * kWave == e) key[i] = -inf;
    if (lane == j) {
      id = e;
      chosen = of;
    }
  }
  double sum = 1.0;
  if (!a.sigmoid && !a.renormalize) {
    float of[kWavePer];
#pragma unroll
    for (int i = 0; i < kWavePer; ++i) of[i] = exp_f32(l[i] - (masked(top) ? 0.0f : top));
    sum = row_sum<kWave>(of);
  }
  write_choice<kWave>(a, row, lane, id, chosen, top, sum);
}

// ---- the choice ----------------------------------------------------------------------
// A group's two largest keys joined over the lanes that share it.
template <int CTRL>
__device__ __forceinline__ void join_two(float& one, float& two) {
  const float o = dpp<CTRL>(one), t = dpp<CTRL>(two);
  two = fmaxf(fmaxf(two, t), fminf(one, o));
  one = fmaxf(one, o);
}

// A group's score, and by how much it may be off.
struct GroupScore {
  float of, error;
  __device__ __forceinline__ GroupScore(const float2& two, bool by_two, float score_error) {
    const bool both = by_two && two.y > -__builtin_inff();
    of = both ? two.x + two.y : two.x;
    error = score_error + kGroupError * (fabsf(two.x) + (both ? fabsf(two.y) : 0.0f));
  }
  // What it is at least and at most (anything, where the sizes leave fp32).
  __device__ __forceinline__ float low() const {
    return error < __builtin_inff() ? of - error : -__builtin_inff();
  }
  __device__ __forceinline__ float high() const {
    if (of == -__builtin_inff()) return of;  // no expert is left
    return error < __builtin_inff() ? of + error : __builtin_inff();
  }
};

// The groups that stay, of a row whose keys lie in `keys`: bit g << shift for
// group g.  `near`: a group that stays and one that does not are too near to
// tell.
template <int LANES>
__device__ __forceinline__ uint64_t kept_groups(const RouteArgs& a, const float* keys, int lane,
                                                float score_error, int& shift, bool& near) {
  const float inf = __builtin_inff();
  const int size = a.num_experts / a.groups;
  const int first = (threadIdx.x & (kWave - 1)) / LANES * LANES;
  const auto best_two = [&](int g, int part, int step) {
    float one = -inf, two = -inf;
    if (g < a.groups) {
#pragma unroll 4
      for (int i = part; i < size; i += step) {
        const float v = keys[g * size + i];
        two = fmaxf(two, fminf(one, v));
        one = fmaxf(one, v);
      }
    }
    return float2{one, two};
  };
  uint64_t kept = 0;
  float least = inf, most = -inf;
  shift = 0;
  if (a.groups <= LANES) {
    // 1, 2, 4, 8 or 16 neighbouring lanes a group.
    while (shift < 4 && a.groups << (shift + 1) <= LANES) ++shift;
    const int g = lane >> shift;
    const float2 two = best_two(g, lane & ((1 << shift) - 1), 1 << shift);
    float x = two.x, y = two.y;
    if (shift > 0) join_two<0xB1>(x, y);   // quad_perm 1 0 3 2
    if (shift > 1) join_two<0x4E>(x, y);   // quad_perm 2 3 0 1
    if (shift > 2) join_two<0x141>(x, y);  // row_half_mirror
    if (shift > 3) join_two<0x140>(x, y);  // row_mirror
    const GroupScore mine(float2{x, y}, a.by_two, score_error);
    const float of = mine.of;
    int rank = 0;
    for (int j = 0; j < a.groups; ++j) {
      const float o = LANES == kWave ? of_lane(of, j << shift) : __shfl(of, j << shift, LANES);
      rank += o > of || (o == of && j < g);
    }
    const bool stays = g < a.groups && rank < a.top_groups && of > -inf;
    kept = __ballot(stays) >> first;
    if (stays) least = mine.low();
    if (g < a.groups && !stays) most = mine.high();
  } else {  // more groups than lanes: several a lane
    constexpr int kRounds = kMaxGroups / LANES;
    float of[kRounds], low[kRounds], high[kRounds];
    int rank[kRounds] = {};
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const GroupScore mine(best_two(lane + r * LANES, 0, 1), a.by_two, score_error);
      of[r] = mine.of;
      low[r] = mine.low();
      high[r] = mine.high();
    }
#pragma unroll
    for (int q = 0; q < kRounds; ++q)
#pragma unroll 1
      for (int j = 0; j < LANES && j + q * LANES < a.groups; ++j) {
        const float o = __shfl(of[q], j, LANES);
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
          rank[r] += o > of[r] || (o == of[r] && j + q * LANES < lane + r * LANES);
      }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const bool stays = rank[r] < a.top_groups && of[r] > -inf;
      uint64_t bits = __ballot(stays) >> first;
      if (LANES < kWave) bits &= (uint64_t(1) << (LANES % kWave)) - 1;
      kept |= bits << (r * LANES % 64);
      if (stays)
        least = fminf(least, low[r]);
      else
        most = fmaxf(most, high[r]);
    }
  }
  least = over_row<LANES, Min>(least);
  most = over_row<LANES, Max>(most);
  near = score_error > 0.0f && most > -inf && !(least > most);
  return kept;
}

// PLAIN: no bias and no groups, experts are ranked by their logits alone.
template <int LANES, int PER, bool BF16, bool PLAIN>
__global__ __launch_bounds__(kThreads, 4) void route_kernel(const RouteArgs a) {
  constexpr int kRowsAWave = kWave / LANES;
  constexpr int kRows = kWaves * kRowsAWave;
  constexpr int kKeep = PER < kFirst ? PER : kFirst;
  __shared__ union {  // a wave's own
    float row[PLAIN ? 1 : kRowsAWave][PLAIN ? 1 : LANES * PER];
    double wave[kMaxExperts];
  } keys[kWaves];
  const float inf = __builtin_inff();
  const int in_wave = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int lane = in_wave % LANES, slot = threadIdx.x / LANES;
  const bool grouped = !PLAIN && a.groups > 1;
  const bool two_keys = grouped && a.by_two && !a.bias;  // groups by scores, experts by logits
  const bool by_score = !PLAIN && (a.bias || two_keys);
  const bool exact = PLAIN || !a.bias;                   // experts ranked by logits
  const bool sums = !a.sigmoid && (by_score || !a.renormalize);
  // Rows past the end repeat the last one.
  const int32_t row = min((int32_t)blockIdx.x * kRows + slot, a.bs - 1);
  float key[PER], top = -inf;
  read_row<LANES, PER, BF16>(a, row, lane, key);
  float bias[PLAIN ? 1 : PER];
  if constexpr (!PLAIN) read_bias<LANES, PER>(a, lane, bias);
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, key[i]);
  float most = top;  // of the lane
  top = over_row<LANES, Max>(top);
  double sum = 1.0;
  if (sums) {
    float of[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) of[i] = exp_f32(key[i] - (masked(top) ? 0.0f : top));
    sum = row_sum<LANES>(of);
  }
  bool near = false;
  float score_error = 0.0f;
  if (!PLAIN) {
    float l[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = key[i];
    if (by_score) {
      const float by = 1.0f / (float)sum;
      score_error = a.sigmoid ? kSigmoidError : kSoftmaxError * by;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float s = (a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + exp_f32(-l[i]))
                                   : exp_f32(l[i] - top) * by) + bias[i];
        key[i] = masked(l[i]) || !(s > -inf) ? -inf : s;
      }
    }
    if (grouped) {
      float* mine = keys[wave].row[in_wave / LANES];
#pragma unroll
      for (int i = 0; i < PER; ++i) mine[lane + i * LANES] = key[i];
      __builtin_amdgcn_wave_barrier();
      keep_order();
      int shift;
      const uint64_t kept = kept_groups<LANES>(a, mine, lane, score_error, shift, near);
      keep_order();
      // e / size for e < 512.
      const uint32_t size = a.num_experts / a.groups;
      const uint32_t inverse = ((1u << 20) + size - 1) / size;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const uint32_t e = lane + i * LANES;
        const bool stays = kept >> ((e * inverse >> 20) << shift & 63) & 1;
        key[i] = stays ? (two_keys ? l[i] : key[i]) : -inf;
      }
    }
    most = -inf;
#pragma unroll
    for (int i = 0; i < PER; ++i) most = fmaxf(most, key[i]);
  }
  // Distances below the largest key, in the unit that spreads the lanes' own
  // largest over 22 bits: the k best are not below all of those (where lanes
  // are empty they may be, and share the last unit).
  const float least = over_row<LANES, Min>(masked(most) ? inf : most);
  most = over_row<LANES, Max>(most);
  const float range = __builtin_amdgcn_fmed3f(most - least, 1e-20f, 1e20f);
  const float unit = __builtin_ldexpf(1.0f, 31 - kIndexBits - __builtin_amdgcn_frexp_expf(range));
  const float from = most * unit;
  constexpr float kMost = (float)((1 << (32 - kIndexBits)) - 2);
  uint32_t x[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float d = fminf(__builtin_fmaf(-key[i], unit, from), kMost);
    x[i] = masked(key[i]) ? kNone : (uint32_t)d << kIndexBits | (uint32_t)(lane + i * LANES);
  }
  uint32_t best[kKeep];
#pragma unroll
  for (int c = 0; c < kKeep; ++c) best[c] = kNone;
  const auto sort_in = [&](uint32_t v) {
#pragma unroll
    for (int c = 0; c < kKeep; ++c) {
      const uint32_t low = min(best[c], v);
      v = max(best[c], v);
      best[c] = low;
    }
  };
#pragma unroll
  for (int i = 0; i < PER; ++i) sort_in(x[i]);
  // Units by which neighbours have to differ: logits are exact, and equal
  // units then mean a look at the logits.
  const float error = (score_error + kSumError * fabsf(most)) * unit;
  const uint32_t apart = exact ? 1u : 2u + (uint32_t)fminf(error, kMost);
  uint32_t mine = kNone, last = kNone;
  int taken = 0;
  // Takes the row's best of those left to lane j, where `take`.
  const auto take_best = [&](int j, bool take) {
    if (PER > kKeep && __ballot(taken == kKeep)) {  // a lane has given all it had sorted
#pragma unroll
      for (int c = 0; c < kKeep; ++c) best[c] = kNone;
#pragma unroll
      for (int i = 0; i < PER; ++i) sort_in(x[i] > last ? x[i] : kNone);
      taken = 0;
    }
    const uint32_t x0 = over_row<LANES, Min>(best[0]);
    if (!take) return;
    last = x0;
    if (lane == j) mine = x0;
    if (best[0] == x0 && x0 != kNone) {
#pragma unroll
      for (int c = 0; c + 1 < kKeep; ++c) best[c] = best[c + 1];
      best[kKeep - 1] = kNone;
      ++taken;
    }
  };
  // Whether the best of those left is too near to the last one taken.  (A lane
  // that has given all it had sorted has others.)
  const auto next_is_near = [&] {
    uint32_t out = best[0];
    if (PER > kKeep && __ballot(taken == kKeep)) {
      out = kNone;
#pragma unroll
      for (int i = 0; i < PER; ++i) out = min(out, x[i] > last ? x[i] : kNone);
    }
    out = over_row<LANES, Min>(out);
    return out != kNone && (out >> kIndexBits) - (last >> kIndexBits) < apart;
  };
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) take_best(j, true);
  bool level = next_is_near();
  // Whether a lane's expert is too near to the one before it (row_shr 1 within
  // 16 lanes, which hold all k).
  const uint32_t before = dpp<0x111>(mine);
  const bool close = lane > 0 && lane < a.k && mine != kNone &&
                     (mine >> kIndexBits) - (before >> kIndexBits) < apart;

  int id = mine == kNone ? -1 : (int)(mine & (kMaxExperts - 1));
  float chosen = id >= 0 ? logit_at<BF16>(a, row, id) : 0.0f;
  if (exact) {
    // Equal units are in order if their logits are: none below the one before
    // it, and of those left out none above the last.
    const float before_l = dpp<0x111>(chosen);
    near = near || over_row<LANES, Max>((int)(close && before_l < chosen));
    if (__ballot(level)) {
      const float end = __shfl(chosen, a.k - 1, LANES);
      bool above = false;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (x[i] > last && x[i] >> kIndexBits == last >> kIndexBits)
          above = above || logit_at<BF16>(a, row, lane + i * LANES) > end;
      near = near || (level && over_row<LANES, Max>((int)above));
    }
  } else {
    const bool unsure = level || over_row<LANES, Max>((int)close);
    if (__ballot(unsure && !near)) {
      // On past the k-th as long as neighbours are too near (then those taken are
      // the best ones in any case), and what was taken is put in its order by keys
      // in 64 bits (1 us; all of the row's take 7).
      int j = a.k;
      for (; j < kMaxTopK && __ballot(level); ++j) {
        take_best(j, level);
        level = next_is_near() && level;
      }
      near = near || level;
      if (mine != kNone && lane >= a.k) {
        id = (int)(mine & (kMaxExperts - 1));
        chosen = logit_at<BF16>(a, row, id);
      }
      // A softmax's sum is one of fp32 exponentials (off by kShareError of itself,
      // no addition rounds), which shifts two keys by that share of the difference
      // of their scores.
      double total = 1.0;
      if (!a.sigmoid) {
        constexpr int kChunk = PER < 8 ? PER : 8;  // loads under way
        total = 0.0;
#pragma unroll 1
        for (int i0 = 0; i0 < PER; i0 += kChunk) {
          float l[kChunk];
#pragma unroll
          for (int i = 0; i < kChunk; ++i)
            l[i] = logit_at<BF16>(a, row, min(lane + (i0 + i) * LANES, a.num_experts - 1));
#pragma unroll
          for (int i = 0; i < kChunk; ++i)
            if (lane + (i0 + i) * LANES < a.num_experts) total += exp_f32(l[i] - top);
        }
        total = over_row<LANES, Sum>(total);
      }
      const double score = id < 0       ? 0.0
                           : a.sigmoid ? 1.0 / (1.0 + exp(-(double)chosen))
                                       : exp((double)chosen - top) / total;
      const double key64 = id >= 0 ? score + a.bias[id] : -__builtin_inf();
      int place = 0;
#pragma unroll 4
      for (int i = 0; i < kMaxTopK; ++i) {
        const double o = __shfl(key64, i, LANES);
        const int o_id = __shfl(id, i, LANES);
        place += o > key64 || (o == key64 && o_id < id);
      }
      if (!a.sigmoid) {
        bool doubtful = false;
#pragma unroll 4
        for (int i = 0; i < kMaxTopK; ++i) {
          const double apart64 = fabs(__shfl(key64, i, LANES) - key64);
          const double scores = fabs(__shfl(score, i, LANES) - score);
          doubtful = doubtful || (scores > 0.0 && apart64 <= kShareError * scores);
        }
        near = near || (unsure && over_row<LANES, Max>((int)doubtful));
      }
      if (id < 0 || lane >= kMaxTopK || !unsure) place = lane;
      const int to = (in_wave - lane + place) * 4;
      id = __builtin_amdgcn_ds_permute(to, id);
      chosen = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(chosen)));
      if (lane >= a.k) id = -1;
    }
  }
  // A row past the end writes what the last one does, from the same inputs.
  write_choice<LANES>(a, row, lane, id, chosen, top, sum);
  // (Last, with nothing else left in registers.)
  for (uint64_t todo = __ballot(near); todo;) {
    const int at = __builtin_ctzll(todo) / LANES * LANES;  // the row's first lane
    todo &= ~(LANES == kWave ? ~uint64_t(0) : ((uint64_t(1) << (LANES % kWave)) - 1) << at);
    route_exactly<BF16>(a, __builtin_amdgcn_readlane(row, at), keys[wave].wave);
  }
}

// ---- the gradient ---------------------------------------------------------------------
template <int LANES, int PER, bool BF16>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(RouteArgs a) {
  constexpr int kRows = kThreads / LANES;
  const int lane = threadIdx.x % LANES;
  const bool all = !a.sigmoid && !a.renormalize;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
  if (row >= a.bs) return;
  // Lane j holds the j-th chosen expert; an id out of range or of a masked
  // expert counts as none.
  int id = -1;
  float of = 0.0f, g = 0.0f;
  if (lane < a.k) {
    id = a.ids[row * a.k + lane];
    if (id < 0 || id >= a.num_experts) id = -1;
    if (id >= 0) {
      of = logit_at<BF16>(a, row, id);
      g = a.grad_scales[row * a.k + lane];
      if (masked(of)) id = -1;
    }
  }
  float p[PER], top = -__builtin_inff();
  double sum = 1.0;
  if (all) {
    read_row<LANES, PER, BF16>(a, row, lane, p);
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, p[i]);
    top = over_row<LANES, Max>(top);
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i] = masked(p[i]) ? 0.0f : exp_f32(p[i] - top);
    sum = row_sum<LANES>(p);
  }
  const bool real = id >= 0;
  const double q = weight_of(a, of, real, top, sum);
  const double dot = over_row<16, Sum>(real ? g * q : 0.0);
  float d = 0.0f;
  if (real) {
    double v = a.renormalize ? q * (g - dot) : q * g;
    if (a.sigmoid) v *= inverse(1.0 + exp_f64(of));
    d = (float)(a.scale * v);
  }
  // Of every expert's score; nothing left: no gradient.  (Lane 0's: other lanes
  // past the first 16 have no chosen expert's.)
  const float by =
      sum > 0.0 ? __shfl((float)(a.scale * dot * inverse(sum)), 0, LANES) : 0.0f;
  float v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] = all ? -p[i] * by : 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int at = __shfl(id, j, LANES);
    const float add = __shfl(d, j, LANES);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (at == lane + i * LANES) v[i] += add;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + i * LANES;
    if (e >= a.num_experts) continue;
    const int64_t to = row * a.grad_logits_stride + e;
    if (BF16)
      static_cast<uint16_t*>(a.grad_logits)[to] = (uint16_t)f32_to_bf16_rne(v[i]);
    else
      static_cast<float*>(a.grad_logits)[to] = v[i];
  }
}

// A wave a row, or 16 lanes.  Times in us in a graph, a wave a row against 16
// lanes, top-8: 128 rows of 64 experts 3.4 and 3.0, of 256 3.5 and 3.7; by logits,
// 2048 rows of 512 4.5 and 4.8, 4096 5.9 and 5.0; with a bias, 2048 rows of 512 5.5
// and 7.5, 4096 8.1 and 8.0, 8192 12.2 and 9.7; gradient, 4096 rows of 512 5.8 and
// 6.8, 8192 8.7 and 7.9.
constexpr int32_t kFewExperts = 64;
constexpr int32_t kFewRowsPlain = 2560, kFewRows = 4096, kFewRowsGrad = 6144;

dim3 row_grid(int32_t bs, int lanes) {
  const int32_t rows = kThreads / lanes;
  return dim3((uint32_t)((bs - 1) / rows + 1));
}

// Rows of one launch: larger batches take several.
constexpr int32_t kMostRows = most_items(kThreads);

// Rows [from, from + rows) of a batch.
RouteArgs rows_of(RouteArgs a, int32_t from, int32_t rows) {
  const int64_t elem = a.logits_bf16 ? 2 : 4, pairs = (int64_t)from * a.k;
  a.logits = static_cast<const uint8_t*>(a.logits) + from * a.logits_stride * elem;
  a.ids += pairs;
  if (a.scales) a.scales += pairs;
  if (a.grad_scales) a.grad_scales += pairs;
  if (a.grad_logits)
    a.grad_logits = static_cast<uint8_t*>(a.grad_logits) + from * a.grad_logits_stride * elem;
  a.bs = rows;
  return a;
}

}  // namespace

// KERNEL(LANES, PER, BF16) for the batch's size and the experts' count.
#define MOE_ROUTE_BY_SIZE(KERNEL, BF16, FEW_ROWS)  \
  do {                                             \
    if (a.num_experts <= kFewExperts)              \
      KERNEL(16, 4, BF16);                         \
    else if (a.bs < FEW_ROWS && a.num_experts <= 256) \
      KERNEL(64, 4, BF16);                         \
    else if (a.bs < FEW_ROWS)                      \
      KERNEL(64, 8, BF16);                         \
    else if (a.num_experts <= 128)                 \
      KERNEL(16, 8, BF16);                         \
    else if (a.num_experts <= 256)                 \
      KERNEL(16, 16, BF16);                        \
    else                                           \
      KERNEL(16, 32, BF16);                        \
  } while (0)
#define MOE_ROUTE_PLAIN(LANES, PER, BF16) \
  launch_kernel(route_kernel<LANES, PER, BF16, true>, row_grid(a.bs, LANES), kThreads, stream, a)
#define MOE_ROUTE_ANY(LANES, PER, BF16) \
  launch_kernel(route_kernel<LANES, PER, BF16, false>, row_grid(a.bs, LANES), kThreads, stream, a)
#define MOE_ROUTE_GRAD(LANES, PER, BF16)                                                     \
  launch_kernel(route_backward_kernel<LANES, PER, BF16>, row_grid(a.bs, LANES), kThreads, stream, \
                a)

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  if (a.bs > kMostRows) {
    const hipError_t err = launch_route(rows_of(a, 0, kMostRows), stream);
    return err != hipSuccess ? err : launch_route(rows_of(a, kMostRows, a.bs - kMostRows), stream);
  }
  if (a.bias == nullptr && a.groups == 1) {
    if (a.logits_bf16)
      MOE_ROUTE_BY_SIZE(MOE_ROUTE_PLAIN, true, kFewRowsPlain);
    else
      MOE_ROUTE_BY_SIZE(MOE_ROUTE_PLAIN, false, kFewRowsPlain);
  } else if (a.logits_bf16) {
    MOE_ROUTE_BY_SIZE(MOE_ROUTE_ANY, true, kFewRows);
  } else {
    MOE_ROUTE_BY_SIZE(MOE_ROUTE_ANY, false, kFewRows);
  }
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs& a, hipStream_t stream) {
  if (a.bs > kMostRows) {
    const hipError_t err = launch_route_backward(rows_of(a, 0, kMostRows), stream);
    return err != hipSuccess
               ? err
               : launch_route_backward(rows_of(a, kMostRows, a.bs - kMostRows), stream);
  }
  if (a.logits_bf16)
    MOE_ROUTE_BY_SIZE(MOE_ROUTE_GRAD, true, kFewRowsGrad);
  else
    MOE_ROUTE_BY_SIZE(MOE_ROUTE_GRAD, false, kFewRowsGrad);
  return hipGetLastError();
}

}  // namespace moe
