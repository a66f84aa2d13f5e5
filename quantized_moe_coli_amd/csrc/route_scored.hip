// route_scored.hip -- the router over softmax or sigmoid scores, with a
// selection bias, expert groups scored by their best or their two best
// experts, top-k and renormalised weights (coli_moe_route_scored).
//
// One wave routes one token.  The lanes are shared out to the groups, L =
// 64 / (groups rounded up to a power of two) lanes each, so that a group's
// best scores are found by a reduction over L neighbouring lanes; lane l of
// a group holds its experts l, l + L, ...  The scores are evaluated in
// binary64 and rounded once to binary32, so the order of a sum and the
// approximation of an exponential change a score only where it lies next to a
// border of that rounding (about one in four million), and then by one step.
//
// Bound by instructions, not by memory: a token's exponentials and the k
// rounds of its selection.  Reductions go by DPP moves instead of the LDS
// permutes of __shfl, a round whose best score is unique (a ballot tells)
// needs no reduction of indices, and the exponential is as exact as the
// rounding to binary32 needs.  One token of 256 experts in 8 groups 4.5 us
// (8.0 with __shfl and the library's exp).
#include <cmath>

#include "exp64.hpp"
#include "q8.hpp"

#pragma clang fp contract(off)

namespace coli {
namespace {

constexpr float kOff = -INFINITY;  // score of an expert that cannot be chosen

// The two largest of (b1 >= b2) and the partner's, by one move of the lanes.
template <int CTRL>
__device__ __forceinline__ void top2_step(float &b1, float &b2) {
  const float o1 = dpp_f32<CTRL>(b1), o2 = dpp_f32<CTRL>(b2);
  b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
  b1 = fmaxf(b1, o1);
}

__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// (dpp moves into lanes outside a row mask bring 0: the smallest of
// non-negative indices is right in lane 63, which is the one that is read)
__device__ __forceinline__ int wave_min_index(int v) {
  v = min(v, dpp_i32<0xB1>(v));
  v = min(v, dpp_i32<0x4E>(v));
  v = min(v, dpp_i32<0x141>(v));
  v = min(v, dpp_i32<0x140>(v));
  v = min(v, dpp_i32<0x142, 0xA>(v));
  v = min(v, dpp_i32<0x143, 0xC>(v));
  return lane_value(v, 63);
}

template <int DT, int EPL>
__device__ __forceinline__ void route_token(const ScoreCfg &c, const typename Elem<DT>::type *row,
                                            const float *bias, int L, int32_t *idx_out, float *w_out) {
  const int lane = threadIdx.x & 63;
  const int per = c.E / c.n_group;
  const int g = lane / L, l = lane % L;

  float p[EPL], s[EPL];
  {
    float lg[EPL], b[EPL];
#pragma unroll
    for (int m = 0; m < EPL; ++m) {
      const int i = l + m * L;
      const bool in = g < c.n_group && i < per;
      const int e = in ? g * per + i : 0;
      const float v = (float)row[e];
      b[m] = bias ? bias[e] : 0.f;
      lg[m] = in && v > kOff ? v : kOff;  // NaN: off
    }
    if (c.score == COLI_SCORE_SOFTMAX) {
      float top = lg[0];
#pragma unroll
      for (int m = 1; m < EPL; ++m) top = fmaxf(top, lg[m]);
      top = wave_max(top);
      double e[EPL], sum = 0.0;
#pragma unroll
      for (int m = 0; m < EPL; ++m) {
        // (equal infinities share the probability; -inf - top is no number, and off)
        e[m] = lg[m] == top ? 1.0 : exp_64((double)lg[m] - (double)top);
        if (lg[m] == kOff) e[m] = 0.0;
        sum += e[m];
      }
      sum = wave_sum_f64(sum);
      const double inv = sum >= 1.0 ? inverse_64(sum) : 0.0;
#pragma unroll
      for (int m = 0; m < EPL; ++m) p[m] = (float)(e[m] * inv);
    } else {
#pragma unroll
      for (int m = 0; m < EPL; ++m)
        p[m] = lg[m] == kOff ? 0.f : (float)inverse_64(1.0 + exp_64(-(double)lg[m]));
    }
#pragma unroll
    for (int m = 0; m < EPL; ++m) {
      const float v = bias ? p[m] + b[m] : p[m];
      s[m] = lg[m] > kOff && v > kOff ? v : kOff;
    }
  }

  if (c.topk_group < c.n_group) {
    float b1 = kOff, b2 = kOff;  // the group's two best
#pragma unroll
    for (int m = 0; m < EPL; ++m) {
      b2 = fmaxf(b2, fminf(b1, s[m]));
      b1 = fmaxf(b1, s[m]);
    }
    if (L >= 2) top2_step<0xB1>(b1, b2);
    if (L >= 4) top2_step<0x4E>(b1, b2);
    if (L >= 8) top2_step<0x141>(b1, b2);
    if (L >= 16) top2_step<0x140>(b1, b2);
    if (L >= 32) {
      const float o1 = __shfl_xor(b1, 16, 64), o2 = __shfl_xor(b2, 16, 64);
      b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
      b1 = fmaxf(b1, o1);
    }
    const float gs = c.group_score == COLI_GROUP_TOP2 && b2 > kOff ? b1 + b2 : b1;
    // kept if fewer than topk_group groups come before it
    int ahead = 0;
    for (int o = 0; o < c.n_group; ++o) {
      const float v = lane_value(gs, o * L);
      ahead += v > gs || (v == gs && o < g);
    }
    if (ahead >= c.topk_group) {
#pragma unroll
      for (int m = 0; m < EPL; ++m) s[m] = kOff;
    }
  }

  int my_idx = -1;
  float my_p = 0.f, total = 0.f;
  for (int j = 0; j < c.k; ++j) {
    // this lane's best: its experts are in rising order, the first of equals stays
    float best = s[0], bp = p[0];
    int bm = 0;
#pragma unroll
    for (int m = 1; m < EPL; ++m) {
      const bool more = s[m] > best;
      best = more ? s[m] : best;
      bp = more ? p[m] : bp;
      bm = more ? m : bm;
    }
    const float wb = wave_max(best);
    if (wb == kOff) break;  // no expert is left
    const int at = g * per + l + bm * L;
    const uint64_t who = __ballot(best == wb);
    int owner = __builtin_ctzll(who);
    int wi;
    if ((who & (who - 1)) == 0) {
      wi = lane_value(at, owner);
    } else {
      wi = wave_min_index(best == wb ? at : 0x7fffffff);
      owner = __builtin_ctzll(__ballot(best == wb && at == wi));
    }
    const float pv = lane_value(bp, owner);
    if (lane == owner) {
#pragma unroll
      for (int m = 0; m < EPL; ++m) s[m] = m == bm ? kOff : s[m];
    }
    total += pv;
    if (lane == j) {
      my_idx = wi;
      my_p = pv;
    }
  }
  if (lane < c.k) {
    float w = my_p;
    if (c.norm) w = total > 0.f ? w / total : 0.f;
    idx_out[lane] = my_idx;
    w_out[lane] = my_idx < 0 ? 0.f : w * c.rsf;
  }
}

// ---------------------------------------------------------------------------
// Four tokens a wave, 16 lanes each: a step of a reduction, a round of the
// selection and a ballot then serve four tokens at once.  For batches that
// fill the chip; a token alone takes longer than by a wave of its own.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float row_max_step(float v) { return fmaxf(v, dpp_f32<CTRL>(v)); }

// The largest value of the 16 lanes, in all of them (rotations by 8, 4, 2, 1).
__device__ __forceinline__ float row_max(float v) {
  v = row_max_step<0x128>(v);
  v = row_max_step<0x124>(v);
  v = row_max_step<0x122>(v);
  return row_max_step<0x121>(v);
}
__device__ __forceinline__ int row_min(int v) {
  v = min(v, dpp_i32<0x128>(v));
  v = min(v, dpp_i32<0x124>(v));
  v = min(v, dpp_i32<0x122>(v));
  return min(v, dpp_i32<0x121>(v));
}
__device__ __forceinline__ double row_sum(double v) {
  v += dpp_f64<0x128>(v);
  v += dpp_f64<0x124>(v);
  v += dpp_f64<0x122>(v);
  return v + dpp_f64<0x121>(v);
}

constexpr int kRowLanes = 16, kRowK = 16;  // lanes of a token, experts at most

// L lanes of the 16 for each group.
template <int DT, int EPL>
__global__ __launch_bounds__(256) void k_route_rows(
    ScoreCfg c, const typename Elem<DT>::type *__restrict__ logits, int64_t ld,
    const float *__restrict__ bias, int T, int L, int32_t *__restrict__ idx_out,
    float *__restrict__ w_out) {
  __shared__ float chosen[256 / kRowLanes][kRowK];
  const int lane = threadIdx.x & 15, slot = threadIdx.x / kRowLanes;
  const int t = blockIdx.x * (256 / kRowLanes) + slot;
  const bool real = t < T;  // (the lanes of no token run along: the moves need all of them)
  const auto *row = logits + (int64_t)(real ? t : 0) * ld;
  const int per = c.E / c.n_group;
  const int g = lane / L, l = lane % L;

  float p[EPL], s[EPL];
  {
    float lg[EPL], b[EPL];
#pragma unroll
    for (int m = 0; m < EPL; ++m) {
      const int i = l + m * L;
      const bool in = g < c.n_group && i < per;
      const int e = in ? g * per + i : 0;
      const float v = (float)row[e];
      b[m] = bias ? bias[e] : 0.f;
      lg[m] = in && v > kOff ? v : kOff;  // NaN: off
    }
    if (c.score == COLI_SCORE_SOFTMAX) {
      float top = lg[0];
#pragma unroll
      for (int m = 1; m < EPL; ++m) top = fmaxf(top, lg[m]);
      top = row_max(top);
      double e[EPL], sum = 0.0;
#pragma unroll
      for (int m = 0; m < EPL; ++m) {
        e[m] = lg[m] == top ? 1.0 : exp_64((double)lg[m] - (double)top);
        if (lg[m] == kOff) e[m] = 0.0;
        sum += e[m];
      }
      sum = row_sum(sum);
      const double inv = sum >= 1.0 ? inverse_64(sum) : 0.0;
#pragma unroll
      for (int m = 0; m < EPL; ++m) p[m] = (float)(e[m] * inv);
    } else {
#pragma unroll
      for (int m = 0; m < EPL; ++m)
        p[m] = lg[m] == kOff ? 0.f : (float)inverse_64(1.0 + exp_64(-(double)lg[m]));
    }
#pragma unroll
    for (int m = 0; m < EPL; ++m) {
      const float v = bias ? p[m] + b[m] : p[m];
      s[m] = lg[m] > kOff && v > kOff ? v : kOff;
    }
  }

  if (c.topk_group < c.n_group) {
    float b1 = kOff, b2 = kOff;  // the group's two best
#pragma unroll
    for (int m = 0; m < EPL; ++m) {
      b2 = fmaxf(b2, fminf(b1, s[m]));
      b1 = fmaxf(b1, s[m]);
    }
    if (L >= 2) top2_step<0xB1>(b1, b2);
    if (L >= 4) top2_step<0x4E>(b1, b2);
    if (L >= 8) top2_step<0x141>(b1, b2);
    const float gs = c.group_score == COLI_GROUP_TOP2 && b2 > kOff ? b1 + b2 : b1;
    int ahead = 0;
    for (int o = 0; o < c.n_group; ++o) {
      const float v = __shfl(gs, o * L, kRowLanes);
      ahead += v > gs || (v == gs && o < g);
    }
    if (ahead >= c.topk_group) {
#pragma unroll
      for (int m = 0; m < EPL; ++m) s[m] = kOff;
    }
  }

  int my_idx = -1;
  float best = kOff, bp = 0.f;
  int bm = 0;
  auto local_best = [&] {
    best = s[0], bp = p[0], bm = 0;
#pragma unroll
    for (int m = 1; m < EPL; ++m) {
      const bool more = s[m] > best;
      best = more ? s[m] : best;
      bp = more ? p[m] : bp;
      bm = more ? m : bm;
    }
  };
  local_best();
  for (int j = 0; j < c.k; ++j) {
    const float wb = row_max(best);
    const int at = g * per + l + bm * L;
    const int wi = row_min(best == wb ? at : 0x7fffffff);
    const bool any = wb > kOff;
    if (lane == j && any) my_idx = wi;
    if (any && best == wb && at == wi) {
      chosen[slot][j] = bp;
#pragma unroll
      for (int m = 0; m < EPL; ++m) s[m] = m == bm ? kOff : s[m];
    } else if (!any && lane == j) {
      chosen[slot][j] = 0.f;
    }
    local_best();
  }
  __syncthreads();
  if (real && lane < c.k) {
    float w = chosen[slot][lane];
    if (c.norm) {
      float total = 0.f;
      for (int j = 0; j < c.k; ++j) total += chosen[slot][j];
      w = total > 0.f ? w / total : 0.f;
    }
    idx_out[(int64_t)t * c.k + lane] = my_idx;
    w_out[(int64_t)t * c.k + lane] = my_idx < 0 ? 0.f : w * c.rsf;
  }
}

constexpr int kRouteWaves = 4;  // tokens of a workgroup

template <int DT, int EPL>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route_scored(
    ScoreCfg c, const typename Elem<DT>::type *__restrict__ logits, int64_t ld,
    const float *__restrict__ bias, int T, int L, int32_t *__restrict__ idx_out,
    float *__restrict__ w_out) {
  const int t = blockIdx.x * kRouteWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (t >= T) return;
  route_token<DT, EPL>(c, logits + (int64_t)t * ld, bias, L, idx_out + (int64_t)t * c.k,
                       w_out + (int64_t)t * c.k);
}

}  // namespace

hipError_t launch_route_scored(int dt, const ScoreCfg &c, const void *logits, int64_t ld,
                               const float *bias, int T, int32_t *idx, float *w, hipStream_t st) {
  if (T == 0) return hipSuccess;
  int gp = 1;
  while (gp < c.n_group) gp *= 2;
  const int L = 64 / gp;
  const int need = (c.E / c.n_group + L - 1) / L;  // at most 32: E <= 1024, gp < 2 n_group
  // Four tokens a wave where they fill the chip and 16 lanes hold a token's experts in 16 registers each
  // (us, a wave for each token / four tokens a wave):
  //   256 experts, softmax, bf16:    1024 tokens 5.2 / 9.2, 4096 8.1 / 9.5, 8192 12.8 / 11.0, 16384 21.7 / 16.6
  //   256 in 8 groups, sigmoid, f32: 1024 tokens 5.5 / 10.2, 4096 8.3 / 10.2, 8192 12.8 / 13.8, 16384 22.4 / 20.4
  //   128 experts, softmax, bf16:    1024 tokens 3.6 / 5.3, 4096 4.9 / 5.4, 8192 7.2 / 6.1, 16384 11.8 / 8.4
  //   64 experts, softmax, bf16:     1024 tokens 4.1 / 5.1, 3000 4.9 / 5.1, 4096 5.5 / 5.1, 16384 13.6 / 7.4
  const int L16 = gp <= kRowLanes ? kRowLanes / gp : 0;
  const int need16 = L16 ? (c.E / c.n_group + L16 - 1) / L16 : 99;
  const bool rows = T >= (need16 <= 4 ? 4096 : 8192) && need16 <= 16 && c.k <= kRowK;
  return by_dtype(dt, [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    const auto *lg = static_cast<const typename Elem<DT>::type *>(logits);
    if (rows) {
      auto by16 = [&](auto epl) {
        hipLaunchKernelGGL((k_route_rows<DT, decltype(epl)::value>), dim3((T + 15) / 16), dim3(256), 0, st, c,
                           lg, ld, bias, T, L16, idx, w);
      };
      if (need16 <= 4) by16(std::integral_constant<int, 4>());
      else if (need16 <= 8) by16(std::integral_constant<int, 8>());
      else by16(std::integral_constant<int, 16>());
      return hipGetLastError();
    }
    auto go = [&](auto epl) {
      hipLaunchKernelGGL((k_route_scored<DT, decltype(epl)::value>), dim3((T + kRouteWaves - 1) / kRouteWaves),
                         dim3(64 * kRouteWaves), 0, st, c, lg, ld, bias, T, L, idx, w);
    };
    if (need <= 1) go(std::integral_constant<int, 1>());
    else if (need <= 2) go(std::integral_constant<int, 2>());
    else if (need <= 4) go(std::integral_constant<int, 4>());
    else if (need <= 8) go(std::integral_constant<int, 8>());
    else if (need <= 16) go(std::integral_constant<int, 16>());
    else go(std::integral_constant<int, 32>());
    return hipGetLastError();
  });
}

}  // namespace coli
