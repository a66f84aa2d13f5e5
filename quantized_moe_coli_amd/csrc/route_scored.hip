// route_scored.hip -- the router over softmax or sigmoid scores, with a
// selection bias, expert groups scored by their best or their two best
// experts, top-k and renormalised weights (coli_moe_route_scored).
//
// One wave routes one token.  The lanes are shared out to the groups, L =
// 64 / (groups rounded up to a power of two) lanes each, so that a group's
// best scores are found by a reduction over L neighbouring lanes; lane l of
// a group holds its experts l, l + L, ...  The scores are evaluated in
// binary64 and rounded once to binary32, so neither the order of a sum nor
// the approximation of an exponential moves an expert past another.
#include <cmath>

#include "q8.hpp"

#pragma clang fp contract(off)

namespace coli {
namespace {

constexpr float kOff = -INFINITY;  // score of an expert that cannot be chosen

template <int DT, int EPL>
__global__ __launch_bounds__(256) void k_route_scored(
    ScoreCfg c, const typename Elem<DT>::type *__restrict__ logits, int64_t ld,
    const float *__restrict__ bias, int T, int L, int32_t *__restrict__ idx_out,
    float *__restrict__ w_out) {
  const int t = blockIdx.x * 4 + threadIdx.x / 64;
  if (t >= T) return;
  const int lane = threadIdx.x & 63;
  const int per = c.E / c.n_group;
  const int g = lane / L, l = lane % L;
  const auto *row = logits + (int64_t)t * ld;

  float lg[EPL], p[EPL], s[EPL];
  float top = kOff;
#pragma unroll
  for (int m = 0; m < EPL; ++m) {
    const int i = l + m * L;
    const bool in = g < c.n_group && i < per;
    const float v = in ? (float)row[g * per + i] : kOff;
    lg[m] = v > kOff ? v : kOff;  // NaN: off
    top = fmaxf(top, lg[m]);
  }
  if (c.score == COLI_SCORE_SOFTMAX) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    double e[EPL], sum = 0.0;
#pragma unroll
    for (int m = 0; m < EPL; ++m) {
      // equal infinities share the probability
      e[m] = lg[m] == kOff ? 0.0 : lg[m] == top ? 1.0 : exp((double)lg[m] - (double)top);
      sum += e[m];
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
#pragma unroll
    for (int m = 0; m < EPL; ++m) p[m] = sum > 0.0 ? (float)(e[m] / sum) : 0.f;
  } else {
#pragma unroll
    for (int m = 0; m < EPL; ++m)
      p[m] = lg[m] == kOff ? 0.f : (float)(1.0 / (1.0 + exp(-(double)lg[m])));
  }
#pragma unroll
  for (int m = 0; m < EPL; ++m) {
    s[m] = kOff;
    if (lg[m] > kOff) {
      const float v = bias ? p[m] + bias[g * per + l + m * L] : p[m];
      s[m] = v > kOff ? v : kOff;
    }
  }

  if (c.topk_group < c.n_group) {
    float b1 = kOff, b2 = kOff;  // the group's two best
#pragma unroll
    for (int m = 0; m < EPL; ++m) {
      b2 = fmaxf(b2, fminf(b1, s[m]));
      b1 = fmaxf(b1, s[m]);
    }
    for (int d = L >> 1; d >= 1; d >>= 1) {
      const float o1 = __shfl_xor(b1, d, 64), o2 = __shfl_xor(b2, d, 64);
      b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
      b1 = fmaxf(b1, o1);
    }
    const float gs = c.group_score == COLI_GROUP_TOP2 && b2 > kOff ? b1 + b2 : b1;
    // kept if fewer than topk_group groups come before it
    int ahead = 0;
    for (int o = 0; o < c.n_group; ++o) {
      const float v = __shfl(gs, o * L, 64);
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
    float best = kOff;
    int at = 0x7fffffff, bm = 0;
#pragma unroll
    for (int m = 0; m < EPL; ++m) {
      // a lane's experts are in rising order: the first of equals stays
      if (s[m] > best) {
        best = s[m];
        bm = m;
        at = g * per + l + m * L;
      }
    }
    float wb = best;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) wb = fmaxf(wb, __shfl_xor(wb, d, 64));
    if (wb == kOff) break;  // no expert is left
    int wi = best == wb ? at : 0x7fffffff;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) wi = min(wi, __shfl_xor(wi, d, 64));
    float pv = 0.f;
    if (at == wi) {
#pragma unroll
      for (int m = 0; m < EPL; ++m)
        if (m == bm) {
          pv = p[m];
          s[m] = kOff;
        }
    }
    const int owner = __ffsll(__ballot(at == wi)) - 1;
    pv = __shfl(pv, owner, 64);
    total += pv;
    if (lane == j) {
      my_idx = wi;
      my_p = pv;
    }
  }
  if (lane < c.k) {
    float w = my_p;
    if (c.norm) w = total > 0.f ? w / total : 0.f;
    idx_out[(int64_t)t * c.k + lane] = my_idx;
    w_out[(int64_t)t * c.k + lane] = my_idx < 0 ? 0.f : w * c.rsf;
  }
}

}  // namespace

hipError_t launch_route_scored(int dt, const ScoreCfg &c, const void *logits, int64_t ld,
                               const float *bias, int T, int32_t *idx, float *w, hipStream_t st) {
  if (T == 0) return hipSuccess;
  int gp = 1;
  while (gp < c.n_group) gp *= 2;
  const int L = 64 / gp;
  const int need = (c.E / c.n_group + L - 1) / L;  // at most 32: E <= 1024, gp < 2 n_group
  return by_dtype(dt, [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    const auto *lg = static_cast<const typename Elem<DT>::type *>(logits);
    auto go = [&](auto epl) {
      hipLaunchKernelGGL((k_route_scored<DT, decltype(epl)::value>), dim3((T + 3) / 4), dim3(256), 0, st,
                         c, lg, ld, bias, T, L, idx, w);
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
