// q8.hpp -- shared by the kernels of the 8-bit products with one scale per
// token and one per output channel (q8_quant.hip, norm_quant.hip, q8_kernels.hpp)
// and by the scored router (route_scored.hip): element types, and the launchers that
// the C-ABI layer (api.hip) calls after checking every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "coli_moe.h"
#include "device.hpp"

namespace coli {

// Element types of coli_dtype.  Widening to binary32 is exact; narrowing
// rounds once to nearest even.
template <int DT> struct Elem;
template <> struct Elem<COLI_F32> { typedef float type; };
template <> struct Elem<COLI_BF16> { typedef __bf16 type; };
template <> struct Elem<COLI_F16> { typedef _Float16 type; };

// N consecutive elements, as one load or store of N * sizeof(T) bytes
// (callers guarantee that alignment).
template <typename T, int N>
struct __attribute__((aligned(N * sizeof(T)))) Pack {
  T v[N];
};

// One call of fn<DT>() for a run-time element type.
template <typename F>
inline hipError_t by_dtype(int dt, F &&fn) {
  switch (dt) {
    case COLI_F32: return fn(std::integral_constant<int, COLI_F32>());
    case COLI_BF16: return fn(std::integral_constant<int, COLI_BF16>());
    default: return fn(std::integral_constant<int, COLI_F16>());
  }
}

// Per-token quantisation of x [T][n] (u null), or of silu(x) * u.
hipError_t launch_quant_token(int dt, const void *x, int64_t ldx, const void *u, int64_t ldu, int T,
                              int n, int8_t *q, float *s, hipStream_t st);

// h = x + res, its root-mean-square norm y, and y's codes; res, gain, h, y, and
// q with s may be null.
struct NormArgs {
  const void *x, *res;  // [T][n], row strides ldx, ldres
  int64_t ldx, ldres;
  const float *gain;    // [n]
  float eps;
  int T, n;
  double inv_n;         // 1 / n
  void *h, *y;          // [T][n], row strides ldh, ldy
  int64_t ldh, ldy;
  int8_t *q;            // [T][n]
  float *s;             // [T]
};
hipError_t launch_norm_quant(int dt, const NormArgs &a, hipStream_t st);

// y[t] = (add ? add[t] : 0) + sum_j w[t][j] * o[t * k + j]; o of type odt, which
// is dt or COLI_F32.
hipError_t launch_combine_rows(int dt, int odt, const void *o, int64_t ldo, const int32_t *idx, const float *w,
                               int T, int k, int H, const void *add, int64_t ldadd, void *y,
                               int64_t ldy, hipStream_t st);

// The products.  Dense: offs null, rows = T, E = 1.  Grouped: the tables of
// coli_moe_dispatch; position i of expert e is pair p = perm[i], reads row
// p / fan of q and writes row p of y.
struct Q8Args {
  const int8_t *q;    // [rows][K]
  const float *s;     // [rows]
  const uint8_t *w;   // [E][N][K]
  const float *ws;    // [E][N]
  const float *bias;  // [N] or null (dense only)
  void *y;            // [rows or P][ldy]
  int64_t ldy;
  int rows, N, K, E;
  const int32_t *offs, *perm;  // grouped only
  int P, fan;
};
// Whether the call's grid stays within a launch's limits.
bool gemm_q8_fits(const Q8Args &a);
hipError_t launch_gemm_q8(int dt, const Q8Args &a, hipStream_t st);

// The dense product with low-rank adapters: L adapters a [L][R][K], b [L][N][R] of
// y's type; ids [rows] a token's adapter (none outside [0, L)), tab_offs [L + 1]
// and tab_perm [rows] the tokens by adapter; u [slices][rows][R] the tokens'
// products with a, in parts of K.
constexpr int kMaxAdapters = 1024;  // (their ranges lie in LDS)
struct Q8LoraArgs : Q8Args {
  const void *x;  // [rows][ldx]
  int64_t ldx;
  const void *a, *b;
  const float *scale;  // [L] or null
  const int32_t *ids, *tab_offs, *tab_perm;
  float *u;
  // [rows] tokens and their adapters, by adapter, those without one (-1) last, token -1: none;
  // null: as they are
  int2 *order;
  int L, R, slices;
  bool pieces;  // u as bfloat16 pieces, times the adapters' scales, by position in order (lora.hpp)
};
bool gemm_q8_lora_fits(const Q8LoraArgs &a);
size_t gemm_q8_lora_workspace(int T, int R);  // bytes of u and order
hipError_t launch_gemm_q8_lora(int dt, Q8LoraArgs a, void *workspace, hipStream_t st);

struct ScoreCfg {
  int E, k, n_group, topk_group, score, group_score, norm;
  float rsf;
};
hipError_t launch_route_scored(int dt, const ScoreCfg &c, const void *logits, int64_t ld,
                               const float *bias, int T, int32_t *idx, float *w, hipStream_t st);

}  // namespace coli
