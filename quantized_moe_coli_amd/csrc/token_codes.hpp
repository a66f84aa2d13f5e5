// token_codes.hpp -- shared by the kernels that make int8 codes with one scale
// per token (q8_quant.hip, norm_quant.hip).
#pragma once

#include "q8.hpp"

#pragma clang fp contract(off)

namespace coli {

constexpr int kPiece = 8;        // elements of a piece of a row
constexpr int kGridX = 1 << 20;  // workgroups along x (a launch's threads along one axis fit 32 bits)

// Codes of one piece, with the row's scale and its reciprocal.  x * inv
// differs from the correctly rounded x / s by less than 127 * 2^-22, so
// rounding it to a whole number gives the same code unless it lies within
// that of a half; there, and for scales too small for a reciprocal (inv =
// 0), the division is made.
__device__ __forceinline__ void codes(const float *v, float s, float inv, uint32_t *out) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < kPiece; ++j) {
    float r = v[j] * inv;
    float c = rintf(r);
    if (fabsf(r - c) > 0.4999f || inv == 0.f) c = rintf(v[j] / s);
    c = fminf(fmaxf(c, -127.f), 127.f);
    w[j >> 2] |= ((uint32_t)(int32_t)c & 0xFFu) << (8 * (j & 3));
  }
  out[0] = w[0];
  out[1] = w[1];
}

template <int DT>
inline bool rows_aligned(const void *p, int64_t ld, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 &&
         (uint64_t)ld * sizeof(typename Elem<DT>::type) % bytes == 0;
}

}  // namespace coli
