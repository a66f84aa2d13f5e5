// lora.hpp -- the adapters' part of a product's results, as the kernels of
// the 8-bit product add it: c_a sum_r u[t][r] b_a[n][r] for token t's adapter a,
// with u [T][R] in binary32, in `slices` parts that are added in order.
#pragma once

#include "q8.hpp"

#pragma clang fp contract(off)

namespace coli {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// y's element from the exact sum.  (The product of two small scales could be
// subnormal where the result is not, so the sum comes first.  The last
// product and the bias's addition are one rounding by the source's own word,
// not by the compiler's choice in each kernel.  To fp16 they are one
// instruction, which rounds the exact value straight to fp16.)
__device__ __forceinline__ float finish(int acc, float st, float sn, float b) {
  return __builtin_fmaf((float)acc * sn, st, b);
}

// u[t][r .. r + 7]
__device__ __forceinline__ void lora_u(const Q8LoraArgs &a, int t, int r, float *u) {
  const float *p = a.u + (int64_t)t * a.R + r;
  *reinterpret_cast<Pack<float, 4> *>(u) = reinterpret_cast<const Pack<float, 4> *>(p)[0];
  *reinterpret_cast<Pack<float, 4> *>(u + 4) = reinterpret_cast<const Pack<float, 4> *>(p)[1];
  for (int s = 1; s < a.slices; ++s) {
    p += (int64_t)a.rows * a.R;
    const Pack<float, 4> lo = reinterpret_cast<const Pack<float, 4> *>(p)[0];
    const Pack<float, 4> hi = reinterpret_cast<const Pack<float, 4> *>(p)[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] += lo.v[j];
      u[4 + j] += hi.v[j];
    }
  }
}

// Eight elements in 16-byte words.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float *v) {
  constexpr int N = 16 / (int)sizeof(T);
#pragma unroll
  for (int k = 0; k < 8 / N; ++k) {
    const Pack<T, N> w = reinterpret_cast<const Pack<T, N> *>(p)[k];
#pragma unroll
    for (int j = 0; j < N; ++j) v[k * N + j] = (float)w.v[j];
  }
}

// Adds to d channels n .. n + 3 of token t, by vector instructions: with few tokens
// nearly every one has an adapter of its own, and the work is reading them.
template <int DT>
__device__ __forceinline__ void lora_four(const Q8LoraArgs &a, int t, int n, float *d) {
  typedef typename Elem<DT>::type T;
  const int id = a.ids[t];
  if ((uint32_t)id >= (uint32_t)a.L) return;
  float l[4] = {0.f, 0.f, 0.f, 0.f};
  const T *b[4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    b[r] = static_cast<const T *>(a.b) + ((int64_t)id * a.N + min(n + r, a.N - 1)) * a.R;
  for (int p = 0; p < a.R; p += 8) {
    float u[8], v[8];
    lora_u(a, t, p, u);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      load8(b[r] + p, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) l[r] = fmaf(u[j], v[j], l[r]);
    }
  }
  const float f = a.scale ? a.scale[id] : 1.f;
#pragma unroll
  for (int r = 0; r < 4; ++r) d[r] = fmaf(f, l[r], d[r]);
}

// v as a sum of P bfloat16 pieces, each the rounding of what is left: 8 bits a
// piece and one more by the sign of the rest, so two hold 2^-18 of v, three all
// of binary32.
template <int P>
__device__ __forceinline__ void split8(const float *v, v8bf *o) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float rest = v[j];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      o[p][j] = (__bf16)rest;
      rest -= (float)o[p][j];
    }
  }
}

// The 32 tokens of group j (lane lr has token t, if `there`) and 32 TN channels
// from nw on, by matrix instructions, one adapter of the group's tokens after
// another.  A lane's results are one token's, so a token takes none of what
// another's adapter gives, whatever it holds.  acc [TN][TMV] has the sums, and
// gets the results as binary32 bits; chans [32 TN] their channels' scales, and
// BN further their biases, in LDS.
//
// u stays in binary32: it enters as two bfloat16 pieces (2^-18 of it is lost
// where the result has 8 or 11 bits) or three; adapters in fp16 as two, which
// hold them whole, in fp32 as three.
template <int DT, int TN, int TMV, int BN>
__device__ __forceinline__ void lora_tile(const Q8LoraArgs &a, int t, bool there, float st, int nw,
                                          const float *chans, int j, v16i (*acc)[TMV]) {
  typedef typename Elem<DT>::type T;
  constexpr int PB = DT == COLI_BF16 ? 1 : DT == COLI_F16 ? 2 : 3, PU = DT == COLI_F32 ? 3 : 2;
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  int id = a.ids[t];
  if (!there || (uint32_t)id >= (uint32_t)a.L) id = -1;
  const float f = id < 0 || !a.scale ? 1.f : a.scale[id];
  // (read where they are used: held for the tile they would fill its registers)
  auto at = [&](int i, int g, int off = 0) {
    return reinterpret_cast<const Pack<float, 4> *>(chans + off + 32 * i + 8 * g + 4 * lh);
  };
  auto done = [&](const v16f *l, float f) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const Pack<float, 4> sn = *at(i, g), bn = *at(i, g, BN);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][4 * g + r] =
              __float_as_int(finish(acc[i][j][4 * g + r], st, sn.v[r], fmaf(f, l[i][4 * g + r], bn.v[r])));
      }
  };
  uint64_t todo = __ballot(id >= 0);
  while (todo) {
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    todo &= ~__ballot(id == e);
    const T *b = static_cast<const T *>(a.b) + (int64_t)e * a.N * a.R;
    v16f l[TN];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) l[i][r] = 0.f;
    for (int c = 0; c < a.R; c += 16) {
      const int r = min(c + 8 * lh, a.R - 8);
      const bool in = c + 8 * lh < a.R;
      float v[8];
      v8bf u[PU];
      lora_u(a, t, r, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = in ? v[k] : 0.f;
      split8<PU>(v, u);
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        v8bf w[PB];
        load8(b + (int64_t)min(nw + 32 * i + lr, a.N - 1) * a.R + r, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = in ? v[k] : 0.f;
        split8<PB>(v, w);
#pragma unroll
        for (int p = 0; p < PB; ++p)
#pragma unroll
          for (int q = 0; q < PU; ++q)
            if (p + q < (PB > PU ? PB : PU))
              l[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[p], u[q], l[i], 0, 0, 0);
      }
    }
    if (id == e) done(l, f);
  }
  if (id < 0) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const Pack<float, 4> sn = *at(i, g), bn = *at(i, g, BN);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // (rounded to y's type in the step itself, as without adapters)
          const T y = (T)finish(acc[i][j][4 * g + r], st, sn.v[r], bn.v[r]);
          acc[i][j][4 * g + r] = __float_as_int((float)y);
        }
      }
  }
}

}  // namespace
}  // namespace coli
