// q8_quant.hip -- int8 codes with one scale per token (row), of a row of
// activations or of SwiGLU's result, and the weighted sum of a token's
// expert outputs.
//
// A row's codes: a = max|x|, s = fl32(a * fl32(1 / 127)), q = clamp(
// round_half_even(fl32(x / s)), -127, 127); s = 0 gives q = 0.  This is the
// rule of the library's other containers with the row as the block, but for
// the scale: one product with the reciprocal, as a tensor divided by a number
// gives it on the GPU.  With c = fl32(1 / 127), 127 c = 1 - 2^-28, so s is off
// max|x| / 127 by at most 2^-24 + 2^-28 of it where the quotient's rounding
// alone is 2^-24.  About 5 % of rows get the neighbouring scale, in which one
// code in 10^7 moves to its neighbour, from next to the one side of a half to
// next to the other: no further from x.  A row that holds a
// NaN or an infinity has no scale: s = NaN and q = 0, so that every product
// made from it is NaN and the fault stays visible.
//
// SwiGLU's h = silu(g) * u is evaluated in binary64 and rounded once to
// binary32, as the layer's own gate/up kernels do, so that how the exponential
// was approximated moves h by one step in about one case in four million, and
// a code only where its quotient lies next to a half then.
//
// 8192 x 6144 bfloat16 30-32 us (150 MB, 4.7-5.0 TB/s: what a copy reaches);
// SwiGLU of 32768 x 2048 96-111 us (335 MB), bound by the binary64 instructions
// of its exponential; the sum of 4096 x 8 rows of 6144 to bfloat16 85 us from
// bfloat16 rows (453 MB, 5.3 TB/s), 170 us from fp32 rows (856 MB, 5.0 TB/s).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "exp64.hpp"
#include "q8.hpp"
#include "token_codes.hpp"

#pragma clang fp contract(off)

namespace coli {
namespace {

constexpr int kPieces = 4;   // pieces a thread keeps in registers

__device__ __forceinline__ float silu_mul(float g, float u) {
  const double gd = (double)g;
  return (float)(gd * inverse_64(1.0 + exp_64(-gd)) * (double)u);
}

template <int DT, bool VEC>
__device__ __forceinline__ void load_piece(const typename Elem<DT>::type *p, float *v) {
  typedef typename Elem<DT>::type T;
  if constexpr (VEC) {
    constexpr int N = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < kPiece / N; ++i) {
      const Pack<T, N> pk = reinterpret_cast<const Pack<T, N> *>(p)[i];
#pragma unroll
      for (int j = 0; j < N; ++j) v[i * N + j] = (float)pk.v[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPiece; ++j) v[j] = (float)p[j];
  }
}

// A row by TR threads (64, 256 or 1024), in workgroups of at least 256.  Rows of up to kPieces * TR pieces are read once
// and held in registers between the maximum and the codes; longer ones are
// read again.
template <int DT, bool GLU, bool VEC, int TR>
__global__ __launch_bounds__(TR < 256 ? 256 : TR) void k_quant_token(
    const typename Elem<DT>::type *__restrict__ x, int64_t ldx,
    const typename Elem<DT>::type *__restrict__ u, int64_t ldu, int T, int n,
    int8_t *__restrict__ q, float *__restrict__ s) {
  constexpr int RPB = TR < 256 ? 256 / TR : 1;
  __shared__ int part[TR / 64];
  const int row = (blockIdx.y * gridDim.x + blockIdx.x) * RPB + threadIdx.x / TR;
  if (row >= T) return;  // whole waves (TR >= 64): no barrier is missed, rows of TR > 64 have their own workgroup
  const int tr = threadIdx.x % TR;
  const int np = n / kPiece;
  const auto *xr = x + (int64_t)row * ldx;
  const auto *ur = GLU ? u + (int64_t)row * ldu : nullptr;

  auto get = [&](int p, float *v) {
    load_piece<DT, VEC>(xr + (int64_t)p * kPiece, v);
    if constexpr (GLU) {
      float w[kPiece];
      load_piece<DT, VEC>(ur + (int64_t)p * kPiece, w);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) v[j] = silu_mul(v[j], w[j]);
    }
  };
  // |x| as its bits: ordered as the values are, infinities and NaN above
  // every finite one
  float v[kPieces][kPiece];
  int amax = 0;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int p = i * TR + tr;
    if (p < np) {
      get(p, v[i]);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) amax = max(amax, __float_as_int(v[i][j]) & 0x7fffffff);
    }
  }
  for (int p = kPieces * TR + tr; p < np; p += TR) {
    float t[kPiece];
    get(p, t);
#pragma unroll
    for (int j = 0; j < kPiece; ++j) amax = max(amax, __float_as_int(t[j]) & 0x7fffffff);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) amax = max(amax, __shfl_xor(amax, d, 64));
  if constexpr (TR > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = amax;
    __syncthreads();
    amax = part[0];
#pragma unroll
    for (int i = 1; i < TR / 64; ++i) amax = max(amax, part[i]);
  }
  const bool bad = amax >= 0x7f800000;
  const float sc = bad ? __int_as_float(0x7fc00000) : __int_as_float(amax) * (1.f / 127.f);
  const float inv = sc > 1e-30f ? 1.f / sc : 0.f;  // 0: divide
  if (tr == 0) s[row] = sc;
  const bool zero = bad || sc == 0.f;
  int8_t *qr = q + (int64_t)row * n;
  auto put = [&](int p, const float *t) {
    uint32_t w[2] = {0, 0};
    if (!zero) codes(t, sc, inv, w);
    *reinterpret_cast<uint2 *>(qr + (int64_t)p * kPiece) = make_uint2(w[0], w[1]);
  };
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int p = i * TR + tr;
    if (p < np) put(p, v[i]);
  }
  for (int p = kPieces * TR + tr; p < np; p += TR) {
    float t[kPiece];
    get(p, t);
    put(p, t);
  }
}

// y[t][h] = (add[t][h]) + sum_j w[t][j] o[t k + j][h], slots in order, in
// binary32, rounded once to the type.  A slot whose idx is -1 is not read:
// its row of o may hold anything.  o is of y's type or binary32.
template <int DT, int ODT, int N>
__global__ __launch_bounds__(256) void k_combine_rows(
    const typename Elem<ODT>::type *__restrict__ o, int64_t ldo, const int32_t *__restrict__ idx,
    const float *__restrict__ w, int k, int H, const typename Elem<DT>::type *add, int64_t ldadd,
    typename Elem<DT>::type *y, int64_t ldy) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<ODT>::type O;
  constexpr int NO = N * (int)sizeof(O) > 16 ? 16 / (int)sizeof(O) : N;  // elements of a load of o
  const int t = blockIdx.x;
  const int h = (blockIdx.y * 256 + threadIdx.x) * N;
  if (h >= H) return;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  if (add) {
    const Pack<T, N> a = *reinterpret_cast<const Pack<T, N> *>(add + (int64_t)t * ldadd + h);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = (float)a.v[i];
  }
  for (int j = 0; j < k; ++j) {
    const int64_t p = (int64_t)t * k + j;
    if (idx && idx[p] < 0) continue;
    const float wj = w[p];
#pragma unroll
    for (int g = 0; g < N / NO; ++g) {
      const Pack<O, NO> a = reinterpret_cast<const Pack<O, NO> *>(o + p * ldo + h)[g];
#pragma unroll
      for (int i = 0; i < NO; ++i) acc[g * NO + i] = fmaf(wj, (float)a.v[i], acc[g * NO + i]);
    }
  }
  Pack<T, N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) r.v[i] = (T)acc[i];
  *reinterpret_cast<Pack<T, N> *>(y + (int64_t)t * ldy + h) = r;
}

}  // namespace

hipError_t launch_quant_token(int dt, const void *x, int64_t ldx, const void *u, int64_t ldu, int T,
                              int n, int8_t *q, float *s, hipStream_t st) {
  if (T == 0) return hipSuccess;
  return by_dtype(dt, [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    typedef typename Elem<DT>::type E;
    const E *xe = static_cast<const E *>(x), *ue = static_cast<const E *>(u);
    const bool vec = rows_aligned<DT>(x, ldx, 16) && (!u || rows_aligned<DT>(u, ldu, 16));
    auto go = [&](auto glu, auto vecc, auto trc) {
      constexpr int TR = decltype(trc)::value;
      constexpr int NT = TR < 256 ? 256 : TR, RPB = NT / TR;
      const int wgs = (T + RPB - 1) / RPB;
      hipLaunchKernelGGL((k_quant_token<DT, decltype(glu)::value, decltype(vecc)::value, TR>),
                         dim3(std::min(wgs, kGridX), (wgs + kGridX - 1) / kGridX), dim3(NT), 0, st, xe,
                         ldx, ue, ldu, T, n, q, s);
    };
    auto by_len = [&](auto glu, auto vecc) {
      // few rows: as many threads as a row has pieces, which is the shortest way
      // through it (us, by pieces / by 4 pieces a thread; bfloat16):
      //   2048 columns:          8 rows 2.8 / 4.0, 512 rows 3.1 / 4.5, 1024 3.5 / 4.8, 4096 7.2 / 6.8
      //   2048 columns, SwiGLU:  8 rows 3.2 / 5.9, 512 rows 4.2 / 6.4, 1024 5.7 / 6.5, 4096 16.0 / 16.0
      //   6144 columns:          8 rows 3.0 / 3.7, 512 rows 4.5 / 4.6, 1024 7.0 / 5.8, 4096 20.5 / 16.4
      //   6144 columns, SwiGLU:  8 rows 4.5 / 5.1, 512 rows 8.2 / 7.8, 1024 14.4 / 12.4, 4096 52.1 / 39.8
      const int few = T <= 512 ? kPieces : 1;
      if (n * few <= 64 * kPieces * kPiece) go(glu, vecc, std::integral_constant<int, 64>());
      else if (n * few <= 256 * kPieces * kPiece) go(glu, vecc, std::integral_constant<int, 256>());
      else go(glu, vecc, std::integral_constant<int, 1024>());
    };
    auto by_vec = [&](auto glu) {
      if (vec) by_len(glu, std::true_type());
      else by_len(glu, std::false_type());
    };
    if (u) by_vec(std::true_type());
    else by_vec(std::false_type());
    return hipGetLastError();
  });
}

hipError_t launch_combine_rows(int dt, int odt, const void *o, int64_t ldo, const int32_t *idx, const float *w,
                               int T, int k, int H, const void *add, int64_t ldadd, void *y,
                               int64_t ldy, hipStream_t st) {
  if (T == 0) return hipSuccess;
  return by_dtype(dt, [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    typedef typename Elem<DT>::type E;
    constexpr int N = 16 / (int)sizeof(E);
    auto go = [&](auto odtc, auto nc) {
      constexpr int ODT = decltype(odtc)::value, NN = decltype(nc)::value;
      const int per_row = (H + 256 * NN - 1) / (256 * NN);
      hipLaunchKernelGGL((k_combine_rows<DT, ODT, NN>), dim3(T, per_row), dim3(256), 0, st,
                         static_cast<const typename Elem<ODT>::type *>(o), ldo, idx, w, k, H,
                         static_cast<const E *>(add), ldadd, static_cast<E *>(y), ldy);
    };
    auto by_width = [&](auto odtc) {
      if (H % N == 0 && rows_aligned<decltype(odtc)::value>(o, ldo, 16) && rows_aligned<DT>(y, ldy, 16) &&
          (!add || rows_aligned<DT>(add, ldadd, 16)))
        go(odtc, std::integral_constant<int, N>());
      else
        go(odtc, std::integral_constant<int, 1>());
    };
    if (odt == dt) by_width(dtc);
    else by_width(std::integral_constant<int, COLI_F32>());
    return hipGetLastError();
  });
}

}  // namespace coli
