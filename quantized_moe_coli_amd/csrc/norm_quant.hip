// norm_quant.hip -- the residual's addition, the root-mean-square norm of the
// sum, and the norm as int8 codes with one scale per token, in one pass:
//   h = fl32(x + res),  y = fl32(h * r * g),  r = 1 / sqrt(mean(h^2) + eps),
//   s = fl32(max|y| * fl32(1 / 127)),  q = clamp(rint(fl32(y / s)), -127, 127).
//
// The sum of squares, r and the products h r g are evaluated in binary64 and y
// is rounded once to binary32 from them, as SwiGLU's result is: neither the
// order of the sum nor the root moves y by more than one step in some 10^7
// values, so codes do not depend on how a row is shared out.  A square of a
// binary32 value neither overflows nor vanishes in binary64.  A row that holds a
// NaN or an infinity gives r = NaN or 0 and a NaN in y where it stood, so its
// scale is NaN and its codes 0, as the other quantisers have it.
//
// Bound by the memory: every element of x, res, h, y and q is moved once, as
// long as a row fits the registers of the threads that share it.  What lies past a
// row's first 32768 elements, or 8192 where rows are loaded by elements, is read
// three times with codes, twice without.  8192 x 6144 bfloat16 with h, y and
// codes 95.5 us (453 MB, 4.7 TB/s; a copy reaches 5.06), float32 with h and y 148 us
// (5.4 TB/s); 2048 x 16384 69 us (4.4 TB/s), 256 x 65536 38 us (3.9); rows of a wider
// buffer that start at any element 1.4 to 1.7 times as long (638 x 9952 35 us, 20 where
// aligned, 2048 x 16384 103).  One row of 6144 4.4 us, of which a launch is 2, two sums
// over its workgroup the most of the rest; of 131040 43 us, by one workgroup.
#include <algorithm>
#include <type_traits>

#include "token_codes.hpp"

#pragma clang fp contract(off)

namespace coli {
namespace {

// One piece of a row in its own type.  VEC: kPiece consecutive elements, 16
// bytes a load.  Otherwise (rows that start at any element, lengths that are
// no multiple of kPiece) the lanes of the row take neighbouring elements, so
// that a load still covers a run.
template <int DT, bool VEC>
struct Piece {
  typedef typename Elem<DT>::type T;
  static constexpr int N = 16 / (int)sizeof(T);
  alignas(16) T v[kPiece];

  // element j of piece i for thread tr of TR
  template <int TR>
  __device__ __forceinline__ static int64_t at(int i, int tr, int j) {
    return VEC ? ((int64_t)i * TR + tr) * kPiece + j : ((int64_t)i * kPiece + j) * TR + tr;
  }
  // elements past the row's end read its last (VEC: its last piece)
  template <int TR>
  __device__ __forceinline__ void load(const T *row, int i, int tr, int n) {
    if constexpr (VEC) {
      const T *p = row + min((int)at<TR>(i, tr, 0), n - kPiece);
#pragma unroll
      for (int k = 0; k < kPiece / N; ++k)
        *reinterpret_cast<Pack<T, N> *>(v + k * N) = reinterpret_cast<const Pack<T, N> *>(p)[k];
    } else {
#pragma unroll
      for (int j = 0; j < kPiece; ++j) v[j] = row[min((int)at<TR>(i, tr, j), n - 1)];
    }
  }
  template <int TR>
  __device__ __forceinline__ static void store(T *row, int i, int tr, int n, const float *f) {
    if constexpr (VEC) {
      if (at<TR>(i, tr, 0) >= n) return;
      T *p = row + at<TR>(i, tr, 0);
#pragma unroll
      for (int k = 0; k < kPiece / N; ++k) {
        Pack<T, N> o;
#pragma unroll
        for (int j = 0; j < N; ++j) o.v[j] = (T)f[k * N + j];
        reinterpret_cast<Pack<T, N> *>(p)[k] = o;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPiece; ++j)
        if (at<TR>(i, tr, j) < n) row[at<TR>(i, tr, j)] = (T)f[j];
    }
  }
};

// 1 / sqrt(v) of a positive v: the instruction's estimate and one step of third
// order, to a few units of binary64's last place; 0 of an infinity, NaN of NaN.
__device__ __forceinline__ double inverse_root(double v) {
  const double r = __builtin_amdgcn_rsq(v);
  const double e = fma(-v * r, r, 1.0);
  return r == 0.0 ? 0.0 : fma(r * e, fma(e, 0.375, 0.5), r);
}

// A row by TR threads (16, 64, 256 or 1024), in workgroups of at least 256.
// Its first NP * TR pieces are read once and held as h, then as y.
template <int DT, bool VEC, int TR, int NP>
__global__ __launch_bounds__(TR < 256 ? 256 : TR) void k_norm_quant(NormArgs a) {
  typedef typename Elem<DT>::type T;
  typedef Piece<DT, VEC> P;
  constexpr int RPB = TR < 256 ? 256 / TR : 1;
  __shared__ double psum[TR < 64 ? 1 : TR / 64];
  __shared__ int pmax[TR < 64 ? 1 : TR / 64];
  const int row = (blockIdx.y * gridDim.x + blockIdx.x) * RPB + threadIdx.x / TR;
  if (row >= a.T) return;  // whole rows, whose lanes are apart from the others' in every step below
  const int tr = threadIdx.x % TR, n = a.n;
  const T *x = static_cast<const T *>(a.x) + row * a.ldx;
  const T *res = a.res ? static_cast<const T *>(a.res) + row * a.ldres : nullptr;

  auto sum_of = [&](const P &px, const P &pr, float *h) {
#pragma unroll
    for (int j = 0; j < kPiece; ++j) h[j] = res ? (float)px.v[j] + (float)pr.v[j] : (float)px.v[j];
  };
  auto get = [&](int i, float *h) {
    P px, pr;
    px.template load<TR>(x, i, tr, n);
    if (res) pr.template load<TR>(res, i, tr, n);
    sum_of(px, pr, h);
  };
  auto inside = [&](int i, int j) { return P::template at<TR>(i, tr, j) < n; };
  auto gains = [&](int i, float *g) {
    if constexpr (VEC) {
      const Pack<float, 4> *p = reinterpret_cast<const Pack<float, 4> *>(
          a.gain + min((int)P::template at<TR>(i, tr, 0), n - kPiece));
      *reinterpret_cast<Pack<float, 4> *>(g) = p[0];
      *reinterpret_cast<Pack<float, 4> *>(g + 4) = p[1];
    } else {
#pragma unroll
      for (int j = 0; j < kPiece; ++j) g[j] = a.gain[min((int)P::template at<TR>(i, tr, j), n - 1)];
    }
  };

  // (the pieces that no thread has are passed over by the whole workgroup)
  auto any = [&](int i) { return i == 0 || i * TR * kPiece < n; };
  float v[NP][kPiece], g0[kPiece];
  {
    P px[NP], pr[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (any(i)) px[i].template load<TR>(x, i, tr, n);
    if (res) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (any(i)) pr[i].template load<TR>(res, i, tr, n);
    }
    if (NP == 1 && a.gain) gains(0, g0);  // (one row's latency: asked for with its elements)
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (any(i)) sum_of(px[i], pr[i], v[i]);
  }
  double ss = 0;
  auto square = [&](int i, const float *h) {
    if constexpr (VEC) {
      if (!inside(i, 0)) return;
    }
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      const double d = VEC || inside(i, j) ? (double)h[j] : 0.0;
      ss = fma(d, d, ss);
    }
  };
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (any(i)) square(i, v[i]);
  const int pieces = (n + kPiece * TR - 1) / (kPiece * TR);
  for (int i = NP; i < pieces; ++i) {
    float h[kPiece];
    get(i, h);
    square(i, h);
  }
  if constexpr (TR < 64) {
    ss = group_sum_f64<TR>(ss);
  } else {
    ss = wave_sum_f64(ss);
    if constexpr (TR > 64) {
      if ((threadIdx.x & 63) == 0) psum[threadIdx.x / 64] = ss;
      __syncthreads();
      double p[TR / 64];
#pragma unroll
      for (int i = 0; i < TR / 64; ++i) p[i] = psum[i];
#pragma unroll
      for (int d = TR / 128; d >= 1; d /= 2)
#pragma unroll
        for (int i = 0; i < d; ++i) p[i] += p[i + d];
      ss = p[0];
    }
  }
  const double r = inverse_root(ss * a.inv_n + (double)a.eps);

  auto norm = [&](int i, const float *h, const float *g, float *y) {
#pragma unroll
    for (int j = 0; j < kPiece; ++j) y[j] = (float)((double)h[j] * r * (a.gain ? (double)g[j] : 1.0));
  };
  T *ho = a.h ? static_cast<T *>(a.h) + row * a.ldh : nullptr;
  T *yo = a.y ? static_cast<T *>(a.y) + row * a.ldy : nullptr;
  // (h and y may lie on x and res: a piece is written by the thread that has
  // read it, after it has; pieces that are read again are written last)
  int amax = 0;
  auto largest = [&](int i, const float *y) {
    if constexpr (VEC) {
      if (!inside(i, 0)) return;
    }
#pragma unroll
    for (int j = 0; j < kPiece; ++j)
      if (VEC || inside(i, j)) amax = max(amax, __float_as_int(y[j]) & 0x7fffffff);
  };
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if (!any(i)) continue;
    if (ho) P::template store<TR>(ho, i, tr, n, v[i]);
    float g[kPiece];
    if (NP > 1 && a.gain) gains(i, g);
    norm(i, v[i], NP == 1 ? g0 : g, v[i]);
    if (yo) P::template store<TR>(yo, i, tr, n, v[i]);
    largest(i, v[i]);
  }
  if (a.q) {
    for (int i = NP; i < pieces; ++i) {
      float h[kPiece], g[kPiece];
      get(i, h);
      if (a.gain) gains(i, g);
      norm(i, h, g, h);
      largest(i, h);
    }
    // (lanes outside a step's rows read 0, which is no larger)
    amax = max(amax, dpp_i32<0xB1>(amax));
    amax = max(amax, dpp_i32<0x4E>(amax));
    amax = max(amax, dpp_i32<0x141>(amax));
    amax = max(amax, dpp_i32<0x140>(amax));
    if constexpr (TR >= 64) {
      amax = max(amax, dpp_i32<0x142, 0xA>(amax));
      amax = max(amax, dpp_i32<0x143, 0xC>(amax));
      amax = __builtin_amdgcn_readlane(amax, 63);
      if constexpr (TR > 64) {
        if ((threadIdx.x & 63) == 0) pmax[threadIdx.x / 64] = amax;
        __syncthreads();
        amax = pmax[0];
#pragma unroll
        for (int i = 1; i < TR / 64; ++i) amax = max(amax, pmax[i]);
      }
    }
  }
  const bool bad = amax >= 0x7f800000;
  const float sc = bad ? __int_as_float(0x7fc00000) : __int_as_float(amax) * (1.f / 127.f);
  const float inv = sc > 1e-30f ? 1.f / sc : 0.f;  // 0: divide
  const bool zero = bad || sc == 0.f;
  if (a.q && tr == 0) a.s[row] = sc;
  int8_t *qo = a.q ? a.q + (int64_t)row * n : nullptr;
  auto put = [&](int i, const float *y) {
    uint32_t w[2] = {0, 0};
    if (!zero) codes(y, sc, inv, w);
    if constexpr (VEC) {
      if (inside(i, 0)) *reinterpret_cast<uint2 *>(qo + P::template at<TR>(i, tr, 0)) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int j = 0; j < kPiece; ++j)
        if (inside(i, j)) qo[P::template at<TR>(i, tr, j)] = (int8_t)(w[j >> 2] >> (8 * (j & 3)));
    }
  };
  if (qo) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (any(i)) put(i, v[i]);
  }
  for (int i = NP; i < pieces; ++i) {
    float h[kPiece], g[kPiece];
    get(i, h);
    if (a.gain) gains(i, g);
    if (ho) P::template store<TR>(ho, i, tr, n, h);
    norm(i, h, g, h);
    if (yo) P::template store<TR>(yo, i, tr, n, h);
    if (qo) put(i, h);
  }
}

}  // namespace

hipError_t launch_norm_quant(int dt, const NormArgs &a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  return by_dtype(dt, [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    const bool vec = a.n % kPiece == 0 && rows_aligned<DT>(a.x, a.ldx, 16) &&
                     (!a.res || rows_aligned<DT>(a.res, a.ldres, 16)) &&
                     (!a.h || rows_aligned<DT>(a.h, a.ldh, 16)) &&
                     (!a.y || rows_aligned<DT>(a.y, a.ldy, 16)) && reinterpret_cast<uintptr_t>(a.gain) % 16 == 0;
    auto go = [&](auto vecc, auto trc, auto npc) {
      constexpr int TR = decltype(trc)::value, NT = TR < 256 ? 256 : TR, RPB = NT / TR;
      const int wgs = (a.T + RPB - 1) / RPB;
      hipLaunchKernelGGL((k_norm_quant<DT, decltype(vecc)::value, TR, decltype(npc)::value>),
                         dim3(std::min(wgs, kGridX), (wgs + kGridX - 1) / kGridX), dim3(NT), 0, st, a);
    };
    // Few rows: a thread for every piece, the shortest way through a row; many: four
    // pieces a thread, more rows at a time.  With h, y and codes in bfloat16 (us, the one
    // / the other):
    //   by 16 and by 64 threads, 2304, 8192 and 33564 rows:
    //     192 columns  4.5 / 4.2, 5.9 / 8.3, 14.9 / 25.1;   320  5.8 / 4.3, 9.0 / 9.3, 22.2 / 25.8
    //     384          5.9 / 4.4, 9.3 / 9.5, 23.9 / 26.3;   512  7.2 / 4.5, 11.6 / 10.1, 34.5 / 34.9
    //   512 columns:   256 rows 3.1 / 3.4, 1024 3.4 / 3.7, 4096 7.3 / 7.1
    //   2048 columns:  256 rows 3.6 / 6.8, 1024 7.5 / 9.3, 4096 16.6 / 16.5
    //   6144 columns:  16 rows 4.6 / 5.6, 256 6.2 / 7.3, 512 10.6 / 9.5, 4096 63.6 / 46.4
    auto by_len = [&](auto vecc) {
      constexpr std::integral_constant<int, 1> one{};
      constexpr std::integral_constant<int, 4> four{};
      // (1024 threads that load by elements have registers for one piece: 638 rows of
      // 9952 33 us, with four, which are kept in memory, 1581)
      constexpr std::integral_constant<int, decltype(vecc)::value ? 4 : 1> most{};
      if (a.n <= 16 * kPiece) {
        go(vecc, std::integral_constant<int, 16>(), one);
      } else if (a.T <= (a.n <= 256 * kPiece ? 2048 : 384)) {
        if (a.n <= 64 * kPiece) go(vecc, std::integral_constant<int, 64>(), one);
        else if (a.n <= 256 * kPiece) go(vecc, std::integral_constant<int, 256>(), one);
        else if (a.n <= 1024 * kPiece) go(vecc, std::integral_constant<int, 1024>(), one);
        else go(vecc, std::integral_constant<int, 1024>(), most);
      } else {
        if (a.n <= 16 * kPiece * 3) go(vecc, std::integral_constant<int, 16>(), four);
        else if (a.n <= 64 * kPiece * 4) go(vecc, std::integral_constant<int, 64>(), four);
        else if (a.n <= 256 * kPiece * 4) go(vecc, std::integral_constant<int, 256>(), four);
        else go(vecc, std::integral_constant<int, 1024>(), most);
      }
    };
    if (vec) by_len(std::true_type());
    else by_len(std::false_type());
    return hipGetLastError();
  });
}

}  // namespace coli
