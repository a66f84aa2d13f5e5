// lora.hpp -- the adapters' part of a product's results, as the kernels of
// the 8-bit product add it: c_a sum_r u[t][r] b_a[n][r] for token t's adapter a.
// For the kernels of few tokens u [T][R] is in binary32, in `slices` parts that
// are added in order.
#pragma once

#include "q8.hpp"

#pragma clang fp contract(off)

namespace coli {
namespace {

// Whether a kernel's arguments are the product's with adapters.
template <typename ARGS>
constexpr bool kLora = std::is_same<ARGS, Q8LoraArgs>::value;

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

// u[t][r .. r + 3], of up to S parts of K, all asked for together
template <int S>
struct UParts {
  Pack<float, 4> v[S];
  __device__ __forceinline__ void load(const Q8LoraArgs &a, int t, int r) {
    const float *p = a.u + (int64_t)t * a.R + r;
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (s < a.slices) v[s] = *reinterpret_cast<const Pack<float, 4> *>(p + (int64_t)s * a.rows * a.R);
  }
  __device__ __forceinline__ Pack<float, 4> sum(const Q8LoraArgs &a) const {
    Pack<float, 4> o = v[0];
#pragma unroll
    for (int s = 1; s < S; ++s)
      if (s < a.slices) {
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] += v[s].v[j];
      }
    return o;
  }
};

// Parts of K that a kernel of tiles of bm tokens takes u in.
constexpr int lora_parts(int bm) { return bm == 16 ? 8 : 4; }

// Adds the adapters' part to the biases of the 16 x 16 results that a wave of
// k_q8_ring finishes, by vector instructions: with few tokens nearly every one has
// an adapter of its own, and the work is reading it.  Lane (li, lg) has channels
// 4 lg .. of token li.  What it needs is asked for while the last stages of the
// sums are on their way: the first ranks of its rows of b, and its workgroup's
// share of u, which goes through LDS for all the waves.  (As much is asked for
// ahead as leaves the registers for two workgroups a CU.)
template <int DT, int BM, int NT, int TPW>
struct LoraRing {
  typedef typename Elem<DT>::type T;
  static constexpr int N = 16 / (int)sizeof(T);          // ranks of a 16-byte piece
  static constexpr int FIRST = TPW > 1 && NT > 256 ? 0 : N / 4;  // eights of ranks asked for ahead
  static constexpr int BYTES = BM * (128 + 4) * 4;       // u, rows of R + 4
  int id[TPW];
  Pack<T, N> w[TPW][FIRST ? FIRST : 1][4][8 / N];
  UParts<lora_parts(BM)> part;
  float scale[TPW];

  __device__ __forceinline__ static void piece(Pack<T, N> *o, const T *p) {
#pragma unroll
    for (int k = 0; k < 8 / N; ++k) o[k] = reinterpret_cast<const Pack<T, N> *>(p)[k];
  }
  // item o of u: token o / (R / 4), ranks 4 (o % (R / 4)) ..
  __device__ __forceinline__ static int token(const Q8LoraArgs &a, int o) {
    return (int)((uint32_t)o * (262144u / (uint32_t)a.R + 1) >> 16);  // (exact: o < 2^11, R / 4 <= 32)
  }

  // q: results (channels n ..) of token t
  __device__ __forceinline__ void ask(const Q8LoraArgs &a, int q, int n) {
    const int e = (uint32_t)id[q] < (uint32_t)a.L ? id[q] : 0;
    scale[q] = a.scale ? a.scale[e] : 1.f;
#pragma unroll
    for (int p = 0; p < FIRST; ++p)
#pragma unroll
      for (int r = 0; r < 4; ++r) piece(w[q][p][r], row(a, e, n + r) + min(8 * p, a.R - 8));
  }
  __device__ __forceinline__ static const T *row(const Q8LoraArgs &a, int e, int n) {
    return static_cast<const T *>(a.b) + ((int64_t)e * a.N + min(n, a.N - 1)) * a.R;
  }
  __device__ __forceinline__ void ask_u(const Q8LoraArgs &a, int t0, int n) {
    const int o = threadIdx.x, t = token(a, o);
    if (t < n) part.load(a, t0 + t, 4 * o - t * a.R);
  }
  __device__ __forceinline__ void put_u(const Q8LoraArgs &a, int t0, int n, float *us) {
    for (int o = threadIdx.x; token(a, o) < n; o += NT) {
      const int t = token(a, o), r = 4 * o - t * a.R;
      if (o != (int)threadIdx.x) part.load(a, t0 + t, r);
      *reinterpret_cast<Pack<float, 4> *>(us + t * (a.R + 4) + r) = part.sum(a);
    }
  }
  __device__ __forceinline__ void add(const Q8LoraArgs &a, int q, int n, const float *u, float *d) const {
    if ((uint32_t)id[q] >= (uint32_t)a.L) return;
    float l[4] = {0.f, 0.f, 0.f, 0.f};
    auto mul = [&](int p, int r, const Pack<T, N> *x) {
#pragma unroll
      for (int k = 0; k < 8; ++k) l[r] = fmaf(u[8 * p + k], (float)x[k / N].v[k % N], l[r]);
    };
#pragma unroll
    for (int p = 0; p < FIRST; ++p)
      if (8 * p < a.R) {
#pragma unroll
        for (int r = 0; r < 4; ++r) mul(p, r, w[q][p][r]);
      }
    for (int p = FIRST; 8 * p < a.R; ++p) {
      Pack<T, N> x[4][8 / N];
#pragma unroll
      for (int r = 0; r < 4; ++r) piece(x[r], row(a, id[q], n + r) + 8 * p);
#pragma unroll
      for (int r = 0; r < 4; ++r) mul(p, r, x[r]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) d[r] = fmaf(scale[q], l[r], d[r]);
  }
};

// Bfloat16 pieces of u for a type's results.  They lie [32 positions][16 ranks]
// [piece][lane][8]: lane l has position l % 32 and ranks 8 (l / 32) .. of the 16.
constexpr int u_pieces(int dt) { return dt == COLI_F32 ? 3 : 2; }

// v as a sum of P bfloat16 pieces, each the rounding of what is left: 8 bits a
// piece and one more by the sign of the rest, so two hold 2^-18 of v, three all
// of binary32.
template <int P, int M, typename V>
__device__ __forceinline__ void split(const float *v, V *o) {
#pragma unroll
  for (int j = 0; j < M; ++j) {
    float rest = v[j];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      o[p][j] = (__bf16)rest;
      rest -= (float)o[p][j];
    }
  }
}
template <int P>
__device__ __forceinline__ void split8(const float *v, v8bf *o) {
  split<P, 8>(v, o);
}

// The adapters' part of a tile of k_q8_tile, by matrix instructions, after its
// sums: for each group of 32 tokens one adapter of the group after another.  The
// tile's tokens are in order of their adapters, so a group has few of them.  u
// comes as bfloat16 pieces, times the adapters' scales, in the order of the operand
// registers, as k_lora_down leaves it for these kernels, ranks from R to a multiple
// of 16 zero; b's rows go straight from memory to registers too (past R a row's last
// ranks again, of which the result has its part already), without LDS or a barrier.
//
// u is a binary32 sum: two bfloat16 pieces lose 2^-18 of it where the result has 8
// or 11 bits, three none.  Adapters in fp16 enter as two pieces, which hold them
// whole, in fp32 as three.
//
// A lane's results are one token's: where a group has one adapter its products go
// straight to the results, otherwise a token takes those of its own adapter and
// none of another's, whatever they hold.
template <int DT, int BM, int BN, int WM, int WN>
struct LoraTile {
  typedef typename Elem<DT>::type T;
  static constexpr int TN = BN / WN / 32;
  static constexpr int PB = DT == COLI_BF16 ? 1 : DT == COLI_F16 ? 2 : 3, PU = u_pieces(DT);
  static constexpr int N = 16 / (int)sizeof(T), H = 8 / N;  // elements and words of an eighth of ranks
  static constexpr int CS = H == 1 ? 4 : 2;                 // steps of 16 ranks asked for together

  const Q8LoraArgs &a;
  int t0, n;        // first position and tokens of the tile
  const int *rows;  // [BM] tokens
  const int *ids;   // [BM] their adapters, -1 none
  const float *chans;  // [BN] the channels' scales, then their biases

  template <int TMV>
  __device__ __forceinline__ void add(v16i (*acc)[TMV], int n0) const {
    const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int steps = (a.R + 15) / 16;
    uint32_t boff[TN];  // of this lane's rows of an adapter's b, in elements
#pragma unroll
    for (int i = 0; i < TN; ++i) boff[i] = (uint32_t)(min(n0 + (wn * TN + i) * 32 + lr, a.N - 1) - n0) * (uint32_t)a.R;
    int id[TMV];
    float st[TMV];
#pragma unroll
    for (int j = 0; j < TMV; ++j) {
      const int pos = (j * WM + wm) * 32 + lr;
      id[j] = pos < n ? ids[pos] : -1;
      st[j] = a.s[max(rows[min(pos, n - 1)], 0)];
    }
    v8bf u[CS][PU];
    auto load_u = [&](int j, int s0) {
      const v8bf *p = reinterpret_cast<const v8bf *>(a.u) + ((int64_t)((t0 / 32 + j * WM + wm) * steps + s0) * PU) * 64;
#pragma unroll
      for (int s = 0; s < CS; ++s)
        if (s0 + s < steps) {
#pragma unroll
          for (int q = 0; q < PU; ++q) u[s][q] = p[(s * PU + q) * 64 + lane];
        }
    };
#pragma unroll
    for (int j = 0; j < TMV; ++j)
      if (id[j] >= 0) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int at = (wn * TN + i) * 32 + 8 * g + 4 * lh;
            const Pack<float, 4> sn = *reinterpret_cast<const Pack<float, 4> *>(chans + at);
            const Pack<float, 4> bn = *reinterpret_cast<const Pack<float, 4> *>(chans + BN + at);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[i][j][4 * g + r] = __float_as_int(finish(acc[i][j][4 * g + r], st[j], sn.v[r], bn.v[r]));
          }
      }
    for (int s0 = 0; s0 < steps; s0 += CS) {
      Pack<T, N> b[CS][TN][H];
      int held = -1;  // the adapter whose rows are in b
#pragma unroll
      for (int j = 0; j < TMV; ++j) {
        const int g0 = (j * WM + wm) * 32;
        uint64_t todo = __ballot(id[j] >= 0);
        if (todo) load_u(j, s0);
        while (todo) {
          const int e = __builtin_amdgcn_readlane(id[j], __builtin_ctzll(todo));
          todo &= ~__ballot(id[j] == e);
          const bool whole = __ballot(g0 + lr < n && id[j] != e) == 0;
          if (e != held) {
            const T *b0 = static_cast<const T *>(a.b) + ((int64_t)e * a.N + n0) * a.R;
#pragma unroll
            for (int s = 0; s < CS; ++s)
              if (s0 + s < steps) {
                const int r = min(16 * (s0 + s) + 8 * lh, a.R - 8);
#pragma unroll
                for (int i = 0; i < TN; ++i)
#pragma unroll
                  for (int h = 0; h < H; ++h) b[s][i][h] = reinterpret_cast<const Pack<T, N> *>(b0 + boff[i] + r)[h];
              }
            held = e;
          }
#pragma unroll
          for (int i = 0; i < TN; ++i) {
            v16f l;
#pragma unroll
            for (int r = 0; r < 16; ++r) l[r] = whole ? __int_as_float(acc[i][j][r]) : 0.f;
#pragma unroll
            for (int s = 0; s < CS; ++s)
              if (s0 + s < steps) {
                v8bf w[PB];
                if constexpr (PB == 1) {
                  __builtin_memcpy(&w[0], &b[s][i][0], 16);
                } else {
                  float v[8];
#pragma unroll
                  for (int k = 0; k < 8; ++k) v[k] = (float)b[s][i][k / N].v[k % N];
                  split8<PB>(v, w);
                }
#pragma unroll
                for (int p = 0; p < PB; ++p)
#pragma unroll
                  for (int q = 0; q < PU; ++q)
                    if (p + q < (PB > PU ? PB : PU))
                      l = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[p], u[s][q], l, 0, 0, 0);
              }
            if (whole || id[j] == e) {
#pragma unroll
              for (int r = 0; r < 16; ++r)
                acc[i][j][r] = __float_as_int(whole ? l[r] : __int_as_float(acc[i][j][r]) + l[r]);
            }
          }
        }
      }
    }
  }
};

}  // namespace
}  // namespace coli
