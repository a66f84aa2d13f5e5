// lora.hpp -- the adapters' part of a product's results, as the kernels of
// the 8-bit product add it: c_a sum_r u[t][r] b_a[n][r] for token t's adapter a,
// with u [T][R] in binary32, in `slices` parts that are added in order.
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

// The adapters' part of a tile of k_q8_tile, by matrix instructions, after its
// sums.  The tile's tokens are in order of their adapters (the kernel takes them
// by `order`), so they form runs; for each run the adapter's rows of b for the
// tile's channels go through one of two buffers in LDS, the next run's on the
// way while one is multiplied, and serve all the run's tokens.  u of all the
// tile's tokens, times their adapters' scales, is put in LDS before, as bfloat16
// pieces.  Ranks go by chunks of 128 bytes of b's rows.
//
// u stays in binary32: it enters as two bfloat16 pieces (2^-18 of it is lost
// where the result has 8 or 11 bits) or three; adapters in fp16 as two, which
// hold them whole, in fp32 as three.
//
// A lane's results are one token's: where a group of 32 tokens has one adapter
// its products go straight to the results, otherwise a token takes those of its
// own adapter and none of another's, whatever they hold.
template <int DT, int BM, int BN, int WM, int WN, int LDS>
struct LoraTile {
  typedef typename Elem<DT>::type T;
  static constexpr int NW = WM * WN, TN = BN / WN / 32;
  static constexpr int PB = DT == COLI_BF16 ? 1 : DT == COLI_F16 ? 2 : 3, PU = DT == COLI_F32 ? 3 : 2;
  static constexpr int KC = 128 / (int)sizeof(T);       // ranks of a chunk
  static constexpr int UP = KC / 8;                     // 16-byte pieces of a row of u
  static constexpr int UPLANE = BM * UP * 16, BBUF = BN * 128;
  static constexpr int NL = BN * 8 / 64 / NW;           // loads of a wave for a whole chunk of b
  static constexpr int UI = BM * UP / (64 * NW);        // eighths of a chunk's rows of u for a thread
  static_assert(PU * UPLANE + 2 * BBUF <= LDS, "u and two buffers");

  const Q8LoraArgs &a;
  int n;            // tokens of the tile
  unsigned char *lds;
  const int *rows;  // [BM] tokens
  const int *ids;   // [BM] their adapters, -1 none
  const int *runs;  // first positions of the runs
  int nruns;
  const float *chans;  // [BN] the channels' scales, then their biases

  __device__ __forceinline__ static int uplace(int row, int p) {
    return (row * UP + (p ^ (UP == 8 ? row >> 1 & 7 : row >> 2 & 3))) * 16;
  }
  // place of piece p of row `row` of b, rows of pc pieces (lanes of 16 rows at one
  // p meet all banks, but with 6 pieces half of them)
  __device__ __forceinline__ static int bplace(int row, int p, int pc) {
    return row * pc + (pc == 8 ? p ^ (row >> 1 & 7) : pc == 4 ? p ^ (row >> 2 & 3) : p);
  }

  // results of token `pos` of the tile: binary32 bits in place of the sums
  __device__ __forceinline__ bool has(int pos) const { return pos < n && ids[pos] >= 0; }

  template <int TMV>
  __device__ __forceinline__ void add(v16i (*acc)[TMV], int n0) const {
    const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
#pragma unroll
    for (int j = 0; j < TMV; ++j) {
      const int pos = (j * WM + wm) * 32 + lr;
      if (!has(pos)) continue;
      const float st = a.s[max(rows[pos], 0)];
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int at = (wn * TN + i) * 32 + 8 * g + 4 * lh;
          const Pack<float, 4> sn = *reinterpret_cast<const Pack<float, 4> *>(chans + at);
          const Pack<float, 4> bn = *reinterpret_cast<const Pack<float, 4> *>(chans + BN + at);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][j][4 * g + r] = __float_as_int(finish(acc[i][j][4 * g + r], st, sn.v[r], bn.v[r]));
        }
    }
    const char *b0 = static_cast<const char *>(a.b) + (int64_t)n0 * a.R * sizeof(T);
    for (int c = 0; c < a.R; c += KC) {
      const int pc = min(8, (a.R - c) * (int)sizeof(T) / 16);
      const uint32_t magic = 65536 / pc + 1;
      uint32_t off[NL];
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int slot = ((i * NW + wave) * 64 + lane) & (BN * 8 - 1);
        const int row = (int)(slot * magic >> 16);
        off[i] = (uint32_t)(min(row, a.N - 1 - n0) * a.R + c) * (uint32_t)sizeof(T) +
                 16 * (bplace(row, slot - row * pc, pc) - row * pc);
      }
      auto load_b = [&](int k) {
        const int e = __builtin_amdgcn_readfirstlane(ids[runs[k]]);
        if (e < 0) return;
        const char *be = b0 + (int64_t)e * a.N * a.R * sizeof(T);
        unsigned char *buf = lds + PU * UPLANE + (k & 1) * BBUF;
#pragma unroll
        for (int i = 0; i < NL; ++i)
          if ((i * NW + wave) * 64 < BN * pc)
            __builtin_amdgcn_global_load_lds(be + off[i], (__attribute__((address_space(3))) void *)(buf + (i * NW + wave) * 1024),
                                             16, 0, 0);
      };
      lds_barrier();  // the sums' last operands, or the chunk before, have been read
      load_b(0);
      // u: each thread has up to UI eighths of a chunk's row
      float v[UI][8];
      int at[UI];  // position and eighth, or -1
      const float *up[UI];
#pragma unroll
      for (int i = 0; i < UI; ++i) {
        const int o = i * 64 * NW + threadIdx.x, row = o / UP, r = c + 8 * (o % UP);
        at[i] = row < n && r < ((a.R + 15) & ~15) && ids[min(row, n - 1)] >= 0 ? o : -1;
        up[i] = a.u + (int64_t)max(rows[min(row, n - 1)], 0) * a.R + min(r, a.R - 8);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
      }
      for (int s = 0; s < a.slices; ++s) {
        Pack<float, 4> x[UI][2];
#pragma unroll
        for (int i = 0; i < UI; ++i)
          if (at[i] >= 0) {
            x[i][0] = reinterpret_cast<const Pack<float, 4> *>(up[i])[0];
            x[i][1] = reinterpret_cast<const Pack<float, 4> *>(up[i])[1];
          }
#pragma unroll
        for (int i = 0; i < UI; ++i) {
          up[i] += (int64_t)a.rows * a.R;
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][k] += x[i][k / 4].v[k % 4];
        }
      }
#pragma unroll
      for (int i = 0; i < UI; ++i) {
        if (at[i] < 0) continue;
        const int row = at[i] / UP, p = at[i] % UP;
        const float f = a.scale ? a.scale[ids[row]] : 1.f;
        v8bf u[PU];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = c + 8 * p < a.R ? f * v[i][k] : 0.f;
        split8<PU>(v[i], u);
#pragma unroll
        for (int q = 0; q < PU; ++q) *reinterpret_cast<v8bf *>(lds + q * UPLANE + uplace(row, p)) = u[q];
      }
      for (int k = 0; k < nruns; ++k) {
        lds_barrier();  // this run's rows are there, and the run before has been multiplied
        if (k + 1 < nruns) load_b(k + 1);
        const int p0 = __builtin_amdgcn_readfirstlane(runs[k]);
        const int p1 = k + 1 < nruns ? __builtin_amdgcn_readfirstlane(runs[k + 1]) : n;
        if (__builtin_amdgcn_readfirstlane(ids[p0]) < 0) continue;
        const unsigned char *buf = lds + PU * UPLANE + (k & 1) * BBUF;
        const int steps = (min(KC, a.R - c) + 15) / 16;
#pragma unroll
        for (int j = 0; j < TMV; ++j) {
          const int g0 = (j * WM + wm) * 32;
          if (g0 >= p1 || g0 + 32 <= p0) continue;
          const bool whole = p0 <= g0 && (p1 >= g0 + 32 || p1 == n);
          const bool mine = g0 + lr >= p0 && g0 + lr < p1;
#pragma unroll
          for (int i = 0; i < TN; ++i) {
            v16f l;
#pragma unroll
            for (int r = 0; r < 16; ++r) l[r] = whole ? __int_as_float(acc[i][j][r]) : 0.f;
            for (int s = 0; s < steps; ++s) {
              v8bf u[PU], w[PB];
#pragma unroll
              for (int q = 0; q < PU; ++q)
                u[q] = *reinterpret_cast<const v8bf *>(lds + q * UPLANE + uplace(g0 + lr, 2 * s + lh));
              operand_b(buf, (wn * TN + i) * 32 + lr, 2 * s + lh, pc, c + 16 * s + 8 * lh < a.R, w);
#pragma unroll
              for (int p = 0; p < PB; ++p)
#pragma unroll
                for (int q = 0; q < PU; ++q)
                  if (p + q < (PB > PU ? PB : PU))
                    l = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[p], u[q], l, 0, 0, 0);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r)
              acc[i][j][r] = whole  ? __float_as_int(l[r])
                             : mine ? __float_as_int(__int_as_float(acc[i][j][r]) + l[r])
                                    : acc[i][j][r];
          }
        }
      }
    }
  }

  // ranks 8 p .. 8 p + 7 of the chunk of row `row` of b, zero if not `in`
  __device__ __forceinline__ static void operand_b(const unsigned char *buf, int row, int p, int pc, bool in,
                                                   v8bf *w) {
    if constexpr (PB == 1) {
      w[0] = *reinterpret_cast<const v8bf *>(buf + 16 * bplace(row, p, pc));
#pragma unroll
      for (int k = 0; k < 8; ++k) w[0][k] = in ? w[0][k] : (__bf16)0.f;
    } else {
      constexpr int N = 16 / (int)sizeof(T);
      float v[8];
#pragma unroll
      for (int h = 0; h < 8 / N; ++h) {
        const Pack<T, N> x = *reinterpret_cast<const Pack<T, N> *>(buf + 16 * bplace(row, 8 / N * p + h, pc));
#pragma unroll
        for (int k = 0; k < N; ++k) v[h * N + k] = in ? (float)x.v[k] : 0.f;
      }
      split8<PB>(v, w);
    }
  }

  // s_waitcnt vmcnt(0) lgkmcnt(0) and a barrier.
  __device__ __forceinline__ static void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(7 << 4);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
};

}  // namespace
}  // namespace coli
