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
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));

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

// Bfloat16 pieces of u for a type's results.  They lie [32 positions][16 ranks]
// [piece][lane][8]: lane l has position l % 32 and ranks 8 (l / 32) .. of the 16.
constexpr int u_pieces(int dt) { return dt == COLI_F32 ? 3 : 2; }

// v as a sum of P bfloat16 pieces, each the rounding of what is left, by at most half a
// step of its 8 bits: one leaves up to 2^-8 of v, two 2^-17, three nothing of binary32.
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

// Bfloat16 pieces of an adapter's element: fp16's 11 bits are two whole, fp32's 24
// three.
constexpr int b_pieces(int dt) { return dt == COLI_BF16 ? 1 : dt == COLI_F16 ? 2 : 3; }

// Whether piece k of b's element is multiplied by piece m of u.  What is left out is up
// to 2^-24 of the product in fp32 (k + m = 3: 2^-8 of one by 2^-17 of the other, twice)
// and nothing in fp16, whose two low pieces would be 2^-16.
constexpr bool pieces_meet(int k, int m) { return k + m < 3; }

// The operand of ranks 8 p .. 8 p + 7 of a row of b in LDS, whose 16-byte piece h
// lies at place(h); zero if not `in`.
template <int DT, typename F>
__device__ __forceinline__ void b_operand(const unsigned char *row, F place, int p, bool in, v8bf *w) {
  typedef typename Elem<DT>::type T;
  constexpr int N = 16 / (int)sizeof(T);
  if constexpr (b_pieces(DT) == 1) {
    w[0] = *reinterpret_cast<const v8bf *>(row + place(p));
    w[0] = in ? w[0] : v8bf{};
  } else {
    float v[8];
#pragma unroll
    for (int h = 0; h < 8 / N; ++h) {
      const Pack<T, N> x = *reinterpret_cast<const Pack<T, N> *>(row + place(8 / N * p + h));
#pragma unroll
      for (int k = 0; k < N; ++k) v[h * N + k] = in ? (float)x.v[k] : 0.f;
    }
    split8<b_pieces(DT)>(v, w);
  }
}

// Adds the adapters' part to the biases of the 16 x 16 results that a wave of
// k_q8_ring finishes, by matrix instructions.  With few tokens nearly every one has
// an adapter of its own, and the work is reading it: each wave brings the rows of b
// for its 16 channels of one adapter of its 16 tokens after another, which lie
// together, as whole lines into LDS of its own, D of them on the way, without a
// barrier.  (300 tokens x 4000 channels x 6144 with 64 adapters of rank 16, 64 and
// 128: 40, 51 and 72 us for both launches, with each lane reading its own token's
// rows into registers 45, 97 and 159; the product's alone 28, 37 and 48.  Asking for
// the rows' lines while the sums are still made does not help: 28, 37 and 55 us
// instead of 28, 33 and 46 at 61 x 6144.)
// u's parts are added, cut into bfloat16 pieces and put in LDS for all the waves
// before.  Ranks go by chunks of 128 bytes of b's rows.  Lane (li, lg) has channels 4
// lg .. of token li, and takes its own adapter's results and no other's, whatever
// they hold.
template <int DT, int BM, int NT, int TPW, int LDS>
struct LoraRing {
  typedef typename Elem<DT>::type T;
  static constexpr int PB = b_pieces(DT), PU = u_pieces(DT);
  static constexpr int KC = 128 / (int)sizeof(T), UP = KC / 8;  // ranks of a chunk, and eighths of them
  static constexpr int UPLANE = BM * UP * 16;
  static constexpr int ROOM = (LDS - PU * UPLANE) / (NT / 64) / 1024;  // KB of b for a wave
  int id[TPW];
  float scale[TPW], sum[TPW][4];
  UParts<lora_parts(BM)> part;

  __device__ __forceinline__ static int uplace(int row, int p) {
    return (row * UP + (p ^ (UP == 8 ? row >> 1 & 7 : row >> 2 & 3))) * 16;
  }
  // place of piece p of row `row` of b, rows of pc pieces of 16 bytes
  __device__ __forceinline__ static int bplace(int row, int p, int pc) {
    return row * pc + (pc == 8 ? p ^ (row >> 1 & 7) : pc == 4 ? p ^ (row >> 2 & 3) : p);
  }

  // this thread's first share of u, asked for ahead
  __device__ __forceinline__ void ask_u(const Q8LoraArgs &a, const int *rows, int n) {
    const int t = threadIdx.x / (KC / 4), r = threadIdx.x % (KC / 4) * 4;
    if (t < n && r < a.R) part.load(a, max(rows[t], 0), r);
#pragma unroll
    for (int q = 0; q < TPW; ++q) {
      scale[q] = a.scale && (uint32_t)id[q] < (uint32_t)a.L ? a.scale[id[q]] : 1.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[q][k] = 0.f;
    }
  }
  // u's pieces of the chunk from rank c on, zero from R to a multiple of 32
  __device__ __forceinline__ void put_u(const Q8LoraArgs &a, const int *rows, int n, int c, unsigned char *lds) {
    for (int o = threadIdx.x; o < n * (KC / 4); o += NT) {
      const int t = o / (KC / 4), r = c + o % (KC / 4) * 4;
      if (r >= ((a.R + 31) & ~31)) continue;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < a.R) {
        if (c > 0 || o != (int)threadIdx.x) part.load(a, max(rows[t], 0), r);
        const Pack<float, 4> s = part.sum(a);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = s.v[k];
      }
      v4bf u[PU];
      split<PU, 4>(v, u);
#pragma unroll
      for (int p = 0; p < PU; ++p)
        *reinterpret_cast<v4bf *>(lds + p * UPLANE + uplace(t, (r - c) / 8) + r % 8 * 2) = u[p];
    }
  }
  // Results q: 16 channels from n on, tokens row .. row + 15 of the tile.  An
  // adapter's rows are NI KB.  G adapters are multiplied together, so that one's
  // wait for LDS is the other's too, and D are on the way.
  template <int NI>
  __device__ __forceinline__ void mul(const Q8LoraArgs &a, int q, int row, int n, int c, unsigned char *lds) {
    // (as many as leave the registers for two workgroups a CU)
    constexpr int FIT = ROOM / NI, MOST = NT <= 256 ? 4 : TPW > 1 || PB > 1 ? 2 : 3;
    constexpr int G = FIT / 2 < MOST ? FIT / 2 : MOST, D = FIT / G < 3 ? FIT / G * G : 3 * G;
    static_assert(G >= 1 && D >= 2 * G && (D - G) * NI < 16, "buffers of b");
    const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int pc = min(8, (a.R - c) * (int)sizeof(T) / 16);
    uint32_t off[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int slot = min(i * 64 + lane, 16 * pc - 1), r = slot * (65536 / pc + 1) >> 16;
      off[i] = (uint32_t)(min(n + r, a.N - 1) - n) * (uint32_t)a.R * (uint32_t)sizeof(T) +
               16 * (bplace(r, slot - r * pc, pc) - r * pc);
    }
    const char *b0 = static_cast<const char *>(a.b) + ((int64_t)n * a.R + c) * (int64_t)sizeof(T);
    unsigned char *mine = lds + PU * UPLANE + wave * ROOM * 1024;
    const uint32_t tokens = (uint32_t)__ballot((uint32_t)id[q] < (uint32_t)a.L) & 0xFFFF;
    uint32_t ask = tokens, todo = tokens;
    auto next = [&](uint32_t &m) {  // the first token's adapter; its tokens leave m
      const int e = __builtin_amdgcn_readlane(id[q], __builtin_ctz(m));
      m &= ~(uint32_t)__ballot(id[q] == e);
      return e;
    };
    auto issue = [&](int to) {
      const char *p = b0 + (int64_t)next(ask) * a.N * a.R * (int64_t)sizeof(T);
#pragma unroll
      for (int i = 0; i < NI; ++i)
        __builtin_amdgcn_global_load_lds(p + off[i], (__attribute__((address_space(3))) void *)(mine + (to * NI + i) * 1024),
                                         16, 0, 0);
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (ask) issue(d);
    const int steps = (min(KC, a.R - c) + 31) / 32;
    for (int at = 0; todo; at = at + G == D ? 0 : at + G) {
      // the oldest G are there: all but the others' loads have come
      if (ask) lds_wait<(D - G) * NI>();
      else lds_wait<0>();
      int e[G];
      v4f l[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        e[g] = todo ? next(todo) : -1;
        l[g] = v4f{0.f, 0.f, 0.f, 0.f};
      }
      const unsigned char *buf = mine + at * NI * 1024;
      for (int s = 0; s < steps; ++s) {
        const int p = 4 * s + lg;
        v8bf u[PU], w[G][PB];
#pragma unroll
        for (int k = 0; k < PU; ++k)
          u[k] = *reinterpret_cast<const v8bf *>(lds + k * UPLANE + uplace(row + li, p));
#pragma unroll
        for (int g = 0; g < G; ++g)
          b_operand<DT>(buf + g * NI * 1024, [&](int h) { return 16 * bplace(li, h, pc); }, p, c + 8 * p < a.R, w[g]);
#pragma unroll
        for (int k = 0; k < PB; ++k)
#pragma unroll
          for (int m = 0; m < PU; ++m)
            if (pieces_meet(k, m))
#pragma unroll
              for (int g = 0; g < G; ++g)
                l[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[g][k], u[m], l[g], 0, 0, 0);
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (e[g] >= 0 && id[q] == e[g]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) sum[q][k] += l[g][k];
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the buffers have been read
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (ask) issue(at + g);
    }
  }
  // s_waitcnt vmcnt(N)
  template <int N>
  __device__ __forceinline__ static void lds_wait() {
    static_assert(N >= 0 && N < 16, "vmcnt");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
  }

  // lds may hold what other waves have still to read until the first barrier
  template <typename ROW, typename CHANNEL>
  __device__ __forceinline__ void add(const Q8LoraArgs &a, const int *rows, int n, ROW row, CHANNEL channel, unsigned char *lds,
                                      float (*d)[4]) {
    for (int c = 0; c < a.R; c += KC) {
      __syncthreads();
      put_u(a, rows, n, c, lds);
      __syncthreads();
#pragma unroll
      for (int q = 0; q < TPW; ++q) {
        if (row(q) < 0 || row(q) >= n || channel(q) >= a.N) continue;
        if ((a.R - c) * (int)sizeof(T) <= 64) mul<1>(a, q, row(q), channel(q), c, lds);
        else mul<2>(a, q, row(q), channel(q), c, lds);
      }
    }
#pragma unroll
    for (int q = 0; q < TPW; ++q)
      if ((uint32_t)id[q] < (uint32_t)a.L) {
#pragma unroll
        for (int k = 0; k < 4; ++k) d[q][k] = fmaf(scale[q], sum[q][k], d[q][k]);
      }
  }
};

// The adapters' part of a tile of k_q8_tile, by matrix instructions, after its
// sums: for each group of 32 tokens one adapter of the group after another.  The
// tile's tokens are in order of their adapters, so a group has few of them.  u
// comes as bfloat16 pieces, times the adapters' scales, in the order of the operand
// registers, as k_lora_down leaves it for these kernels, ranks from R to a multiple
// of 16 zero; b's rows go straight from memory to registers too (past R a row's last
// ranks again, of which the result has its part already), without LDS or a barrier.
//
// u is a binary32 sum: two bfloat16 pieces lose up to 2^-17 of it where the result has 8
// or 11 bits, three none.  Adapters in fp16 enter as two pieces, which hold them
// whole, in fp32 as three.
//
// A lane's results are one token's: it takes those of its token's adapter and none of
// another's, whatever they hold.  The products of up to CS steps are summed by
// themselves and then added, one rounding at the result's size for 64 (bfloat16) or
// 32 ranks.  (Products that go straight to the results round there in every matrix
// instruction, 3 R / 8 of them in binary32: parts of an adapter that lie below half a
// step of a large result were lost one by one.)
//
// 8192 x 6144 x 6144, the product's launch alone: 288 us where no token has an
// adapter, 292 with one of rank 16, 301 with eight of rank 64, 322 with sixteen of
// rank 128 (least of 24).  Each adapter of a group costs a wait for its rows, so
// where a group has many they are what it waits for: 509 x 6144 x 6144 of rank 16 38
// us with one, 45 with 64 in any order, of rank 64 56.
template <int DT, int BM, int BN, int WM, int WN>
struct LoraTile {
  typedef typename Elem<DT>::type T;
  static constexpr int TN = BN / WN / 32;
  static constexpr int PB = b_pieces(DT), PU = u_pieces(DT);
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
        uint64_t todo = __ballot(id[j] >= 0);
        if (todo) load_u(j, s0);
        while (todo) {
          const int e = __builtin_amdgcn_readlane(id[j], __builtin_ctzll(todo));
          todo &= ~__ballot(id[j] == e);
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
            for (int r = 0; r < 16; ++r) l[r] = 0.f;
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
                    if (pieces_meet(p, q))
                      l = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[p], u[s][q], l, 0, 0, 0);
              }
            if (id[j] == e) {
#pragma unroll
              for (int r = 0; r < 16; ++r) acc[i][j][r] = __float_as_int(__int_as_float(acc[i][j][r]) + l[r]);
            }
          }
        }
      }
    }
  }
};

}  // namespace
}  // namespace coli
