// q8_gemm.hip -- the matrix product in 8-bit integers with one scale per
// token and one per output channel, dense and over experts:
//   y[t][n] = s_t * ws_n * sum_k q[t][k] w[n][k]  (+ bias[n]).
//
// Unlike a product against Q8_0 blocks, no scale changes along k, so the
// whole sum stays in the int32 accumulators of the matrix instructions and
// is exact for K < 2^17 (128 * 128 * K < 2^31); one conversion and two
// multiplications in binary32 (the second fused with the bias's addition)
// finish it, and a rounding to y's type.  Exact sums also make every split
// of k, and so every kernel below, give the same bits.
//
// Both operands are contiguous along k, which is what the instructions take:
// v_mfma_i32_32x32x32_i8 reads 16 consecutive bytes of row (lane % 32) at
// k = 16 (lane / 32), v_mfma_i32_16x16x64_i8 of row (lane % 16) at
// k = 16 (lane / 16).  Weight rows are the A operand and tokens the B
// operand, so a lane's results are one token's consecutive channels.
//
// Three kernels:
//   k_q8_ring   few tokens: bound by reading the weights, with k split over
//               the waves so that few channels still fill the chip.
//   k_q8_sweep  few tokens per expert, many weights: bound by reading them
//               from memory, straight into operand registers.
//   k_q8_tile   many tokens: bound by the matrix cores.  Large tiles, each
//               operand read from LDS once for several products.
#include <type_traits>

#include "q8.hpp"

#pragma clang fp contract(off)

namespace coli {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

// ---------------------------------------------------------------------------
// The tokens of one tile.  Dense: rows r0 .. r0 + n - 1 of both q and y.
// Grouped: positions of one expert's range of perm; each names a pair, whose
// row of q is pair / fan and whose row of y is the pair.  Table entries
// outside the buffers are never followed: such a position reads row 0 and
// writes nothing.
// ---------------------------------------------------------------------------
struct Tile {
  int e;      // expert (0 in the dense product)
  int r0, n;  // first position, positions in the tile
  int nb;     // block of output channels
};

template <bool GROUPED>
__device__ __forceinline__ int out_row(const Q8Args &a, int pos) {
  if constexpr (GROUPED) {
    const int p = a.perm[pos];
    return (uint32_t)p < (uint32_t)a.P && p / a.fan < a.rows ? p : -1;
  } else {
    return pos;
  }
}
template <bool GROUPED>
__device__ __forceinline__ int in_row(const Q8Args &a, int out) {
  if constexpr (GROUPED) return out < 0 ? 0 : out / a.fan;
  else return out;
}

// Keeps what is before it before what is after it.  The waits below count the
// loads issued since the one that is waited for, so loads of one stage must
// not be moved past those of another.
__device__ __forceinline__ void keep_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Workgroup b runs on XCD b % 8, each with its own L2: an XCD takes a
// contiguous run of the `total` items, so that neighbours share it.
__device__ __forceinline__ int xcd_item(int b, int total) {
  const int per = (total + 7) / 8;
  const int i = (b % 8) * per + b / 8;
  return b / 8 < per && i < total ? i : -1;
}

// The grouped product's tile of this workgroup among (expert, channel block,
// token tile).  Each wave sums the experts' tile counts itself (E <= 1024, at
// most 16 a lane, all loaded at once), so no table and no extra launch is
// needed.  The grid is the host's bound; workgroups past the experts' tiles
// get t.n = 0.  Token tiles of one expert and channel block are neighbours, so
// that their weights are read from memory once.
template <int BM, int EPL>
__device__ __forceinline__ Tile expert_tile_n(const Q8Args &a, int nbn) {
  const int lane = threadIdx.x & 63;
  const int per = (a.E + 63) / 64;
  const int lo = lane * per;
  int o[EPL + 1];
#pragma unroll
  for (int i = 0; i <= EPL; ++i)
    if (i <= per) o[i] = a.offs[min(lo + i, a.E)];
  // (offs that are no running sum could count more tiles than there are)
  const int bound = a.P / BM + min(a.P, a.E);
  int mine = 0;
#pragma unroll
  for (int i = 0; i <= EPL; ++i)
    if (i <= per) {
      o[i] = min(max(o[i], 0), a.P);
      if (i > 0 && o[i] > o[i - 1]) mine += (o[i] - o[i - 1] + BM - 1) / BM;
    }
  mine = min(mine, bound);
  // inclusive sum over the lanes: row shifts by 1, 2, 4, 8, then rows' totals
  int sum = mine;
  sum += dpp_i32<0x111>(sum);
  sum += dpp_i32<0x112>(sum);
  sum += dpp_i32<0x114>(sum);
  sum += dpp_i32<0x118>(sum);
  sum += dpp_i32<0x142, 0xA>(sum);
  sum += dpp_i32<0x143, 0xC>(sum);
  const int total = min(__builtin_amdgcn_readlane(sum, 63), bound);
  const int id = xcd_item(blockIdx.x, total * nbn);
  Tile t{0, 0, 0, 0};
  if (id < 0) return t;
  int before = sum - mine;
  bool found = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (i < per) {
      const int n = o[i + 1] - o[i], mt = n > 0 ? (n + BM - 1) / BM : 0;
      const int64_t local = id - (int64_t)before * nbn;
      if (!found && local >= 0 && local < (int64_t)mt * nbn) {
        found = true;
        const int l = (int)local, nb = mt == 1 ? l : l / mt, m = l - nb * mt;
        t = Tile{lo + i, o[i] + m * BM, min(BM, n - m * BM), nb};
      }
      before += mt;
    }
  const uint64_t who = __ballot(found);
  if (!who) return Tile{0, 0, 0, 0};
  const int owner = __builtin_ctzll(who);
  t.e = __builtin_amdgcn_readlane(t.e, owner);
  t.r0 = __builtin_amdgcn_readlane(t.r0, owner);
  t.n = __builtin_amdgcn_readlane(t.n, owner);
  t.nb = __builtin_amdgcn_readlane(t.nb, owner);
  return t;
}

template <int BM>
__device__ __forceinline__ Tile expert_tile(const Q8Args &a, int nbn) {
  return a.E <= 256 ? expert_tile_n<BM, 4>(a, nbn) : expert_tile_n<BM, 16>(a, nbn);
}

// y's element from the exact sum.  (The product of two small scales could be
// subnormal where the result is not, so the sum comes first.  The last
// product and the bias's addition are one rounding by the source's own word,
// not by the compiler's choice in each kernel.  To fp16 they are one
// instruction, which rounds the exact value straight to fp16.)
__device__ __forceinline__ float finish(int acc, float st, float sn, float b) {
  return __builtin_fmaf((float)acc * sn, st, b);
}

// s_waitcnt vmcnt(N) lgkmcnt(0) and a barrier.
template <int N>
__device__ __forceinline__ void stage_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// Few tokens.  A workgroup takes up to BM tokens and BN channels: WM x WN
// waves share them out, and KS such sets share out k, whose exact partial
// sums are added through LDS at the end.  k goes by stages of 256 bytes of
// every row through a ring of STAGES in LDS, filled by direct loads, of which
// all but the one being multiplied are in flight; one barrier a stage both
// publishes the oldest and frees the one before it.
//
// Loads of whole 256-byte runs of rows are what this kernel is about: read
// straight into operand registers (64 bytes of 16 rows an instruction) the
// tokens' codes cost more than the weights from 16 tokens on (1.25 times as
// long at 1 token of 6144 x 6144, 1.4 at 16, 1.9 at 61).  6144 x 6144, launches
// one after another, with 18 matrices in turn, which come from memory: 1 token
// 9.9 us, 16 tokens 10.7, 61 tokens 15.6; with one, which stays in the Infinity
// Cache: 9.2, 9.7, 11.6.  Bound by latency: 37.7 MB from memory take 6.3 us.
//
// LDS: a row's stage is 16 pieces of 16 bytes, piece p of row r at place p ^
// (r % 16): 16 lanes that read 16 rows at one k meet all 64 banks.
// ---------------------------------------------------------------------------
constexpr int kRingBytes = 256;
constexpr int kRingPieces = kRingBytes / 16;

template <int DT, int BM, int BN, int WM, int WN, int KS, int STAGES, bool GROUPED>
struct RingKernel {
  typedef typename Elem<DT>::type T;
  static constexpr int NW = WM * WN * KS;
  static constexpr int ROWS = BM + BN;
  static constexpr int NL = ROWS / 4 / NW;  // loads of a wave in a stage (4 rows each)
  static constexpr int STAGE = ROWS * kRingBytes;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
  static constexpr int STEPS = 4 / KS;      // steps of k = 64 of a wave in a stage
  static constexpr int PART = KS * BM * BN * 4;
  static constexpr int LDS = STAGES * STAGE > PART ? STAGES * STAGE : PART;
  static_assert(ROWS % (4 * NW) == 0 && BM % 4 == 0 && 4 % KS == 0, "whole loads and steps");

  __device__ __forceinline__ static void run(const Q8Args &a, const Tile &t, unsigned char *ring,
                                             const int *rows) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int wm = wave % WM, wn = (wave / WM) % WN, kq = wave / (WM * WN);
    const int n0 = t.nb * BN;
    const int pieces = a.K / 16, full = pieces / kRingPieces;
    const int stages = (pieces + kRingPieces - 1) / kRingPieces;

    // this lane's source of each load: row 4 (i NW + wave) + lane / 16
    // (tokens first), piece (lane % 16) ^ (row % 16)
    const uint8_t *src[NL];
    uint32_t pl[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int r = (i * NW + wave) * 4 + lane / 16;
      pl[i] = (lane & 15) ^ (r & 15);
      if ((i * NW + wave) * 4 < BM) {
        const int tt = min(r, t.n - 1);
        const int row = GROUPED ? in_row<GROUPED>(a, rows[tt]) : t.r0 + tt;
        src[i] = reinterpret_cast<const uint8_t *>(a.q) + (size_t)row * a.K;
      } else {
        src[i] = a.w + ((size_t)t.e * a.N + min(n0 + r - BM, a.N - 1)) * a.K;
      }
    }
    auto issue = [&](int c) {
      unsigned char *buf = ring + (c % STAGES) * STAGE;
      const uint32_t last = c < full ? kRingPieces - 1 : (uint32_t)(pieces - kRingPieces * c - 1);
#pragma unroll
      for (int i = 0; i < NL; ++i)
        __builtin_amdgcn_global_load_lds(src[i] + (size_t)c * kRingBytes + 16 * min(pl[i], last),
                                         (lds_void *)(buf + (i * NW + wave) * 1024), 16, 0, 0);
    };

    // The scales and biases of the 16 x 16 results this wave will finish, so
    // that nothing is waited for after the last product: lane (li, lg) has
    // token li and channels 4 lg .. of each.
    constexpr int TILES = (BM / 16) * (BN / 16), TPW = (TILES + NW - 1) / NW;
    float st[TPW], sn[TPW][4], bn[TPW][4];
    int orow[TPW];  // -1: none
#pragma unroll
    for (int q = 0; q < TPW; ++q) {
      const int tl = min(q * NW + wave, TILES - 1);
      const int tt = min((tl / (BN / 16)) * 16 + li, t.n - 1), n = n0 + (tl % (BN / 16)) * 16 + 4 * lg;
      orow[q] = GROUPED ? rows[tt] : t.r0 + tt;
      st[q] = a.s[in_row<GROUPED>(a, orow[q])];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int nr = min(n + r, a.N - 1);
        sn[q][r] = a.ws[(size_t)t.e * a.N + nr];
        bn[q][r] = a.bias ? a.bias[nr] : 0.f;
      }
    }
    keep_order();

    v4i acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = v4i{0, 0, 0, 0};

    // step s (k = 64 s ..) of a stage; a part stage's pieces past the row's
    // end count as zero weights
    auto step = [&](const unsigned char *buf, int s, int left) {
      const int p = 4 * s + lg;
      v4i x[TM], w[TN];
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int r = (wm * TM + j) * 16 + li;
        x[j] = *reinterpret_cast<const v4i *>(buf + r * kRingBytes + 16 * (p ^ li));
      }
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const int r = BM + (wn * TN + i) * 16 + li;
        w[i] = *reinterpret_cast<const v4i *>(buf + r * kRingBytes + 16 * (p ^ li));
        if (left < kRingPieces) w[i] = p < left ? w[i] : v4i{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i], x[j], acc[i][j], 0, 0, 0);
    };

#pragma unroll
    for (int c = 0; c < STAGES - 1; ++c) {
      if (c < stages) issue(c);
      keep_order();
    }
    for (int c = 0; c < stages; ++c) {
      // stage c has landed for every wave, and no wave reads stage c - 1 any more
      if (c + STAGES - 1 <= stages) stage_barrier<NL *(STAGES - 2)>();
      else stage_barrier<0>();
      if (c + STAGES - 1 < stages) issue(c + STAGES - 1);
      const unsigned char *buf = ring + (c % STAGES) * STAGE;
      if (c < full) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) step(buf, kq * STEPS + s, kRingPieces);
      } else {
        const int left = pieces - kRingPieces * c;
        for (int s = 0; s < STEPS; ++s)
          if (4 * (kq * STEPS + s) < left) step(buf, kq * STEPS + s, left);
      }
    }

    stage_barrier<0>();
    int *part = reinterpret_cast<int *>(ring);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int tl = (wm * TM + j) * (BN / 16) + wn * TN + i;
        *reinterpret_cast<v4i *>(part + (kq * TILES + tl) * 256 + 4 * lane) = acc[i][j];
      }
    __syncthreads();
    T *y = static_cast<T *>(a.y);
    const bool vec = reinterpret_cast<uintptr_t>(a.y) % (4 * sizeof(T)) == 0 && a.ldy % 4 == 0;
#pragma unroll
    for (int q = 0; q < TPW; ++q) {
      const int tl = q * NW + wave;
      const int tt = (tl / (BN / 16)) * 16 + li, n = n0 + (tl % (BN / 16)) * 16 + 4 * lg;
      if (tl >= TILES || tt >= t.n || n >= a.N || orow[q] < 0) continue;
      v4i sum = *reinterpret_cast<const v4i *>(part + tl * 256 + 4 * lane);
#pragma unroll
      for (int k = 1; k < KS; ++k)
        sum += *reinterpret_cast<const v4i *>(part + (k * TILES + tl) * 256 + 4 * lane);
      Pack<T, 4> v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v.v[r] = (T)finish(sum[r], st[q], sn[q][r], bn[q][r]);
      T *d = y + (int64_t)orow[q] * a.ldy + n;
      if (vec && n + 4 <= a.N) {
        *reinterpret_cast<Pack<T, 4> *>(d) = v;
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < a.N) d[r] = v.v[r];
      }
    }
  }
};

template <int DT, int BM, int BN, int WM, int WN, int KS, int STAGES, bool GROUPED>
__global__ __launch_bounds__(64 * WM * WN * KS) void k_q8_ring(Q8Args a, int nbm, int nbn) {
  typedef RingKernel<DT, BM, BN, WM, WN, KS, STAGES, GROUPED> K;
  __shared__ __align__(16) unsigned char ring[K::LDS];
  __shared__ int rows[GROUPED ? BM : 1];
  Tile t;
  if constexpr (GROUPED) {
    t = expert_tile<BM>(a, nbn);
    if (t.n <= 0) return;
    if (threadIdx.x < t.n) rows[threadIdx.x] = out_row<GROUPED>(a, t.r0 + threadIdx.x);
    __syncthreads();
  } else {
    const int id = xcd_item(blockIdx.x, nbm * nbn);
    if (id < 0) return;
    const int m = id % nbm;  // the token tiles of a channel block are neighbours
    t = Tile{0, m * BM, min(BM, a.rows - m * BM), id / nbm};
  }
  K::run(a, t, ring, rows);
}

// ---------------------------------------------------------------------------
// Weights once through, for as many tokens as they are read for (up to BM).
// A workgroup of NW waves takes 32 NW channels; each wave has 32 of them for
// itself, so their weights need no LDS: they go from memory to operand
// registers, D chunks of 128 bytes of k ahead.  The registers of a CU hold
// several times what its LDS does, and that many bytes have to be in flight
// for the full rate of the memory.  The tokens' codes, which all waves use,
// go through a ring of D + 1 chunks in LDS as in the other kernels, with one
// barrier a chunk.
//
// The products are 16 x 16 x 64, MT groups of 16 tokens (as many as the tile
// has tokens for) by two of 16 channels for each wave.
//
// Bound by the memory: 24 experts of 4096 x 6144 with a token each 104-109 us,
// 5.5-5.8 TB/s (a plain read reaches 6.0); 64 experts of 6144 x 2048 with 31
// tokens 162-171 us, 4.7-5.0 TB/s.  Workgroups of few waves, several to a CU,
// hide one another's start and end (eight waves with 64 tokens take 1.17 times
// as long).
// ---------------------------------------------------------------------------
template <int DT, int BM, int NW, int D, bool GROUPED>
struct SweepKernel {
  typedef typename Elem<DT>::type T;
  static constexpr int BN = 32 * NW;
  static constexpr int SB = 128, PPR = 8;
  static constexpr int RINGB = (D + 1) * BM * SB;
  static constexpr int ROWB = BN * (int)sizeof(T);       // a row of the result area
  static constexpr int AREAB = 16 * ROWB;
  static constexpr int LDS = RINGB > AREAB ? RINGB : AREAB;
  __device__ __forceinline__ static int key(int r) { return (r >> 1) & 7; }

  const Q8Args &a;
  const Tile &t;
  unsigned char *ring;
  const int *rows;

  template <int MT>
  __device__ __forceinline__ void run() {
    constexpr int LW = 4;                              // weight loads of a wave in a chunk
    constexpr int LX = (2 * MT + NW - 1) / NW;         // token loads of a wave (8 rows each)
    constexpr int XB = 16 * MT * SB;
    static_assert(D * (LX + LW) < 64, "vmcnt range");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int n0 = t.nb * BN;
    const int pieces = a.K / 16, full = pieces / PPR, chunks = (pieces + PPR - 1) / PPR;

    const uint8_t *xb = reinterpret_cast<const uint8_t *>(a.q) + (GROUPED ? 0 : (size_t)t.r0 * a.K);
    const uint8_t *wb = a.w + ((size_t)t.e * a.N + n0) * a.K;
    uint32_t xoff[LX], xpl[LX], woff[2];
    // (waves past the last group of 8 rows load that group again)
    auto xgroup = [&](int i) { return min(i * NW + wave, 2 * MT - 1); };
#pragma unroll
    for (int i = 0; i < LX; ++i) {
      const int r = 8 * xgroup(i) + lane / 8, tt = min(r, t.n - 1);
      xpl[i] = (lane & 7) ^ key(r);
      xoff[i] = (uint32_t)(GROUPED ? in_row<GROUPED>(a, rows[tt]) : tt) * (uint32_t)a.K;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      woff[i] = (uint32_t)min(32 * wave + 16 * i + li, a.N - 1 - n0) * (uint32_t)a.K + 16 * lg;

    auto issue = [&](int c) {
      unsigned char *buf = ring + (c % (D + 1)) * XB;
      uint64_t xc = reinterpret_cast<uint64_t>(xb) + (uint64_t)c * SB;
      asm("" : "+s"(xc));
      const uint32_t last = c < full ? PPR - 1 : (uint32_t)(pieces - PPR * c - 1);
#pragma unroll
      for (int i = 0; i < LX; ++i)
        __builtin_amdgcn_global_load_lds(reinterpret_cast<const uint8_t *>(xc) + (xoff[i] + 16 * min(xpl[i], last)),
                                         (lds_void *)(buf + xgroup(i) * 1024), 16, 0, 0);
    };
    v4i w[D][2][2];  // [chunk][k half][channel group]
    auto load = [&](v4i (*v)[2], int c) {
      uint64_t wc = reinterpret_cast<uint64_t>(wb) + (uint64_t)c * SB;
      asm("" : "+s"(wc));
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v[h][i] = *reinterpret_cast<const v4i *>(reinterpret_cast<const uint8_t *>(wc) + woff[i] + 64 * h);
    };
    // the part chunk: pieces past the row's end count as zero weights
    auto load_part = [&](v4i (*v)[2], int c) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int p = PPR * c + 4 * h + lg;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const v4i x = *reinterpret_cast<const v4i *>(wb + woff[i] - 16 * lg + 16 * (size_t)min(p, pieces - 1));
          v[h][i] = p < pieces ? x : v4i{0, 0, 0, 0};
        }
      }
    };
    v4i acc[2][MT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] = v4i{0, 0, 0, 0};
    // a chunk's products go by the halves of its k, each half's token operands
    // read from LDS while the half before is multiplied
    v4i x[2][MT];
    auto read = [&](int c, int h) {
      const unsigned char *buf = ring + (c % (D + 1)) * XB + li * SB + 16 * ((4 * h + lg) ^ key(li));
#pragma unroll
      for (int j = 0; j < MT; ++j) x[h][j] = *reinterpret_cast<const v4i *>(buf + 16 * j * SB);
    };
    auto mul = [&](const v4i (*v)[2], int h) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[h][i], x[h][j], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    };

    // Step c multiplies chunk c, whose first half has been read.  Before its
    // second half, a barrier: chunk c + 1's codes have landed for every wave,
    // and every wave has read chunk c's, whose place the codes D + 1 chunks
    // ahead take.  (The loop of whole chunks is entered from straight code:
    // with a branch on the way the compiler would not know how many loads are
    // in flight behind the weights it waits for, and wait for all.)
    int c = 0;
    if (full >= 2 * D + 1) {
      issue(0);
      keep_order();
#pragma unroll
      for (int u = 0; u < D; ++u) {
        issue(u + 1);
        keep_order();
        load(w[u], u);
        keep_order();
      }
      stage_barrier<D *(LX + LW)>();
      read(0, 0);
      do {
#pragma unroll
        for (int u = 0; u < D; ++u) {
          read(c + u, 1);
          mul(w[u], 0);
          stage_barrier<(D - 1) * (LX + LW) + LW>();
          read(c + u + 1, 0);
          issue(c + u + 1 + D);
          mul(w[u], 1);
          keep_order();
          load(w[u], c + u + D);
          keep_order();
        }
        c += D;
      } while (c + 2 * D + 1 <= full);
    } else {
#pragma unroll
      for (int u = 0; u <= D; ++u)
        if (u < chunks) {
          issue(u);
          if (u < D) {
            if (u < full) load(w[u], u);
            else load_part(w[u], u);
          }
        }
      stage_barrier<0>();
      read(0, 0);
    }
    for (; c < chunks; c += D) {
#pragma unroll
      for (int u = 0; u < D; ++u)
        if (c + u < chunks) {
          read(c + u, 1);
          mul(w[u], 0);
          stage_barrier<0>();
          if (c + u + 1 < chunks) read(c + u + 1, 0);
          if (c + u + 1 + D < chunks) issue(c + u + 1 + D);
          mul(w[u], 1);
          if (c + u + D < full) load(w[u], c + u + D);
          else if (c + u + D < chunks) load_part(w[u], c + u + D);
        }
    }
    finish_sweep<MT>(acc, wave, n0);
  }

  // y, 16 tokens at a time: the waves put their channels side by side in LDS
  // (8-byte or 16-byte pieces, swizzled by the token), and whole rows of BN
  // channels are written.
  template <int MT>
  __device__ __forceinline__ void finish_sweep(const v4i (*acc)[MT], int wave, int n0) {
    constexpr int EPC = 16 / (int)sizeof(T);   // elements of a 16-byte chunk
    constexpr int CH = ROWB / 16;              // chunks of a row
    const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
    const float *ws = a.ws + (size_t)t.e * a.N;
    float sn[2][4], bn[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = min(n0 + 32 * wave + 16 * i + 4 * lg + r, a.N - 1);
        sn[i][r] = ws[n];
        bn[i][r] = a.bias ? a.bias[n] : 0.f;
      }
    const bool vec = reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && (uint64_t)a.ldy * sizeof(T) % 16 == 0;
    T *y = static_cast<T *>(a.y);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      if (16 * j >= t.n) break;
      const int tt = min(16 * j + li, t.n - 1);
      const float st = a.s[GROUPED ? in_row<GROUPED>(a, rows[tt]) : t.r0 + tt];
      stage_barrier<0>();  // the last operands, or the rows before, have been read
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        Pack<T, 4> v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v.v[r] = (T)finish(acc[i][j][r], st, sn[i][r], bn[i][r]);
        const int e = 32 * wave + 16 * i + 4 * lg;
        *reinterpret_cast<Pack<T, 4> *>(ring + li * ROWB + (((e / EPC) ^ (li & 7)) * 16) +
                                        (e % EPC) * (int)sizeof(T)) = v;
      }
      stage_barrier<0>();
      if (vec) {
        for (int q = threadIdx.x; q < 16 * CH; q += 64 * NW) {
          const int rr = q / CH, ch = q % CH, n = n0 + ch * EPC;
          if (16 * j + rr >= t.n || n >= a.N) continue;
          const int row = GROUPED ? rows[16 * j + rr] : t.r0 + 16 * j + rr;
          if (row < 0) continue;
          const Pack<T, EPC> v = *reinterpret_cast<const Pack<T, EPC> *>(ring + rr * ROWB + ((ch ^ (rr & 7)) * 16));
          T *d = y + (int64_t)row * a.ldy + n;
          if (n + EPC <= a.N) {
            *reinterpret_cast<Pack<T, EPC> *>(d) = v;
          } else {
#pragma unroll
            for (int k = 0; k < EPC - 1; ++k)
              if (n + k < a.N) d[k] = v.v[k];
          }
        }
      } else {
        for (int q = threadIdx.x; q < 16 * BN; q += 64 * NW) {
          const int rr = q / BN, k = q % BN;
          if (16 * j + rr >= t.n || n0 + k >= a.N) continue;
          const int row = GROUPED ? rows[16 * j + rr] : t.r0 + 16 * j + rr;
          if (row < 0) continue;
          y[(int64_t)row * a.ldy + n0 + k] = *reinterpret_cast<const T *>(
              ring + rr * ROWB + (((k / EPC) ^ (rr & 7)) * 16) + (k % EPC) * (int)sizeof(T));
        }
      }
    }
  }
};

// The smallest of the variants MT = 1, 2, 4, ... MAX that holds n tokens.
template <int MAX, int M = 1, typename K>
__device__ __forceinline__ void sweep_dispatch(K &k, int n) {
  if constexpr (M >= MAX) {
    k.template run<MAX>();
  } else {
    if (n <= 16 * M) k.template run<M>();
    else sweep_dispatch<MAX, 2 * M>(k, n);
  }
}

template <int DT, int BM, int NW, int D, bool GROUPED>
__global__ __launch_bounds__(64 * NW) void k_q8_sweep(Q8Args a, int nbm, int nbn) {
  typedef SweepKernel<DT, BM, NW, D, GROUPED> K;
  __shared__ __align__(16) unsigned char ring[K::LDS];
  __shared__ int rows[GROUPED ? BM : 1];
  Tile t;
  if constexpr (GROUPED) {
    t = expert_tile<BM>(a, nbn);
    if (t.n <= 0) return;
    for (int i = threadIdx.x; i < t.n; i += 64 * NW) rows[i] = out_row<GROUPED>(a, t.r0 + i);
    __syncthreads();
  } else {
    const int id = xcd_item(blockIdx.x, nbm * nbn);
    if (id < 0) return;
    const int m = id % nbm;
    t = Tile{0, m * BM, min(BM, a.rows - m * BM), id / nbm};
  }
  K k{a, t, ring, rows};
  sweep_dispatch<BM / 16>(k, t.n);
}

// ---------------------------------------------------------------------------
// Many tokens.  A workgroup of WM x WN waves takes up to BM tokens and BN
// channels in 32 x 32 products: wave (wm, wn) the token groups of 32 wm, wm +
// WM, ... and BN / WN consecutive channels.  A tile with fewer tokens (an
// expert's, or the last) runs the same loop over fewer groups, TMV for each
// wave, so that its cost follows its tokens and the LDS they leave free holds
// more stages.
//
// k goes by stages of SB bytes of every row through a ring of STAGES in LDS,
// filled by direct loads.  The operands of a step (k = 32) are read from LDS
// while the step before is multiplied, across stages too: before a stage's
// last step, one barrier both publishes the next stage and frees this one,
// so there is one barrier a stage and none of its wait is exposed.
//
// LDS: piece p (16 bytes) of row r's stage lies at place p ^ key(r), so that
// the 16 rows which 16 lanes read at one k lie in different banks.  The
// loads write LDS in lane order, so the swizzle is in the addresses they
// read.  Rows past the tile and pieces past the row's end read valid
// addresses near them; what they bring in is never used.
//
// 8192 x 6144 x 6144 to bfloat16: 282-293 us, 2.11-2.19 POPS, where the
// library's int8 product reaches 2.19.  What bounds it is power: on zeros the
// same launch takes 220 us; other wave shapes and operands two steps ahead
// change nothing, and stages of 64 bytes, which ask for each line twice, cost
// (1.23 times as long at 128 x 147456 x 6144).  Storing rows whole instead of 8
// bytes of each took 32 us off.
// ---------------------------------------------------------------------------
template <int DT, int BM, int BN, int WM, int WN, int LDS, bool GROUPED>
struct TileKernel {
  typedef typename Elem<DT>::type T;
  static constexpr int SB = 128;
  static constexpr int NW = WM * WN;
  static constexpr int TN = BN / WN / 32;       // channel groups of a wave
  static constexpr int TMAX = BM / WM / 32;     // token groups of a wave, at most
  static constexpr int PPR = SB / 16;           // pieces of a row in a stage
  static constexpr int RPL = 64 / PPR;          // rows of a load
  static constexpr int KSN = SB / 32;           // steps of a stage
  static constexpr int LW = BN / RPL / NW;      // weight loads of a wave in a stage
  static_assert(BN % (RPL * NW) == 0, "whole loads");
  // place of piece p of row r: p ^ key(r); 256 / SB rows span the banks
  __device__ __forceinline__ static int key(int r) { return (r / (256 / SB)) & (PPR - 1); }

  const Q8Args &a;
  const Tile &t;
  unsigned char *ring;   // LDS bytes
  const int *rows;       // [BM] output rows of the tile's tokens (-1: none)
  const float *chans;    // [BN] the channels' scales

  template <int TMV>
  __device__ __forceinline__ void run() {
    constexpr int XROWS = 32 * WM * TMV;
    // token loads of a wave: whole ones, and one by half the lanes where the
    // rows are an odd multiple of what half the loads bring
    constexpr int LXF = XROWS / (RPL * NW), HALF = XROWS % (RPL * NW) ? 1 : 0;
    constexpr int LX = LXF + HALF, NL = LX + LW;
    static_assert(HALF == 0 || XROWS % (RPL * NW) == RPL * NW / 2, "whole or half loads");
    constexpr int STAGE = (XROWS + BN) * SB;
    constexpr int STAGES = LDS / STAGE < 6 ? LDS / STAGE : 6;
    static_assert(STAGES >= 2 && NL * (STAGES - 1) < 64, "ring");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int n0 = t.nb * BN;
    const int pieces = a.K / 16, full = pieces / PPR, stages = (pieces + PPR - 1) / PPR;

    // this lane's source of each load: its row (tokens first, then weights)
    // and the piece of it that belongs at its place
    const uint8_t *xb = reinterpret_cast<const uint8_t *>(a.q) + (GROUPED ? 0 : (size_t)t.r0 * a.K);
    const uint8_t *wb = a.w + ((size_t)t.e * a.N + n0) * a.K;
    uint32_t off[NL], pl[NL];
    // first row of load i in the stage
    auto row_of = [&](int i) {
      if (i < LXF) return (i * NW + wave) * RPL;
      if (i < LX) return LXF * NW * RPL + wave * (RPL / 2);
      return XROWS + ((i - LX) * NW + wave) * RPL;
    };
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int r = row_of(i) + lane / PPR;
      pl[i] = (lane % PPR) ^ key(r);
      int src;
      if (i < LX) {
        const int tt = min(r, t.n - 1);
        src = GROUPED ? in_row<GROUPED>(a, rows[tt]) : tt;
      } else {
        src = min(r - XROWS, a.N - 1 - n0);
      }
      off[i] = (uint32_t)src * (uint32_t)a.K;
    }
    auto issue = [&](int c) {
      unsigned char *buf = ring + (c % STAGES) * STAGE;
      // (opaque: kept as a scalar base and the lane's 32-bit offset)
      uint64_t xc = reinterpret_cast<uint64_t>(xb) + (uint64_t)c * SB;
      uint64_t wc = reinterpret_cast<uint64_t>(wb) + (uint64_t)c * SB;
      asm("" : "+s"(xc), "+s"(wc));
      const uint32_t last = c < full ? PPR - 1 : (uint32_t)(pieces - PPR * c - 1);
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const uint32_t o = off[i] + 16 * min(pl[i], last);
        if (i < LXF || i >= LX || lane < 32)
          __builtin_amdgcn_global_load_lds(reinterpret_cast<const uint8_t *>(i < LX ? xc : wc) + o,
                                           (lds_void *)(buf + row_of(i) * SB), 16, 0, 0);
      }
    };

    v16i acc[TN][TMV];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TMV; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

    const int lr = lane & 31, lh = lane >> 5, rkey = key(lr);
    struct Ops {
      v4i x[TMV], w[TN];
    };
    auto read = [&](int c, int ks, Ops &o) {
      const unsigned char *buf = ring + (c % STAGES) * STAGE + lr * SB + 16 * ((2 * ks + lh) ^ rkey);
#pragma unroll
      for (int j = 0; j < TMV; ++j)
        o.x[j] = *reinterpret_cast<const v4i *>(buf + (j * WM + wm) * 32 * SB);
#pragma unroll
      for (int i = 0; i < TN; ++i)
        o.w[i] = *reinterpret_cast<const v4i *>(buf + (XROWS + (wn * TN + i) * 32) * SB);
    };
    auto mul = [&](const Ops &o) {
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TMV; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(o.w[i], o.x[j], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    };

    Ops A, B;
#pragma unroll
    for (int c = 0; c < STAGES; ++c) {
      if (c < stages) issue(c);
      keep_order();
    }
    if (stages >= STAGES) stage_barrier<NL *(STAGES - 1)>();
    else stage_barrier<0>();
    read(0, 0, A);
    for (int c = 0; c < full; ++c) {
      read(c, 1, B);
      mul(A);
#pragma unroll
      for (int ks = 2; ks < KSN; ks += 2) {
        read(c, ks, A);
        mul(B);
        read(c, ks + 1, B);
        mul(A);
      }
      // stage c + 1 has landed for every wave, and no wave reads stage c any more
      if (c + STAGES <= stages) stage_barrier<NL *(STAGES - 2)>();
      else stage_barrier<0>();
      if (c + 1 < stages) read(c + 1, 0, A);
      if (c + STAGES < stages) issue(c + STAGES);
      keep_order();
      mul(B);
    }
    // the part of a stage that is left (K is a multiple of 32)
    if (full < stages) {
      const int steps = (pieces - PPR * full) / 2;
      mul(A);
      for (int ks = 1; ks < steps; ++ks) {
        read(full, ks, A);
        mul(A);
      }
    }
    finish_tile<TMV>(acc, wave, wm, wn, n0);
  }

  // y from the accumulators: lane (lr, lh) holds token lr of each group and
  // channels 8 g + 4 lh + 0..3 (g < 4) of each 32.  Each wave turns its 32
  // tokens x 32 TN channels at a time in an LDS area of its own, so that a
  // store writes whole runs of a row.
  template <int TMV>
  __device__ __forceinline__ void finish_tile(const v16i (*acc)[TMV], int wave, int wm, int wn, int n0) {
    constexpr int EPC = 16 / (int)sizeof(T);        // elements of a 16-byte chunk
    constexpr int CH = 32 * TN / EPC;               // chunks of a row
    // bytes of a row in the area: chunk c of row r lies at c ^ (r % 8)
    constexpr int ROWB = 16 * (CH <= 8 ? 8 : 16);
    static_assert(64 % CH == 0 && CH <= 16 && NW * 32 * ROWB <= LDS, "whole rows a store, and the area");
    const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
    const int nw = n0 + wn * TN * 32;
    float sn[TN][16], bn[TN][16];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int n = nw + 32 * i + 8 * (r / 4) + 4 * lh + r % 4;
        sn[i][r] = chans[n - n0];
        bn[i][r] = a.bias ? a.bias[min(n, a.N - 1)] : 0.f;
      }
    const bool vec = reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && (uint64_t)a.ldy * sizeof(T) % 16 == 0;
    stage_barrier<0>();  // every wave has read its last operands
    unsigned char *area = ring + wave * 32 * ROWB;
    T *y = static_cast<T *>(a.y);
#pragma unroll
    for (int j = 0; j < TMV; ++j) {
      const int t0 = (j * WM + wm) * 32;
      if (t0 >= t.n) break;
      const float st = a.s[in_row<GROUPED>(a, rows[min(t0 + lr, t.n - 1)])];
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          Pack<T, 4> v;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            v.v[r] = (T)finish(acc[i][j][4 * g + r], st, sn[i][4 * g + r], bn[i][4 * g + r]);
          const int e = 32 * i + 8 * g + 4 * lh;  // first element: chunk e / EPC, the key swaps chunks
          *reinterpret_cast<Pack<T, 4> *>(area + lr * ROWB + (((e / EPC) ^ (lr & 7)) * 16) +
                                          (e % EPC) * (int)sizeof(T)) = v;
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (vec) {
#pragma unroll
        for (int p = 0; p < 32 * CH / 64; ++p) {
          const int rr = p * (64 / CH) + lane / CH, ch = lane % CH;
          const Pack<T, EPC> v = *reinterpret_cast<const Pack<T, EPC> *>(area + rr * ROWB + ((ch ^ (rr & 7)) * 16));
          const int n = nw + ch * EPC;
          if (t0 + rr >= t.n || n >= a.N) continue;
          const int row = rows[t0 + rr];
          if (row < 0) continue;
          T *d = y + (int64_t)row * a.ldy + n;
          if (n + EPC <= a.N) {
            *reinterpret_cast<Pack<T, EPC> *>(d) = v;
          } else {
#pragma unroll
            for (int k = 0; k < EPC - 1; ++k)
              if (n + k < a.N) d[k] = v.v[k];
          }
        }
      } else {
        for (int rr = 0; rr < 32 && t0 + rr < t.n; ++rr) {
          const int row = rows[t0 + rr];
          if (row < 0) continue;
#pragma unroll
          for (int e = 0; e < 32 * TN; e += 64) {
            const int k = e + lane;
            if (k < 32 * TN && nw + k < a.N)
              y[(int64_t)row * a.ldy + nw + k] = *reinterpret_cast<const T *>(
                  area + rr * ROWB + (((k / EPC) ^ (rr & 7)) * 16) + (k % EPC) * (int)sizeof(T));
          }
        }
      }
      asm volatile("" ::: "memory");
    }
  }
};

// The variant for tm (up to M) token groups of each wave.
template <int M, typename K>
__device__ __forceinline__ void tile_dispatch(K &k, int tm) {
  if constexpr (M == 1) {
    k.template run<1>();
  } else {
    if (tm >= M) k.template run<M>();
    else tile_dispatch<M - 1>(k, tm);
  }
}

template <int DT, int BM, int BN, int WM, int WN, int LDS, bool GROUPED>
__device__ __forceinline__ void tile_body(const Q8Args &a, int nbm, int nbn, unsigned char *ring, int *rows,
                                          float *chans) {
  Tile t;
  if constexpr (GROUPED) {
    t = expert_tile<BM>(a, nbn);
    if (t.n <= 0) return;
  } else {
    const int id = xcd_item(blockIdx.x, nbm * nbn);
    if (id < 0) return;
    // runs of 4 token tiles: the workgroups of an XCD at one time share
    // about as many token rows as weight rows
    const int run = 4 * nbn, g = id / run, h = min(4, nbm - g * 4);
    const int m = g * 4 + (id % run) % h;
    t = Tile{0, m * BM, min(BM, a.rows - m * BM), (id % run) / h};
  }
  // (the channels' scales now, so that the end does not wait for them; the
  // tokens' too would fill the LDS to its last byte, which costs 13 %)
  for (int i = threadIdx.x; i < t.n; i += 64 * WM * WN) rows[i] = out_row<GROUPED>(a, t.r0 + i);
  for (int i = threadIdx.x; i < BN; i += 64 * WM * WN)
    chans[i] = a.ws[(size_t)t.e * a.N + min(t.nb * BN + i, a.N - 1)];
  __syncthreads();
  TileKernel<DT, BM, BN, WM, WN, LDS, GROUPED> k{a, t, ring, rows, chans};
  tile_dispatch<BM / WM / 32>(k, (t.n + 32 * WM - 1) / (32 * WM));
}

template <int DT, int BM, int BN, int WM, int WN, int LDS, bool GROUPED>
// (LDS past half a CU's leaves room for one workgroup)
__global__ __launch_bounds__(64 * WM * WN, WM * WN >= 8 || LDS <= 80 << 10 ? 2 : 1) void k_q8_tile(Q8Args a, int nbm, int nbn) {
  __shared__ __align__(16) unsigned char ring[LDS];
  __shared__ int rows[BM];
  __shared__ float chans[BN];
  tile_body<DT, BM, BN, WM, WN, LDS, GROUPED>(a, nbm, nbn, ring, rows, chans);
}

// ---------------------------------------------------------------------------
// The variants and the choice among them.  A variant's tile (bm tokens x bn
// channels) and threads are its kernel's.
// ---------------------------------------------------------------------------
enum Variant {
  kRing16x16, kRing16x32, kRing32x64, kRing64x32, kRing64x64, kSweep32, kSweep64,
  kTile128, kTile128Deep, kTile256, kVariants
};
struct Shape {
  int bm, bn, threads;
};
constexpr Shape kShapes[kVariants] = {{16, 16, 256}, {16, 32, 256},  {32, 64, 256},   {64, 32, 512},   {64, 64, 512},
                                      {32, 64, 128}, {64, 128, 256}, {128, 128, 256}, {128, 128, 256}, {256, 256, 512}};

// Upper bound of the token tiles of bm over E experts with P pairs.
int64_t max_tiles(const Q8Args &a, int bm) { return a.P / bm + (a.P < a.E ? a.P : a.E); }

int64_t workgroups(const Q8Args &a, Variant v) {
  const Shape &s = kShapes[v];
  const int64_t nbn = (a.N + (int64_t)s.bn - 1) / s.bn;
  const int64_t nbm = a.offs ? max_tiles(a, s.bm) : (a.rows + (int64_t)s.bm - 1) / s.bm;
  return (nbm * nbn + 7) / 8 * 8;
}

// Experts' products, by the tokens of an expert on average (P / E: what the
// host knows; dropped slots count too).  The sweep reads each weight once at
// the rate of the memory as long as its workgroups fill the chip; the rings
// split k and fill it with fewer channels.  In us, launches one after another:
//   64 experts of 6144 x 2048:   16x32, 64x32, sweeps of 32, 64, tile
//     10 tokens each             152,   254,   149,   150,   149
//     31                         219,   268,   168,   162,   161
//     50                         332,   292,   234,   176,   173
//   256 experts of 4096 x 6144:
//     10                         1105,  1694,  1106,  1095,  1070
//     64, 128                    sweep of 64 1345, 1983; tile 1212, 1409
//   24 experts of 4096 x 6144:
//     1                          107,   172,   115,   116,   123
// (The experts' kTile256 gives each wave 32 channels of all tokens: cost
// follows the tokens by 32, and three stages fit up to 160 tokens; 2 x 4 waves
// as in the dense product take 1.03 times as long at 128 tokens.)
// Uneven routing: where the tokens go with 1 / rank over 64 or 256 experts, the
// choice is within 6 % of the best (8192 pairs over 256 experts: 1332, tile
// 1257), and with half of them in one expert 4 % (512: 1060, 16x32 1023).  It
// costs where few experts take all of a batch that would fill many: 8 of 256
// experts with 256 tokens each 216 us by kSweep32, 83 by the tile.
Variant grouped_variant(const Q8Args &a) {
  const int64_t avg = ((int64_t)a.P + a.E - 1) / a.E;
  const int64_t used = a.P < a.E ? a.P : a.E;  // experts with a token, at most
  if (avg <= 12) return used * (a.N / 64) >= 1024 ? kSweep32 : kRing16x32;
  if (avg <= 52) return used * (a.N / 128) >= 512 ? kSweep64 : kRing64x32;
  return kTile256;
}

// The dense product: the variant of the least time, from what each takes at
// 4096 columns (in 0.1 us) with at most one workgroup a CU, and for a full
// round of its slots, the workgroups that the 256 CUs hold at once.  The table
// was made with one matrix again and again, of which the Infinity Cache keeps
// up to 256 MB; a model goes on to its next matrix.  Measured so, with matrices
// of 640 MB together in turn (64 at most), over 1 to 3000 tokens x 300 to 40000
// channels x 1024, 2560 and 6144 columns, the choice is the best variant or
// within 15 % of it at 270 of 273 sizes (3000 x 300 x 6144: 64x32 26.9 us,
// 32x64 20.2; x 2560 13.2, 11.0; 61 x 40000 x 1024: 64x64 17.7, 128x128 15.4).
// Some of both sides (us, 6144 columns, matrices in turn):
//   30 x 2048   16x16 8.4, 64x32 12.7              1 x 6144     16x32 9.9, 64x32 13.6
//   61 x 6144   64x32 15.6, 16x32 20.5             200 x 6144   64x64 27.3, 64x32 27.9
//   509 x 6144  128x128 of one a CU 34.7,          1500 x 6144  256x256 78.1, 128x128 87.7
//               of two 47.8, 64x64 54.6            3000 x 6144  128x128 137.4, 256x256 159.1
// (Blocks whose tokens would be half empty are left out.)  33 to 64 tokens of
// very many channels are bound by the memory in every form; from 65536 channels
// on neither the sweep nor 128x128 is always the better (us, sweep / 128x128 /
// 64x64 / 64x32): 61 x 65536 x 1024 20 / 18 / 23 / 28, 48 x 65536 x 6144 88 / 81 /
// 83 / 99, 61 x 100000 x 6144 159 / 137 / 146 / 162, 48 x 100000 x 4096 106 / 102
// / 106 / 106, 61 x 150000 x 1024 41 / 44 / 51 / 56, 48 x 150000 x 4096 136 / 150 /
// 144 / 154.  Over 33, 48 and 61 tokens x 1024 to 6144 columns the sweep is within
// 16 % of the best of the four, 128x128 13 %, 64x64 28 %, 64x32 54 %.  With fewer
// channels it is not: 64 x 32768 x 6144 53 / 58 / 44 / 56.
Variant dense_variant(const Q8Args &a) {
  struct Time {
    Variant v;
    int slots, first, round;
  };
  constexpr Time kTimes[] = {{kRing16x16, 512, 58, 70},  {kRing16x32, 512, 67, 82},   {kRing32x64, 512, 108, 140},
                             {kRing64x32, 512, 83, 138}, {kRing64x64, 512, 140, 185}, {kTile128Deep, 256, 240, 0},
                             {kTile128, 512, 265, 410},  {kTile256, 256, 565, 693}};
  if (a.rows > 32 && a.rows <= 64 && a.N >= 65536) return kSweep64;
  Variant best = kTile256;
  int64_t least = INT64_MAX;
  for (const Time &t : kTimes) {
    const Shape &s = kShapes[t.v];
    const int64_t n = workgroups(a, t.v);
    if ((s.bm > 16 && s.bm >= 2 * (int64_t)a.rows) || (n > 256 && t.round == 0)) continue;
    const int64_t cost = n <= 256 ? t.first : t.round * ((n + t.slots - 1) / t.slots);
    if (cost < least) {
      least = cost;
      best = t.v;
    }
  }
  return best;
}

Variant variant_of(const Q8Args &a) { return a.offs ? grouped_variant(a) : dense_variant(a); }

template <int DT, bool GROUPED, int BM, int BN, int WM, int WN, int KS, int STAGES>
void run_ring(const Q8Args &a, int64_t wgs, hipStream_t st) {
  const int nbn = (a.N + BN - 1) / BN, nbm = (a.rows + BM - 1) / BM;
  hipLaunchKernelGGL((k_q8_ring<DT, BM, BN, WM, WN, KS, STAGES, GROUPED>), dim3(wgs),
                     dim3(64 * WM * WN * KS), 0, st, a, nbm, nbn);
}

template <int DT, bool GROUPED, int BM, int NW, int D>
void run_sweep(const Q8Args &a, int64_t wgs, hipStream_t st) {
  const int nbn = (a.N + 32 * NW - 1) / (32 * NW), nbm = (a.rows + BM - 1) / BM;
  hipLaunchKernelGGL((k_q8_sweep<DT, BM, NW, D, GROUPED>), dim3(wgs), dim3(64 * NW), 0, st, a, nbm, nbn);
}

template <int DT, bool GROUPED, int BM, int BN, int WM, int WN, int LDS>
void run_tile(const Q8Args &a, int64_t wgs, hipStream_t st) {
  const int nbn = (a.N + BN - 1) / BN, nbm = (a.rows + BM - 1) / BM;
  hipLaunchKernelGGL((k_q8_tile<DT, BM, BN, WM, WN, LDS, GROUPED>), dim3(wgs), dim3(64 * WM * WN), 0, st,
                     a, nbm, nbn);
}

}  // namespace

bool gemm_q8_fits(const Q8Args &a) {
  // (the grouped kernels name rows of q by 32-bit byte offsets)
  if (a.offs && (int64_t)a.rows * a.K >= (int64_t)1 << 32) return false;
  const Variant v = variant_of(a);
  return workgroups(a, v) * kShapes[v].threads < ((int64_t)1 << 31);
}

hipError_t launch_gemm_q8(int dt, const Q8Args &a, hipStream_t st) {
  if ((a.offs ? a.P : a.rows) == 0) return hipSuccess;
  const Variant v = variant_of(a);
  const int64_t wgs = workgroups(a, v);
  return by_dtype(dt, [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    if (a.offs) {
      switch (v) {
        case kRing16x32: run_ring<DT, true, 16, 32, 1, 1, 4, 3>(a, wgs, st); break;
        case kRing64x32: run_ring<DT, true, 64, 32, 2, 1, 4, 3>(a, wgs, st); break;
        case kSweep32: run_sweep<DT, true, 32, 2, 4>(a, wgs, st); break;
        case kSweep64: run_sweep<DT, true, 64, 4, 3>(a, wgs, st); break;
        default: run_tile<DT, true, 256, 256, 1, 8, 157 << 10>(a, wgs, st); break;
      }
    } else {
      switch (v) {
        case kRing16x16: run_ring<DT, false, 16, 16, 1, 1, 4, 8>(a, wgs, st); break;
        case kRing16x32: run_ring<DT, false, 16, 32, 1, 1, 4, 6>(a, wgs, st); break;
        case kRing32x64: run_ring<DT, false, 32, 64, 1, 1, 4, 3>(a, wgs, st); break;
        case kRing64x32: run_ring<DT, false, 64, 32, 2, 1, 4, 3>(a, wgs, st); break;
        case kRing64x64: run_ring<DT, false, 64, 64, 2, 2, 2, 2>(a, wgs, st); break;
        case kSweep64: run_sweep<DT, false, 64, 4, 3>(a, wgs, st); break;
        case kTile128: run_tile<DT, false, 128, 128, 2, 2, 64 << 10>(a, wgs, st); break;
        case kTile128Deep: run_tile<DT, false, 128, 128, 2, 2, 128 << 10>(a, wgs, st); break;
        default: run_tile<DT, false, 256, 256, 2, 4, 144 << 10>(a, wgs, st); break;
      }
    }
    return hipGetLastError();
  });
}

}  // namespace coli
