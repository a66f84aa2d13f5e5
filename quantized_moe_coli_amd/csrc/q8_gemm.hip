// q8_gemm.hip -- the matrix product in 8-bit integers with one scale per
// token and one per output channel, dense and over experts:
//   y[t][n] = s_t * ws_n * sum_k q[t][k] w[n][k]  (+ bias[n]).
//
// Unlike a product against Q8_0 blocks, no scale changes along k, so the
// whole sum stays in the int32 accumulators of the matrix instructions and
// is exact for K < 2^17 (128 * 128 * K < 2^31); one conversion and two
// multiplications in binary32 finish it, and one rounding to y's type.
// Exact sums also make every split of k give the same bits.
//
// Both operands are contiguous along k, which is what the instructions take:
// v_mfma_i32_32x32x32_i8 reads 16 consecutive bytes of row (lane % 32) at
// k = 16 (lane / 32), v_mfma_i32_16x16x64_i8 of row (lane % 16) at
// k = 16 (lane / 16).  Weight rows are the A operand and tokens the B
// operand, so a lane's results are one token's consecutive channels.
//
// Two kernels:
//   k_q8_stream  few tokens (per expert): bound by reading the weights.  They
//                go from memory to registers in operand order, with no LDS.
//   k_q8_tile    many tokens: bound by the matrix cores.  Tiles of both
//                operands go to LDS by direct loads, double-buffered.
#include <type_traits>

#include "q8.hpp"

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

// The grouped product's tile number `id` among (expert, channel block, token
// tile): each wave sums the experts' tile counts itself (E <= 1024, at most
// 16 a lane), so no table and no extra launch is needed.  The grid is the
// host's bound; `total` is what there is to do.  Token tiles of one expert
// and channel block are neighbours, so that their weights are read from
// memory once.
struct Experts {
  int lo, hi;    // this lane's experts
  int before;    // token tiles of the experts before them
  int total;     // token tiles of all experts
};

__device__ __forceinline__ int expert_begin(const Q8Args &a, int e) {
  return min(max(a.offs[e], 0), a.P);
}

template <int BM>
__device__ __forceinline__ Experts scan_experts(const Q8Args &a) {
  const int lane = threadIdx.x & 63;
  const int per = (a.E + 63) / 64;
  Experts x;
  x.lo = min(lane * per, a.E);
  x.hi = min(x.lo + per, a.E);
  int mine = 0;
  if (x.lo < x.hi) {
    int b = expert_begin(a, x.lo);
    for (int e = x.lo; e < x.hi; ++e) {
      const int nx = expert_begin(a, e + 1);
      if (nx > b) mine += (nx - b + BM - 1) / BM;
      b = nx;
    }
  }
  // (offs that are no running sum could count more tiles than there are)
  const int bound = a.P / BM + min(a.P, a.E);
  mine = min(mine, bound);
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(sum, d, 64);
    if (lane >= d) sum += o;
  }
  x.before = sum - mine;
  x.total = min(__shfl(sum, 63, 64), bound);
  return x;
}

// The tile `id` of `x.total * nbn`; id is uniform.
template <int BM>
__device__ __forceinline__ Tile find_tile(const Q8Args &a, const Experts &x, int id, int nbn) {
  const int lane = threadIdx.x & 63;
  // the last lane whose first tile is not past id holds it, if it has any
  const uint64_t le = __ballot((int64_t)x.before * nbn <= id && x.lo < x.hi);
  const int owner = 63 - __clzll(le);
  Tile t{0, 0, 0, 0};
  int4 r = make_int4(0, 0, 0, 0);
  if (lane == owner) {
    int before = x.before, b = expert_begin(a, x.lo);
    for (int e = x.lo; e < x.hi; ++e) {
      const int nx = expert_begin(a, e + 1);
      const int mt = nx > b ? (nx - b + BM - 1) / BM : 0;
      if ((int64_t)(before + mt) * nbn > id) {
        const int local = (int)(id - (int64_t)before * nbn);
        const int m = local % mt;
        r = make_int4(e, b + m * BM, min(BM, nx - b - m * BM), local / mt);
        break;
      }
      before += mt;
      b = nx;
    }
  }
  t.e = __shfl(r.x, owner, 64);
  t.r0 = __shfl(r.y, owner, 64);
  t.n = __shfl(r.z, owner, 64);
  t.nb = __shfl(r.w, owner, 64);
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.r0 = __builtin_amdgcn_readfirstlane(t.r0);
  t.n = __builtin_amdgcn_readfirstlane(t.n);
  t.nb = __builtin_amdgcn_readfirstlane(t.nb);
  return t;
}

// Workgroup b runs on XCD b % 8, each with its own L2: an XCD takes a
// contiguous run of the `total` items, so that neighbours share it.
__device__ __forceinline__ int xcd_item(int b, int total) {
  const int per = (total + 7) / 8;
  const int i = (b % 8) * per + b / 8;
  return b / 8 < per && i < total ? i : -1;
}

// y's element from the exact sum.
__device__ __forceinline__ float finish(int acc, float st, float sn, float b) {
  return (float)acc * (st * sn) + b;
}

// ---------------------------------------------------------------------------
// Few tokens.  A workgroup of 8 waves takes 16 NT channels and up to 16 MT
// tokens; the waves take the 128-byte chunks of k in turn and their exact
// partial sums are added through LDS.
// ---------------------------------------------------------------------------
constexpr int kStreamWaves = 8;

template <int DT, int MT, int NT, bool GROUPED>
__global__ __launch_bounds__(64 * kStreamWaves) void k_q8_stream(Q8Args a, int nbn) {
  typedef typename Elem<DT>::type T;
  __shared__ int part[kStreamWaves][MT * NT][4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lg = lane >> 4;

  Tile t;
  if constexpr (GROUPED) {
    const Experts x = scan_experts<16 * MT>(a);
    const int id = xcd_item(blockIdx.x, x.total * nbn);
    if (id < 0) return;
    t = find_tile<16 * MT>(a, x, id, nbn);
    if (t.n <= 0) return;
  } else {
    t = Tile{0, (int)blockIdx.y * 16 * MT, min(16 * MT, a.rows - (int)blockIdx.y * 16 * MT),
             (int)blockIdx.x};
  }
  const int n0 = t.nb * 16 * NT;
  const uint8_t *wb = a.w + (size_t)t.e * a.N * a.K;
  const uint8_t *wp[NT];
  const int8_t *xp[MT];
#pragma unroll
  for (int i = 0; i < NT; ++i) wp[i] = wb + (size_t)min(n0 + 16 * i + li, a.N - 1) * a.K;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int pos = t.r0 + min(16 * i + li, t.n - 1);
    xp[i] = a.q + (size_t)in_row<GROUPED>(a, out_row<GROUPED>(a, pos)) * a.K;
  }
  v4i acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = v4i{0, 0, 0, 0};

  const int pieces = a.K / 16, full = pieces / 8;
  auto mul = [&](const v4i (&wv)[2][NT], const v4i (&xv)[2][MT]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[h][i], xv[h][j], acc[i][j], 0, 0, 0);
  };
  // U chunks' loads are in flight together
  constexpr int U = MT * NT == 1 ? 6 : MT + NT <= 4 ? 3 : 2;
  int c = wave;
  for (; c + (U - 1) * kStreamWaves < full; c += U * kStreamWaves) {
    v4i wv[U][2][NT], xv[U][2][MT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const size_t o = (size_t)(c + u * kStreamWaves) * 128 + 64 * h + 16 * lg;
#pragma unroll
        for (int i = 0; i < NT; ++i)
          wv[u][h][i] = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(wp[i] + o));
#pragma unroll
        for (int i = 0; i < MT; ++i) xv[u][h][i] = *reinterpret_cast<const v4i *>(xp[i] + o);
      }
#pragma unroll
    for (int u = 0; u < U; ++u) mul(wv[u], xv[u]);
  }
  // what is left, and the part chunk at the row's end: pieces past it count
  // as zero weights
  for (; c * 8 < pieces; c += kStreamWaves) {
    v4i wv[2][NT], xv[2][MT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int pc = c * 8 + 4 * h + lg;
      const size_t o = (size_t)min(pc, pieces - 1) * 16;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const v4i v = *reinterpret_cast<const v4i *>(wp[i] + o);
        wv[h][i] = pc < pieces ? v : v4i{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) xv[h][i] = *reinterpret_cast<const v4i *>(xp[i] + o);
    }
    mul(wv, xv);
  }

#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][j * NT + i][r][lane] = acc[i][j][r];
  __syncthreads();
  T *y = static_cast<T *>(a.y);
  for (int o = threadIdx.x; o < 256 * MT * NT; o += 64 * kStreamWaves) {
    const int nn = o % (16 * NT), tt = o / (16 * NT);
    const int n = n0 + nn;
    if (tt >= t.n || n >= a.N) continue;
    const int row = out_row<GROUPED>(a, t.r0 + tt);
    if (row < 0) continue;
    const int tile = (tt / 16) * NT + nn / 16, l = tt % 16 + 16 * ((nn % 16) / 4);
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kStreamWaves; ++w) sum += part[w][tile][nn % 4][l];
    const float b = a.bias ? a.bias[n] : 0.f;
    y[(int64_t)row * a.ldy + n] =
        (T)finish(sum, a.s[in_row<GROUPED>(a, row)], a.ws[(size_t)t.e * a.N + n], b);
  }
}

// ---------------------------------------------------------------------------
// Many tokens.  A workgroup of WM x WN waves takes BM tokens and BN
// channels, each wave BM / WM by BN / WN of them in 32 x 32 products.  k
// goes by stages of 128 bytes of every row, two stages of LDS: while one is
// multiplied the next is loaded, and one barrier a stage separates them.
//
// LDS: a row's stage is 8 pieces of 16 bytes, piece p of row r at place
// p ^ ((r / 2) % 8), so the 16 rows that 16 lanes read at one k lie in
// different banks (two rows span the 64 banks).  The loads write LDS in lane
// order, so the swizzle is in the addresses they read.  Rows past the tile
// and pieces past the row's end read valid addresses near them; what they
// bring in is never used.
// ---------------------------------------------------------------------------
constexpr int kStageBytes = 128;

template <int DT, int BM, int BN, int WM, int WN, bool GROUPED>
__device__ __forceinline__ void tile_body(const Q8Args &a, int nbm, int nbn) {
  typedef typename Elem<DT>::type T;
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;  // 32 x 32 products of a wave
  constexpr int ROWS = BM + BN;
  constexpr int LD = ROWS / 8 / NW;  // load instructions of a wave in a stage (8 rows each)
  static_assert(ROWS % (8 * NW) == 0, "whole loads");
  __shared__ __align__(16) unsigned char ring[2][ROWS * kStageBytes];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;

  Tile t;
  if constexpr (GROUPED) {
    const Experts x = scan_experts<BM>(a);
    const int id = xcd_item(blockIdx.x, x.total * nbn);
    if (id < 0) return;
    t = find_tile<BM>(a, x, id, nbn);
    if (t.n <= 0) return;
  } else {
    const int id = xcd_item(blockIdx.x, nbm * nbn);
    if (id < 0) return;
    // runs of 8 token tiles: the workgroups of an XCD at one time share
    // about as many token rows as weight rows
    const int run = 8 * nbn, g = id / run, h = min(8, nbm - g * 8);
    const int m = g * 8 + (id % run) % h;
    t = Tile{0, m * BM, min(BM, a.rows - m * BM), (id % run) / h};
  }
  const int n0 = t.nb * BN;
  const int pieces = a.K / 16;
  const uint8_t *wb = a.w + (size_t)t.e * a.N * a.K;

  // this lane's source of each load: row 8 (i NW + wave) + lane / 8 of the
  // tile (tokens first), piece (lane % 8) ^ key
  const uint8_t *src[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const int r = 8 * (i * NW + wave) + lane / 8;
    if (r < BM) {
      const int pos = t.r0 + min(r, t.n - 1);
      src[i] = reinterpret_cast<const uint8_t *>(a.q) +
               (size_t)in_row<GROUPED>(a, out_row<GROUPED>(a, pos)) * a.K;
    } else {
      src[i] = wb + (size_t)min(n0 + r - BM, a.N - 1) * a.K;
    }
  }
  // (BM is a multiple of 16, so the key of a row is the same counted from BM)
  const int pl = (lane & 7) ^ ((lane >> 4) & 3);  // key = (r / 2) % 8; r = 8 j + lane / 8
  auto issue = [&](int c) {
    unsigned char *buf = ring[c & 1];
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int j = i * NW + wave;                 // group of 8 rows
      const int p = c * 8 + (pl ^ (4 * (j & 1)));  // rows 8 j ..: key = 4 (j % 2) + (lane / 16)
      __builtin_amdgcn_global_load_lds(src[i] + 16 * (size_t)min(p, pieces - 1),
                                       (lds_void *)(buf + (size_t)j * 1024), 16, 0, 0);
    }
  };

  v16i acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  const int lr = lane & 31, lh = lane >> 5;
  const int key = (lr >> 1) & 7;
  auto step = [&](const unsigned char *buf, int ks) {
    v4i x[TM], w[TN];
    const int p = 16 * ((2 * ks + lh) ^ key);
#pragma unroll
    for (int j = 0; j < TM; ++j)
      x[j] = *reinterpret_cast<const v4i *>(buf + (wm * TM * 32 + 32 * j + lr) * kStageBytes + p);
#pragma unroll
    for (int i = 0; i < TN; ++i)
      w[i] = *reinterpret_cast<const v4i *>(buf + (BM + wn * TN * 32 + 32 * i + lr) * kStageBytes + p);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[i], x[j], acc[i][j], 0, 0, 0);
  };

  const int stages = (pieces + 7) / 8;
  issue(0);
  for (int c = 0; c < stages; ++c) {
    // this wave's loads of stage c have landed; past the barrier every
    // wave's have, and every wave is done with the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (c + 1 < stages) issue(c + 1);
    const unsigned char *buf = ring[c & 1];
    const int left = pieces - c * 8;
    if (left >= 8) {
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) step(buf, ks);
    } else {
      for (int ks = 0; ks < left / 2; ++ks) step(buf, ks);  // K is a multiple of 32
    }
  }

  // lane: token lr of each 32, channels 8 g + 4 lh + 0..3 (g < 4) of each 32
  T *y = static_cast<T *>(a.y);
  const float *ws = a.ws + (size_t)t.e * a.N;
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int tt = wm * TM * 32 + 32 * j + lr;
    if (tt >= t.n) continue;
    const int row = out_row<GROUPED>(a, t.r0 + tt);
    if (row < 0) continue;
    const float st = a.s[in_row<GROUPED>(a, row)];
    T *yr = y + (int64_t)row * a.ldy;
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int n = n0 + wn * TN * 32 + 32 * i + 8 * (r / 4) + 4 * lh + r % 4;
        if (n < a.N) yr[n] = (T)finish(acc[i][j][r], st, ws[n], a.bias ? a.bias[n] : 0.f);
      }
  }
}

template <int DT, int BM, int BN, int WM, int WN, int OCC, bool GROUPED>
__global__ __launch_bounds__(64 * WM * WN, OCC) void k_q8_tile(Q8Args a, int nbm, int nbn) {
  tile_body<DT, BM, BN, WM, WN, GROUPED>(a, nbm, nbn);
}

// Upper bound of the token tiles of BM over E experts with P pairs.
int64_t max_tiles(const Q8Args &a, int bm) { return a.P / bm + (a.P < a.E ? a.P : a.E); }

// The variants, by the tokens (for each expert, on average) that share a
// weight row: few tokens stream the weights, more take tiles that are as
// large as still leave enough of them.
enum Variant { kStream1, kStream2, kStream4, kTile128, kTile256 };
struct Shape {
  int bm, bn, threads;
};
constexpr Shape kShapes[] = {{16, 16, 512}, {32, 16, 512}, {64, 32, 512}, {128, 128, 256}, {256, 256, 512}};

Variant variant_of(const Q8Args &a) {
  const int64_t avg = a.offs ? ((int64_t)a.P + a.E - 1) / a.E : a.rows;
  if (avg <= 12) return kStream1;
  if (avg <= 28) return kStream2;
  if (avg <= 64) return kStream4;
  if (avg < 1024) return kTile128;
  return kTile256;
}

int64_t workgroups(const Q8Args &a, Variant v) {
  const Shape &s = kShapes[v];
  const int64_t nbn = (a.N + (int64_t)s.bn - 1) / s.bn;
  const int64_t nbm = a.offs ? max_tiles(a, s.bm) : (a.rows + (int64_t)s.bm - 1) / s.bm;
  return (nbm * nbn + 7) / 8 * 8;
}

template <int DT, int MT, int NT>
void run_stream(const Q8Args &a, int64_t wgs, hipStream_t st) {
  const int nbn = (a.N + 16 * NT - 1) / (16 * NT);
  if (a.offs)
    hipLaunchKernelGGL((k_q8_stream<DT, MT, NT, true>), dim3(wgs), dim3(64 * kStreamWaves), 0, st, a, nbn);
  else
    hipLaunchKernelGGL((k_q8_stream<DT, MT, NT, false>), dim3(nbn, (a.rows + 16 * MT - 1) / (16 * MT)),
                       dim3(64 * kStreamWaves), 0, st, a, nbn);
}

template <int DT, int BM, int BN, int WM, int WN>
void run_tile(const Q8Args &a, int64_t wgs, hipStream_t st) {
  const int nbn = (a.N + BN - 1) / BN, nbm = (a.rows + BM - 1) / BM;
  if (a.offs)
    hipLaunchKernelGGL((k_q8_tile<DT, BM, BN, WM, WN, 2, true>), dim3(wgs), dim3(64 * WM * WN), 0, st, a,
                       nbm, nbn);
  else
    hipLaunchKernelGGL((k_q8_tile<DT, BM, BN, WM, WN, 2, false>), dim3(wgs), dim3(64 * WM * WN), 0, st, a,
                       nbm, nbn);
}

}  // namespace

bool gemm_q8_fits(const Q8Args &a) {
  const Variant v = variant_of(a);
  return workgroups(a, v) * kShapes[v].threads < ((int64_t)1 << 31);
}

hipError_t launch_gemm_q8(int dt, const Q8Args &a, hipStream_t st) {
  if ((a.offs ? a.P : a.rows) == 0) return hipSuccess;
  const Variant v = variant_of(a);
  const int64_t wgs = workgroups(a, v);
  return by_dtype(dt, [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    switch (v) {
      case kStream1: run_stream<DT, 1, 1>(a, wgs, st); break;
      case kStream2: run_stream<DT, 2, 1>(a, wgs, st); break;
      case kStream4: run_stream<DT, 4, 2>(a, wgs, st); break;
      case kTile128: run_tile<DT, 128, 128, 2, 2>(a, wgs, st); break;
      case kTile256: run_tile<DT, 256, 256, 2, 4>(a, wgs, st); break;
    }
    return hipGetLastError();
  });
}

}  // namespace coli
