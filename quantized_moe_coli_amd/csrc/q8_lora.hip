// q8_lora.hip -- the dense 8-bit product with low-rank adapters of many
// requests beside it:
//   y[t][n] = s_t ws_n sum_k q[t][k] w[n][k] (+ bias[n]) + c_a sum_r u[t][r] b_a[n][r],
//   u[t][r] = sum_k x[t][k] a_a[r][k],   a = ids[t].
//
// Two launches: u into the caller's workspace, and the product (q8_kernels.hpp),
// whose kernels add the adapters' part to the sums in binary32 before their one
// rounding (lora.hpp).  u is bound by reading x and the adapters' a once.
#include <algorithm>

#include "q8_kernels.hpp"

namespace coli {
namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// The 16 bytes of one row that a lane gives to a product, and 16 rows x 16 rows
// over the 64 bytes of k that four lanes have of each row (lane l's are those of
// row l % 16 at 16 (l / 16)).
template <int DT> struct Oper { typedef v4f type; };
template <> struct Oper<COLI_BF16> { typedef v8bf type; };
template <> struct Oper<COLI_F16> { typedef v8h type; };

template <int DT>
__device__ __forceinline__ v4f mul16(typename Oper<DT>::type w, typename Oper<DT>::type x, v4f c) {
  if constexpr (DT == COLI_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
  } else if constexpr (DT == COLI_F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x, c, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(w[j], x[j], c, 0, 0, 0);
    return c;
  }
}

// u[row][r .. r + 3] of adapter e in slice sl; pos is the token's position in order
template <int DT>
__device__ __forceinline__ void put_u(const Q8LoraArgs &g, int sl, int row, int pos, int e, int r, v4f u) {
  if (g.pieces) {
    constexpr int PU = u_pieces(DT);
    const float f = g.scale ? g.scale[e] : 1.f;
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = r < g.R ? f * u[k] : 0.f;
    v4bf o[PU];
    split<PU, 4>(v, o);
    char *p = reinterpret_cast<char *>(g.u) + (int64_t)(pos / 32 * ((g.R + 15) / 16) + r / 16) * PU * 1024 +
              (r % 16 / 8 * 32 + pos % 32) * 16 + r % 8 * 2;
#pragma unroll
    for (int q = 0; q < PU; ++q) *reinterpret_cast<v4bf *>(p + q * 1024) = o[q];
  } else if (r < g.R) {
    *reinterpret_cast<v4f *>(g.u + ((int64_t)sl * g.rows + row) * g.R + r) = u;
  }
}

// The tokens in order of their adapters: the table's, and behind them, in order,
// the tokens without one, which the table does not list.  A table may be wrong about
// a token (made from other ids): every position is written, by one thread, and names
// no token that the table does not have right, so that nothing but that token's own
// row is lost.  A position counts if it lies in the range of its token's adapter;
// one that does not, and what is left at the end where tokens are not listed, names
// none.  Where listed tokens and those without an adapter are more than there are,
// some of these are listed: they keep the table's place and are passed over behind it.
//
// Workgroup b has `per` blocks of kOrder tokens and positions.  It writes the table's
// part of its positions and its tokens without an adapter; the others it counts itself.
// (Past 256 blocks, one for each CU, a workgroup takes several, since each reads all
// ids: a million tokens x 64 x 64 574 us in all, with a block each 846;
// 8192 x 512 x 512 28, 131072 x 128 x 128 82.)
constexpr int kOrder = 1024;
constexpr int kOrderWgs = 256;
constexpr int kOrderInts = 48 + kOrder / 32 + kMaxAdapters + 1;  // of LDS

template <int NW>
__device__ __forceinline__ void order_tokens(const Q8LoraArgs &g, int b, int per, int *lds) {
  static_assert(NW <= 16 && kOrder % (64 * NW) == 0 && kOrder <= 32 * 64 * NW, "whole rounds");
  constexpr int M = kOrder / 64 / NW, RUN = kOrder / 64;
  // for each wave: tokens without an adapter before this workgroup's, from its first on, in a block
  int *count = lds;
  uint32_t *listed = reinterpret_cast<uint32_t *>(lds + 48);  // a bit for each token of a block
  int *offs = lds + 48 + kOrder / 32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = b * per * kOrder, end = min(first + per * kOrder, g.rows);
  if (first >= end) return;
  const int live = min(max(g.tab_offs[g.L], 0), g.rows);
  auto bare = [&](int e) { return (uint32_t)e >= (uint32_t)g.L; };
  auto wave_sum = [](int v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
  };
  auto waves_sum = [&](const int *c, int n) {
    int v = 0;
    for (int w = 0; w < n; ++w) v += c[w];
    return v;
  };
  for (int i = threadIdx.x; i <= g.L; i += 64 * NW) offs[i] = g.tab_offs[i];
  int row[M], id[M];  // this thread's positions of the table in a block
  auto load_table = [&](int t0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int pos = t0 + i * 64 * NW + threadIdx.x;
      row[i] = pos < live ? g.tab_perm[pos] : -1;
      if ((uint32_t)row[i] >= (uint32_t)g.rows) row[i] = -1;
      id[i] = row[i] < 0 ? -1 : g.ids[row[i]];
    }
  };
  load_table(first);
  {
    // by blocks, a wave two at a time as long as they are whole
    int before = 0, rest = 0;
    auto count_run = [&](int r, const int (&e)[RUN]) __attribute__((always_inline)) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < RUN; ++i) n += __builtin_popcountll(__ballot(bare(e[i])));
      before += r < first ? n : 0;
      rest += r < first ? 0 : n;
    };
    int r = wave * kOrder;
    for (; r + (NW + 1) * kOrder <= g.rows; r += 2 * NW * kOrder) {
      int e[2][RUN];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < RUN; ++i) e[h][i] = (g.ids + r + h * NW * kOrder + lane)[64 * i];
      count_run(r, e[0]);
      count_run(r + NW * kOrder, e[1]);
    }
    for (; r < g.rows; r += NW * kOrder) {
      int e[RUN];
#pragma unroll
      for (int i = 0; i < RUN; ++i) e[i] = r + 64 * i + lane < g.rows ? g.ids[r + 64 * i + lane] : 0;
      count_run(r, e);
    }
    if (lane == 0) {
      count[wave] = before;
      count[16 + wave] = rest;
    }
  }
  int before = 0, all = 0;  // tokens without an adapter before the block and in all, as they lie behind the table's
  bool over = false;
  for (int t0 = first; t0 < end; t0 += kOrder) {
    if (threadIdx.x < kOrder / 32) listed[threadIdx.x] = 0;
    uint64_t m[M];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int t = t0 + (wave * M + i) * 64 + lane;
      m[i] = __ballot(t < g.rows && bare(g.ids[t]));
      mine += __builtin_popcountll(m[i]);
    }
    if (lane == 0) count[32 + wave] = mine;
    __syncthreads();
    if (t0 == first) {
      before = waves_sum(count, NW);
      all = before + waves_sum(count + 16, NW);
      over = live + all > g.rows;  // (in every workgroup)
    }
    if (over) {
      int lb = 0, la = 0;  // listed tokens without an adapter before this workgroup's, and in all
      for (int i = threadIdx.x; i < live; i += 64 * NW) {
        const int r = g.tab_perm[i];
        if ((uint32_t)r >= (uint32_t)g.rows || !bare(g.ids[r])) continue;
        ++la;
        if (r < first) ++lb;
        if (r >= t0 && r < t0 + kOrder) atomicOr(listed + (r - t0) / 32, 1u << (r & 31));
      }
      lb = wave_sum(lb);
      la = wave_sum(la);
      __syncthreads();
      mine = 0;
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const int w = 2 * (wave * M + i);
        m[i] &= ~((uint64_t)listed[w + 1] << 32 | listed[w]);
        mine += __builtin_popcountll(m[i]);
      }
      if (lane == 0) {
        count[wave] = lb;
        count[16 + wave] = la;
        count[32 + wave] = mine;
      }
      __syncthreads();
      if (t0 == first) {
        before -= waves_sum(count, NW);
        all -= waves_sum(count + 16, NW);
      }
    }
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int pos = t0 + i * 64 * NW + threadIdx.x;
      if (pos >= g.rows || (pos >= live && pos < live + all)) continue;
      int2 o = make_int2(-1, -1);
      if (bare(id[i])) o.x = over ? row[i] : -1;
      else if (offs[id[i]] <= pos && pos < offs[id[i] + 1]) o = make_int2(row[i], id[i]);
      g.order[pos] = o;
    }
    int at = live + before + waves_sum(count + 32, wave);
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int to = at + __builtin_popcountll(m[i] & (((uint64_t)1 << lane) - 1));
      if (m[i] >> lane & 1 && (uint32_t)to < (uint32_t)g.rows)
        g.order[to] = make_int2(t0 + (wave * M + i) * 64 + lane, -1);
      at += __builtin_popcountll(m[i]);
    }
    if (t0 + kOrder < end) {
      before += waves_sum(count + 32, NW);
      load_table(t0 + kOrder);
      __syncthreads();  // the counts and bits have been read
    }
  }
}

// Few tokens: a workgroup has one token and one slice of K.  Its waves share the
// ranks; a wave reads 512 consecutive elements of a row of a at a time.
template <int DT, bool VEC, int RW>
__global__ __launch_bounds__(512) void k_lora_down_one(Q8LoraArgs g) {
  typedef typename Elem<DT>::type T;
  constexpr int N = 16 / (int)sizeof(T), H = 8 / N;
  const int row = blockIdx.x / g.slices, sl = blockIdx.x % g.slices;
  const int e = row < g.rows ? g.ids[row] : -1;
  if ((uint32_t)e >= (uint32_t)g.L) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave * RW >= g.R) return;
  const int units = (g.K + 511) / 512;
  const int last = (sl + 1) * units / g.slices;
  const T *x = static_cast<const T *>(g.x) + row * g.ldx;
  const T *a = static_cast<const T *>(g.a) + ((int64_t)e * g.R + wave * RW) * g.K;
  float acc[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) acc[i] = 0.f;
#pragma unroll 2
  for (int u = sl * units / g.slices; u < last; ++u) {
    const int k = 512 * u + 8 * lane, kk = min(k, g.K - 8);
    float v[8];
    Pack<T, N> w[RW][H];
    if constexpr (VEC) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const Pack<T, N> p = reinterpret_cast<const Pack<T, N> *>(x + kk)[h];
#pragma unroll
        for (int j = 0; j < N; ++j) v[h * N + j] = (float)p.v[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)x[kk + j];
    }
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
      for (int h = 0; h < H; ++h)
        w[i][h] = reinterpret_cast<const Pack<T, N> *>(a + (int64_t)min(i, g.R - 1 - wave * RW) * g.K + kk)[h];
    if (k >= g.K) continue;
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i] = fmaf(v[j], (float)w[i][j / N].v[j % N], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < RW; ++i) acc[i] = group_sum<64>(acc[i]);
  if (lane == 63) {
#pragma unroll
    for (int i = 0; i < RW; i += 4)
      put_u<DT>(g, sl, row, 0, e, wave * RW + i, v4f{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]});
  }
}

// u of up to BM tokens of one adapter, over one of the slices of K, by matrix
// instructions.  K goes by stages of SB bytes of every row through a ring in LDS,
// filled by direct loads of whole runs of rows.  A stage costs a barrier and a wait
// for LDS whatever its size, so it is as long as three of them fit (509 tokens x
// 6144 of rank 16: 256 bytes 12.6 us, 512 10.1, 1024 9.5).  Each of the four waves has every
// fourth 64 bytes of a row, and the waves' sums are added through LDS in order.  RT
// groups of 16 ranks (rows past R repeat its last).
//
// LDS: piece p (16 bytes) of row r's stage lies at place p ^ (r % 16).
//
// (Workgroups that each begin at another stage take 1.35 times as long: side by
// side they read an adapter's a while it is near.)
constexpr int down_bytes(int bm, int rt) {
  return bm + 16 * rt <= 96 ? 512 : 256;
}
constexpr int down_stages(int bm, int rt) {
  const int n = (150 << 10) / ((bm + 16 * rt) * down_bytes(bm, rt));
  return n < 6 ? n : 6;
}

template <int DT, bool VEC, int BM, int RT>
__global__ __launch_bounds__(256) void k_lora_down(Q8LoraArgs g, int wgs) {
  typedef typename Elem<DT>::type T;
  typedef typename Oper<DT>::type O;
  constexpr int NW = 4, SB = down_bytes(BM, RT), ROWS = BM + 16 * RT, STAGE = ROWS * SB, PIECES = SB / 16;
  constexpr int STAGES = down_stages(BM, RT), KS = SB / 64 / NW;  // steps of a wave in a stage
  constexpr int RPL = 1024 / SB;                                  // rows of a load
  constexpr int TM = BM / 16;
  constexpr int NX = BM / RPL / NW, NL = ROWS / RPL / NW;  // loads of a wave in a stage, the tokens' NX first
  constexpr int ASYNC = VEC ? NL : NL - NX;                // of them straight to LDS
  static_assert(STAGES >= 3 && STAGES * STAGE >= NW * RT * 1024, "the sums take the ring's place");
  static_assert(ASYNC * (STAGES - 1) < 64, "vmcnt range");
  // (The rows lie behind the ring, in one object with it: beside another object the
  // compiler waits for every load into the ring before it reads it.)
  static_assert(STAGES * STAGE >= kOrderInts * 4, "the order's counts and ranges");
  __shared__ __align__(16) unsigned char ring[STAGES * STAGE + BM * 4];
  int *rows = reinterpret_cast<int *>(ring + STAGES * STAGE);
  if ((int)blockIdx.x >= wgs) {
    const int blocks = (g.rows + kOrder - 1) / kOrder;
    order_tokens<NW>(g, blockIdx.x - wgs, (blocks + kOrderWgs - 1) / kOrderWgs, reinterpret_cast<int *>(ring));
    return;
  }
  Q8Args tab{};
  tab.E = g.L;
  tab.P = g.rows;
  tab.offs = g.tab_offs;
  const Tile t = expert_tile<BM>(tab, g.slices);
  if (t.n <= 0) return;
  if (threadIdx.x < BM) {
    const int p = g.tab_perm[t.r0 + min((int)threadIdx.x, t.n - 1)];
    rows[threadIdx.x] = (int)threadIdx.x < t.n && (uint32_t)p < (uint32_t)g.rows ? p : -1;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pieces = g.K / (16 / (int)sizeof(T)), stages = (pieces + PIECES - 1) / PIECES;
  const int first = (int)((int64_t)t.nb * stages / g.slices), end = (int)((int64_t)(t.nb + 1) * stages / g.slices);

  const char *src[NL];
  uint32_t pl[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int r = (i * NW + wave) * RPL + lane / PIECES;
    pl[i] = (lane & (PIECES - 1)) ^ (r & 15);
    src[i] = i < NX ? static_cast<const char *>(g.x) + max(rows[r], 0) * g.ldx * (int64_t)sizeof(T)
                    : static_cast<const char *>(g.a) +
                          ((int64_t)t.e * g.R + min(r - BM, g.R - 1)) * g.K * (int64_t)sizeof(T);
  }
  auto issue = [&](int c) {
    unsigned char *buf = ring + ((c - first) % STAGES) * STAGE;
    const uint32_t last = min(PIECES, pieces - PIECES * c) - 1;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const char *p = src[i] + (int64_t)c * SB + 16 * min(pl[i], last);
      unsigned char *to = buf + (i * NW + wave) * 1024;
      if (VEC || i >= NX) {
        __builtin_amdgcn_global_load_lds(p, (lds_void *)to, 16, 0, 0);
      } else {  // rows that start at any element
        Pack<T, 16 / (int)sizeof(T)> v;
#pragma unroll
        for (int k = 0; k < 16 / (int)sizeof(T); ++k) v.v[k] = reinterpret_cast<const T *>(p)[k];
        *reinterpret_cast<Pack<T, 16 / (int)sizeof(T)> *>(to + 16 * lane) = v;
      }
    }
  };
  v4f acc[RT][TM];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < STAGES - 1; ++c) {
    if (first + c < end) issue(first + c);
    keep_order();
  }
  for (int c = first; c < end; ++c) {
    // stage c has landed for every wave, and no wave reads stage c - 1 any more
    if (c + STAGES - 1 <= end) stage_barrier<ASYNC *(STAGES - 2)>();
    else stage_barrier<0>();
    if (c + STAGES - 1 < end) issue(c + STAGES - 1);
    const unsigned char *buf = ring + ((c - first) % STAGES) * STAGE + li * SB;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int p = 4 * (k * NW + wave);
      if (PIECES * c + p >= pieces) continue;  // (pieces are a multiple of 4)
      const unsigned char *b = buf + 16 * ((p + lg) ^ li);
      O x[TM], w[RT];
#pragma unroll
      for (int j = 0; j < TM; ++j) x[j] = *reinterpret_cast<const O *>(b + 16 * j * SB);
#pragma unroll
      for (int i = 0; i < RT; ++i) w[i] = *reinterpret_cast<const O *>(b + (BM + 16 * i) * SB);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = mul16<DT>(w[i], x[j], acc[i][j]);
    }
  }
  // lane (li, lg) has token li's ranks 4 lg .. 4 lg + 3 of each 16
  float *part = reinterpret_cast<float *>(ring);
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    stage_barrier<0>();
#pragma unroll
    for (int i = 0; i < RT; ++i)
      *reinterpret_cast<v4f *>(part + (wave * RT + i) * 256 + 4 * lane) = acc[i][j];
    __syncthreads();
    for (int o = threadIdx.x; o < RT * 64; o += 64 * NW) {
      v4f sum = *reinterpret_cast<const v4f *>(part + 4 * o);
#pragma unroll
      for (int w = 1; w < NW; ++w) sum += *reinterpret_cast<const v4f *>(part + w * RT * 256 + 4 * o);
      const int i = 16 * j + (o & 15), r = 16 * (o / 64) + 4 * ((o & 63) / 16);
      if (rows[i] >= 0 && r < ((g.R + 15) & ~15)) put_u<DT>(g, t.nb, rows[i], t.r0 + i, t.e, r, sum);
    }
  }
}

// Parts of K (a power of two), so that a batch's tiles fill the chip even if one
// adapter has all its tokens; the workspace's size bounds them too.
constexpr int kMaxSlices = 8;
int slices_of(int T, int tiles, int most) {
  int s = 1;
  while (s < most && 2 * s * tiles <= 256 && 2 * s <= 1 + 8192 / T) s *= 2;
  return s;
}

bool tiled(Variant v) { return v == kTile128 || v == kTile128Deep || v == kTile256; }

// As without adapters, by times of the product alone: with them the forms have not been
// compared (the 64 x 64 ring has 128 registers then, and in fp32 keeps ten values in
// memory).  The sweep has no form with adapters: the 128 x 128 tiles are within 13 % of
// the best of the forms there.
Variant lora_variant(const Q8LoraArgs &a) {
  const Variant v = dense_variant(a);
  return v == kSweep64 ? kTile128 : v;
}

size_t order_bytes(int T) { return ((size_t)T * sizeof(int2) + 255) / 256 * 256; }

}  // namespace

size_t gemm_q8_lora_workspace(int T, int R) {
  const int64_t parts = 4 * std::min<int64_t>((int64_t)kMaxSlices * T, (int64_t)T + 8192) * R;
  const int64_t pieces = 6 * (((int64_t)T + 31) / 32 * 32) * ((R + 15) / 16 * 16);  // (three of two bytes)
  return order_bytes(T) + (size_t)std::max(parts, pieces);
}

bool gemm_q8_lora_fits(const Q8LoraArgs &a) {
  const Variant v = lora_variant(a);
  // (the tiles name rows of q by 32-bit byte offsets)
  if (tiled(v) && (int64_t)a.rows * a.K >= (int64_t)1 << 32) return false;
  return workgroups(a, v) * kShapes[v].threads < ((int64_t)1 << 31);
}

hipError_t launch_gemm_q8_lora(int dt, Q8LoraArgs a, void *workspace, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  a.order = static_cast<int2 *>(workspace);
  a.u = reinterpret_cast<float *>(static_cast<char *>(workspace) + order_bytes(a.rows));
  const Variant v = lora_variant(a);
  a.pieces = tiled(v);
  const bool one = !a.pieces && a.rows <= 64;  // a workgroup for each token
  const int rt = a.R <= 16 ? 1 : a.R <= 32 ? 2 : a.R <= 64 ? 4 : 8;
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                   (uint64_t)a.ldx * (dt == COLI_F32 ? 4 : 2) % 16 == 0;
  // (x that starts at any element goes by 16 tokens: both launches of 300 tokens x 4000
  // x 6144 of rank 16 and 128 take 38.5 and 57 us, with aligned rows 36 and 49.)
  // Tokens of a tile: a tile costs its tokens' and its adapter's rows, and a CU
  // works through its tiles one after another.  (8192 x 6144 of rank 64, 16 adapters:
  // 272 tiles of 32 tokens 52-56 us, 187 of 48 38-43.)
  int bm = 16;
  if (!one && vec) {
    int64_t least = INT64_MAX;
    for (int m = 16; m <= 64; m += 16) {
      const int64_t cost = (a.rows / m + std::min(a.rows, a.L) + 255) / 256 * (m + 16 * rt);
      if (cost < least) least = cost, bm = m;
    }
  }
  const int tiles = one ? a.rows : a.rows / bm + std::min(a.rows, a.L);  // at most
  a.slices = a.pieces ? 1 : slices_of(a.rows, one ? a.rows : (a.rows + bm - 1) / bm, lora_parts(kShapes[v].bm));
  const int wgs = (int)(((int64_t)tiles * a.slices + 7) / 8 * 8);
  const int extra = std::min((a.rows + kOrder - 1) / kOrder, kOrderWgs);  // workgroups of the order
  if (one) a.order = nullptr;
  return by_dtype(dt, [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    auto few = [&](auto vecc) {
      constexpr bool VEC = decltype(vecc)::value;
      const dim3 grid(a.rows * a.slices), block(512);
      if (a.R <= 32) hipLaunchKernelGGL((k_lora_down_one<DT, VEC, 4>), grid, block, 0, st, a);
      else if (a.R <= 64) hipLaunchKernelGGL((k_lora_down_one<DT, VEC, 8>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((k_lora_down_one<DT, VEC, 16>), grid, block, 0, st, a);
    };
    auto many = [&](auto vecc, auto bmc) {
      constexpr bool VEC = decltype(vecc)::value;
      constexpr int BM = decltype(bmc)::value;
      const dim3 grid(wgs + extra), block(256);
      if (rt == 1) hipLaunchKernelGGL((k_lora_down<DT, VEC, BM, 1>), grid, block, 0, st, a, wgs);
      else if (rt == 2) hipLaunchKernelGGL((k_lora_down<DT, VEC, BM, 2>), grid, block, 0, st, a, wgs);
      else if (rt == 4) hipLaunchKernelGGL((k_lora_down<DT, VEC, BM, 4>), grid, block, 0, st, a, wgs);
      else hipLaunchKernelGGL((k_lora_down<DT, VEC, BM, 8>), grid, block, 0, st, a, wgs);
    };
    if (one && vec) few(std::true_type());
    else if (one) few(std::false_type());
    else if (!vec) many(std::false_type(), std::integral_constant<int, 16>());
    else if (bm == 16) many(std::true_type(), std::integral_constant<int, 16>());
    else if (bm == 32) many(std::true_type(), std::integral_constant<int, 32>());
    else if (bm == 48) many(std::true_type(), std::integral_constant<int, 48>());
    else many(std::true_type(), std::integral_constant<int, 64>());
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    run_dense<DT>(a, v, st);
    return hipGetLastError();
  });
}

}  // namespace coli
