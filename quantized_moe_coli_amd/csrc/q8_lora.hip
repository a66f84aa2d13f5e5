// q8_lora.hip -- the dense 8-bit product with low-rank adapters of many
// requests beside it:
//   y[t][n] = s_t ws_n sum_k q[t][k] w[n][k] (+ bias[n]) + c_a sum_r u[t][r] b_a[n][r],
//   u[t][r] = sum_k x[t][k] a_a[r][k],   a = ids[t].
//
// Two launches: u, by adapter over the batch's table of its tokens, into the
// caller's workspace, and the product (q8_kernels.hpp), whose kernels add the
// adapters' part to the sums in binary32 before their one rounding (lora.hpp).
#include <algorithm>

#include "q8_kernels.hpp"

namespace coli {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// Eight operand elements of one row.
template <int DT> struct Oper { typedef float type __attribute__((ext_vector_type(8))); };
template <> struct Oper<COLI_BF16> { typedef v8bf type; };
template <> struct Oper<COLI_F16> { typedef v8h type; };

template <int DT, bool VEC>
__device__ __forceinline__ typename Oper<DT>::type operand(const typename Elem<DT>::type *p) {
  typedef typename Elem<DT>::type T;
  typename Oper<DT>::type o;
  if constexpr (VEC) {
    constexpr int N = 16 / (int)sizeof(T);
#pragma unroll
    for (int k = 0; k < 8 / N; ++k) {
      const Pack<T, N> w = reinterpret_cast<const Pack<T, N> *>(p)[k];
#pragma unroll
      for (int j = 0; j < N; ++j) o[k * N + j] = w.v[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = p[j];
  }
  return o;
}

// 16 rows x 16 rows over k = 32, of which lane l has elements 8 (l / 16) ..
// of row l % 16 of each.
template <int DT>
__device__ __forceinline__ v4f mul16(typename Oper<DT>::type w, typename Oper<DT>::type x, v4f c) {
  if constexpr (DT == COLI_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
  } else if constexpr (DT == COLI_F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x, c, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(w[j], x[j], c, 0, 0, 0);
    return c;
  }
}

// The tokens in order of their adapters: the table's, and behind them, in order,
// the tokens without one, which the table does not list.  Workgroup b writes the
// table's part of positions kOrder b .. and the tokens without an adapter among
// tokens kOrder b ..; those before them it counts itself.
constexpr int kOrder = 1024;

template <int NW>
__device__ __forceinline__ void order_tokens(const Q8LoraArgs &g, int b, int *count) {
  static_assert(NW <= 16 && kOrder % (64 * NW) == 0, "whole rounds");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t0 = b * kOrder, live = min(max(g.tab_offs[g.L], 0), g.rows);
  auto bare = [&](int t) { return t < g.rows && (uint32_t)g.ids[t] >= (uint32_t)g.L; };
  int before = 0, mine = 0;  // (before: of this wave's share)
  for (int t = threadIdx.x; t < t0; t += 64 * NW) before += bare(t);
  uint64_t m[kOrder / 64 / NW];
#pragma unroll
  for (int i = 0; i < kOrder / 64 / NW; ++i) {
    m[i] = __ballot(bare(t0 + (wave * (kOrder / 64 / NW) + i) * 64 + lane));
    mine += __builtin_popcountll(m[i]);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) before += __shfl_xor(before, d, 64);
  if (lane == 0) {
    count[wave] = before;
    count[16 + wave] = mine;
  }
  for (int i = t0 + threadIdx.x; i < min(t0 + kOrder, live); i += 64 * NW) g.order[i] = g.tab_perm[i];
  __syncthreads();
  int at = live;
  for (int w = 0; w < NW; ++w) at += count[w] + (w < wave ? count[16 + w] : 0);
#pragma unroll
  for (int i = 0; i < kOrder / 64 / NW; ++i) {
    const int to = at + __builtin_popcountll(m[i] & (((uint64_t)1 << lane) - 1));
    if (m[i] >> lane & 1 && to < g.rows) g.order[to] = t0 + (wave * (kOrder / 64 / NW) + i) * 64 + lane;
    at += __builtin_popcountll(m[i]);
  }
}

// u of up to BM tokens of one adapter, over one of the slices of K.  The NW
// waves share the slice's lines (128 bytes of every row) among them, each with D
// of its lines on the way, and their sums are added through LDS in order.  RT
// groups of 16 ranks (rows past R repeat its last).  single: a tile is one token,
// found by its id, with no table to look through.
template <int DT, bool VEC, int BM, int NW, int RT>
__global__ __launch_bounds__(64 * NW) void k_lora_down(Q8LoraArgs g, int wgs, bool single) {
  typedef typename Elem<DT>::type T;
  typedef typename Oper<DT>::type O;
  constexpr int TM = BM / 16;
  constexpr int H = 4 / (int)sizeof(T);          // steps of k = 32 in a line
  constexpr int D = TM + RT <= 3 ? 4 : TM + RT <= 5 ? 3 : 2;
  __shared__ __align__(16) float part[NW][RT * 256];
  __shared__ int rows[BM < 32 ? 32 : BM];
  if ((int)blockIdx.x >= wgs) {
    order_tokens<NW>(g, blockIdx.x - wgs, rows);
    return;
  }
  Tile t;
  if (single) {
    const int row = blockIdx.x / g.slices;
    if (row >= g.rows) return;
    t = Tile{g.ids[row], row, 1, (int)blockIdx.x % g.slices};
    if ((uint32_t)t.e >= (uint32_t)g.L) return;
    if (threadIdx.x < BM) rows[threadIdx.x] = threadIdx.x == 0 ? row : -1;
  } else {
    Q8Args tab{};
    tab.E = g.L;
    tab.P = g.rows;
    tab.offs = g.tab_offs;
    t = expert_tile<BM>(tab, g.slices);
    if (t.n <= 0) return;
    if (threadIdx.x < BM) {
      const int p = g.tab_perm[t.r0 + min((int)threadIdx.x, t.n - 1)];
      rows[threadIdx.x] = (int)threadIdx.x < t.n && (uint32_t)p < (uint32_t)g.rows ? p : -1;
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lines = (g.K / 32 + H - 1) / H;
  const int last = (int)((int64_t)(t.nb + 1) * lines / g.slices);
  int c = (int)((int64_t)t.nb * lines / g.slices) + wave;

  const T *xr[TM], *ar[RT];
#pragma unroll
  for (int j = 0; j < TM; ++j)
    xr[j] = static_cast<const T *>(g.x) + (single ? t.r0 : max(rows[16 * j + li], 0)) * g.ldx + 8 * lg;
#pragma unroll
  for (int i = 0; i < RT; ++i)
    ar[i] = static_cast<const T *>(g.a) + ((int64_t)t.e * g.R + min(16 * i + li, g.R - 1)) * g.K + 8 * lg;
  v4f acc[RT][TM];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  O x[D][H][TM], w[D][H][RT];
  // (lines past the slice's end ask for its last again; a half line for its first half)
  auto load = [&](int d, int l) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int k = min(32 * (H * min(l, last - 1) + h), g.K - 32);
#pragma unroll
      for (int j = 0; j < TM; ++j) x[d][h][j] = operand<DT, VEC>(xr[j] + k);
#pragma unroll
      for (int i = 0; i < RT; ++i) w[d][h][i] = operand<DT, true>(ar[i] + k);
    }
  };
  auto mul = [&](int d, int l) {
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (32 * (H * l + h) < g.K) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < TM; ++j) acc[i][j] = mul16<DT>(w[d][h][i], x[d][h][j], acc[i][j]);
      }
  };
  if (c < last) {
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, c + d * NW);
    for (; c + D * NW < last; c += D * NW) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        mul(d, c + d * NW);
        load(d, c + (D + d) * NW);
      }
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (c + d * NW < last) mul(d, c + d * NW);
  }
  // lane (li, lg) has token li's ranks 4 lg .. 4 lg + 3 of each 16
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    if (j > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i) *reinterpret_cast<v4f *>(&part[wave][i * 256 + 4 * lane]) = acc[i][j];
    __syncthreads();
    for (int o = threadIdx.x; o < RT * 64; o += 64 * NW) {
      v4f sum = *reinterpret_cast<const v4f *>(&part[0][4 * o]);
#pragma unroll
      for (int w = 1; w < NW; ++w) sum += *reinterpret_cast<const v4f *>(&part[w][4 * o]);
      const int row = rows[16 * j + (o & 15)], r = 16 * (o / 64) + 4 * ((o & 63) / 16);
      if (row >= 0 && r < g.R)
        *reinterpret_cast<v4f *>(g.u + ((int64_t)t.nb * g.rows + row) * g.R + r) = sum;
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

// As without adapters, but for the sweep, which has no form with them: the
// 128 x 128 tiles are within 13 % of the best of the forms there.
Variant lora_variant(const Q8LoraArgs &a) {
  const Variant v = dense_variant(a);
  return v == kSweep64 ? kTile128 : v;
}

size_t order_bytes(int T) { return ((size_t)T * sizeof(int32_t) + 255) / 256 * 256; }

}  // namespace

size_t gemm_q8_lora_workspace(int T, int R) {
  return order_bytes(T) + (size_t)std::min<int64_t>((int64_t)kMaxSlices * T, (int64_t)T + 8192) * R * sizeof(float);
}

bool gemm_q8_lora_fits(const Q8LoraArgs &a) {
  const Variant v = lora_variant(a);
  // (the tiles name rows of q by 32-bit byte offsets)
  if (tiled(v) && (int64_t)a.rows * a.K >= (int64_t)1 << 32) return false;
  return workgroups(a, v) * kShapes[v].threads < ((int64_t)1 << 31);
}

hipError_t launch_gemm_q8_lora(int dt, Q8LoraArgs a, void *workspace, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  a.order = static_cast<int32_t *>(workspace);
  a.u = reinterpret_cast<float *>(static_cast<char *>(workspace) + order_bytes(a.rows));
  const Variant v = lora_variant(a);
  // a tile for each token where there are few; tiles of 32 tokens where adapters
  // have that many, on average over those that the caller holds
  const bool single = a.rows <= 64, many = a.rows / a.L >= 32;
  const int bm = many ? 32 : 16;
  a.slices = slices_of(a.rows, single ? a.rows : (a.rows + bm - 1) / bm, lora_parts(kShapes[v].bm));
  const int64_t tiles = single ? a.rows : a.rows / bm + std::min(a.rows, a.L);
  const int wgs = (int)((tiles * a.slices + 7) / 8 * 8);
  const int extra = tiled(v) ? (a.rows + kOrder - 1) / kOrder : 0;
  return by_dtype(dt, [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    typedef typename Elem<DT>::type T;
    const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (uint64_t)a.ldx * sizeof(T) % 16 == 0;
    auto go = [&](auto vecc, auto bmc, auto rtc) {
      constexpr int BM = decltype(bmc)::value, NW = 8;
      hipLaunchKernelGGL((k_lora_down<DT, decltype(vecc)::value, BM, NW, decltype(rtc)::value>), dim3(wgs + extra),
                         dim3(64 * NW), 0, st, a, wgs, single);
    };
    auto by_rank = [&](auto vecc, auto bmc) {
      if (a.R <= 16) go(vecc, bmc, std::integral_constant<int, 1>());
      else if (a.R <= 32) go(vecc, bmc, std::integral_constant<int, 2>());
      else if (a.R <= 64) go(vecc, bmc, std::integral_constant<int, 4>());
      else go(vecc, bmc, std::integral_constant<int, 8>());
    };
    auto by_tile = [&](auto vecc) {
      if (many) by_rank(vecc, std::integral_constant<int, 32>());
      else by_rank(vecc, std::integral_constant<int, 16>());
    };
    if (vec) by_tile(std::true_type());
    else by_tile(std::false_type());
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    run_dense<DT>(a, v, st);
    return hipGetLastError();
  });
}

}  // namespace coli
