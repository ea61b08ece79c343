// Which tile and how many splits of K a product of the feed-forward block takes,
// and its launch.
#pragma once

#include "ffn_gemm.h"

namespace moe {

// A tile: rows x columns (of all panels), K per stage, workgroups that a CU's LDS
// holds, and its times in ns, fitted to measured products (16384 x 2048 x 4096 down to
// 64 x 2048 x 768): a CU that runs n of them takes wait + n busy for a K stage of each;
// fixed is what a workgroup takes beyond its stages (launch, first loads, epilogue).
// The 16-row tiles are for few rows, where the other tiles' MFMAs on rows that are not
// there take longer than the weights' way in (fp32, 1 x 7168 x 2048: up and gate 37 ->
// 22 us, down 22 -> 13 us), and for products of few tiles in all (64 x 128 x 256 fp32:
// down in one launch at 6.8 us instead of 4.3 and a join of 2.9); 3 rows of them instead
// of one of 64 are slower (48 x 512 x 512 fp32: 21 against 16 us with joins).
struct TileCost {
  int bm, bn, bk, per_cu;
  float wait_ns, busy_ns, fixed_ns;
};
constexpr TileCost kBfTiles[] = {
    {256, 256, 64, 1, 0.f, 1560.f, 6000.f},
    {128, 128, 64, 2, 280.f, 440.f, 4000.f},
    {64, 128, 64, 2, 50.f, 370.f, 3500.f},
    {16, 128, 64, 2, 150.f, 250.f, 3000.f},
    {256, 128, 64, 1, 0.f, 950.f, 4500.f},
};
constexpr TileCost kF32Tiles[] = {
    {128, 128, 32, 2, 70.f, 2130.f, 2500.f},
    {64, 64, 32, 5, 300.f, 510.f, 2000.f},
    {16, 64, 32, 5, 250.f, 350.f, 2300.f},
};
constexpr int kCus = 256;
// Workgroups of a launch: with up to 512 threads each, below 2^32 threads. The largest
// tile stays below it for every shape that check_ffn lets through.
constexpr int64_t kMaxGroups = (1 << 22) + (1 << 21);

struct GemmPlan {
  int tile;          // index into the table
  int stages, split_stages, splits;
  int tiles_m, tiles_n;
  size_t part_bytes;
};

// The tile and the splits with the least estimated time: the workgroups of a CU, as
// many at once as it holds, plus the splits' sums' way through memory and the
// launch that joins them. The stages' times are of operands in the caches: weights that
// come from HBM take longer than it expects (64 x 7168 x 2048 bf16: 9 and 7 us expected,
// 17 and 13 taken).
// `tiles`: bit mask of the tiles that the product has kernels for.
inline GemmPlan plan_gemm(bool f32, unsigned tiles, bool dual, int64_t M, int64_t N, int64_t K,
                          int pairs) {
  GemmPlan best = {};
  float best_ns = 3.0e38f;
  const int n = f32 ? 3 : 5;
  for (int t = 0; t < n; ++t) {
    if (!(tiles >> t & 1)) continue;
    const TileCost& c = f32 ? kF32Tiles[t] : kBfTiles[t];
    GemmPlan p = {};
    p.tile = t;
    p.stages = (int)((K + c.bk - 1) / c.bk) * pairs;
    p.tiles_m = (int)((M + c.bm - 1) / c.bm);
    const int cols = dual ? c.bn / 2 : c.bn;
    p.tiles_n = (int)((N + cols - 1) / cols);
    const int64_t wgs = (int64_t)p.tiles_m * p.tiles_n;
    if (wgs > kMaxGroups) continue;
    for (int s = 1; s <= 32 && s <= p.stages; ++s) {
      p.split_stages = (p.stages + s - 1) / s;
      p.splits = (p.stages + p.split_stages - 1) / p.split_stages;
      if (p.splits != s) continue;
      if (s > 1 && wgs * s > 4 * kCus) break;
      const int64_t per = (wgs * s + kCus - 1) / kCus;  // workgroups of the fullest CU
      float ns = 0.f;
      for (int64_t left = per; left > 0; left -= c.per_cu) {
        const float at_once = (float)(left < c.per_cu ? left : c.per_cu);
        ns += c.fixed_ns + p.split_stages * (c.wait_ns + at_once * c.busy_ns);
        if (ns > best_ns) break;
      }
      p.part_bytes = 0;
      if (s > 1) {
        p.part_bytes = (size_t)s * (dual ? 2 : 1) * (size_t)M * (size_t)N * 4;
        ns += 5000.f + (float)p.part_bytes * 2.f / 9000.f;
      }
      if (ns < best_ns) {
        best_ns = ns;
        best = p;
      }
    }
  }
  return best;
}

inline void apply_plan(const GemmPlan& p, GemmArgs* g, void* part) {
  g->stages = p.stages;
  g->split_stages = p.split_stages;
  g->splits = p.splits;
  g->tiles_m = p.tiles_m;
  g->tiles_n = p.tiles_n;
  g->part = (float*)part;
}

template <typename Core, typename EP>
void launch_tile(const GemmArgs& g, const EP& ep, hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)g.tiles_m * g.tiles_n * g.splits);
  gemm_kernel<Core, EP><<<grid, Core::THREADS, 0, st>>>(g, ep);
  if (g.splits > 1) {
    const int64_t n = g.M * ((g.N + 3) / 4);
    const int64_t b = (n + 255) / 256;
    gemm_join_kernel<Core::DUAL, EP><<<(unsigned)(b < 4096 ? b : 4096), 256, 0, st>>>(g, ep);
  }
}

// The tiles of a product with these operand orders.
template <bool DUAL, bool AKC, bool BKC>
constexpr unsigned tile_mask(bool f32) {
  return f32 ? (AKC ? 7u : 3u) : AKC ? 31u : 23u;  // 16 rows: K-contiguous A only
}

template <typename T, bool DUAL, bool AKC, bool BKC, typename EP>
void launch_gemm(const GemmPlan& p, const GemmArgs& g, const EP& ep, hipStream_t st) {
  constexpr int NP = DUAL ? 2 : 1;
  if constexpr (sizeof(T) == 4) {
    if (p.tile == 0) {
      launch_tile<TileCore<T, 128, 128, 2, DUAL, AKC, BKC, 2, 4, 2>>(g, ep, st);
      return;
    }
    if constexpr (AKC) {
      if (p.tile == 2) {
        if (p.tiles_m == 1)
          launch_tile<TileCore<T, 16, 64, NP, DUAL, AKC, BKC, 1, 2, 3, true>>(g, ep, st);
        else
          launch_tile<TileCore<T, 16, 64, NP, DUAL, AKC, BKC, 1, 2, 3>>(g, ep, st);
        return;
      }
    }
    launch_tile<TileCore<T, 64, 64, NP, DUAL, AKC, BKC, 2, 2, 2>>(g, ep, st);
  } else {
    if (p.tile == 0)
      launch_tile<TileCore<T, 256, 256, 2, DUAL, AKC, BKC, 2, 4, 2>>(g, ep, st);
    else if (p.tile == 1)
      launch_tile<TileCore<T, 128, 128, NP, DUAL, AKC, BKC, 2, 4, 2>>(g, ep, st);
    else if (p.tile == 4)
      launch_tile<TileCore<T, 256, 128, NP, DUAL, AKC, BKC, 4, 2, 3>>(g, ep, st);
    else if (p.tile == 2 && p.tiles_m == 1)
      launch_tile<TileCore<T, 64, 128, NP, DUAL, AKC, BKC, 2, 4, 3, true>>(g, ep, st);
    else if (p.tile == 2)
      launch_tile<TileCore<T, 64, 128, NP, DUAL, AKC, BKC, 2, 4, 3>>(g, ep, st);
    else if constexpr (AKC) {
      if (p.tiles_m == 1)
        launch_tile<TileCore<T, 16, 128, NP, DUAL, AKC, BKC, 1, 4, 4, true>>(g, ep, st);
      else
        launch_tile<TileCore<T, 16, 128, NP, DUAL, AKC, BKC, 1, 4, 4>>(g, ep, st);
    }
  }
}

// ------------------------------------------------------------ epilogues
struct NoPre {};

// h = SiLU(u) g from the fp32 sums; u and g kept for a backward pass. In bf16 h is rounded
// to the next product's operand, as the MoE layer's is: the outputs' error against 64 bits
// (2-norm) is 0.0023 so, 0.0017 from their own rounding alone. Kept in two bf16 parts it
// would take a third more MFMAs in the pass, which is bound by them for many tokens.
template <typename T>
struct EpSwiglu {
  T *h, *U, *G;
  int64_t ld;
  template <int W>
  using Pre = NoPre;
  template <typename P>
  __device__ __forceinline__ void pre(int64_t, int64_t, P&) const {}
  template <int W, typename P>
  __device__ __forceinline__ void operator()(int64_t m, int64_t n, const float (&u)[W],
                                             const float (&g)[W], const P&) const {
    const int64_t o = m * ld + n;
    float v[W];
#pragma unroll
    for (int r = 0; r < W; ++r) v[r] = silu_f32(u[r]) * g[r];
    store_n(h + o, v);
    if (U != nullptr) {
      store_n(U + o, u);
      store_n(G + o, g);
    }
  }
};
// One output, or the two panels' (DUAL).
template <typename T, bool DUAL = false>
struct EpStore {
  T *out0, *out1;
  int64_t ld;
  template <int W>
  using Pre = NoPre;
  template <typename P>
  __device__ __forceinline__ void pre(int64_t, int64_t, P&) const {}
  template <int W, typename P>
  __device__ __forceinline__ void operator()(int64_t m, int64_t n, const float (&v0)[W],
                                             const float (&v1)[W], const P&) const {
    store_n(out0 + m * ld + n, v0);
    if constexpr (DUAL) store_n(out1 + m * ld + n, v1);
  }
};
// From dh: dU, dG, and h again (all operands of the products that follow); h may
// be null (frozen weights). In bf16 they are rounded as such: 0.0023 instead of 0.0017 in
// each gradient; in two parts each the pass would take 22 / 12 of its MFMAs.
template <typename T>
struct EpSwigluBwd {
  const T *U, *G;
  T *dU, *dG, *h;
  int64_t ld;
  template <int W>
  struct Pre {
    Pack<T, W> u, g;
  };
  template <int W>
  __device__ __forceinline__ void pre(int64_t m, int64_t n, Pre<W>& p) const {
    p.u.load(U + m * ld + n);
    p.g.load(G + m * ld + n);
  }
  template <int W>
  __device__ __forceinline__ void operator()(int64_t m, int64_t n, const float (&dh)[W],
                                             const float (&)[W], const Pre<W>& p) const {
    const int64_t o = m * ld + n;
    float du[W], dg[W], hv[W];
#pragma unroll
    for (int r = 0; r < W; ++r) {
      const float u = p.u.get(r), g = p.g.get(r);
      const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-u));
      const float a = u * s;
      dg[r] = dh[r] * a;
      du[r] = dh[r] * g * (s * (1.0f + u * (1.0f - s)));
      hv[r] = a * g;
    }
    store_n(dU + o, du);
    store_n(dG + o, dg);
    if (h != nullptr) store_n(h + o, hv);
  }
};

// Clears n floats' worth of bytes (a kernel: a captured graph holds no memset).
hipError_t launch_zero(void* p, size_t bytes, hipStream_t st);

// What both passes' entry points check first.
moe_status check_ffn(const moe_ffn_shape* s);

}  // namespace moe
