// One workgroup's output tile of C = A . B for the dense feed-forward block's
// products, whose operands come in both orders: forward X W (B's columns
// contiguous), dO W^T (both operands' K contiguous), X^T dU (K outermost in both).
//
//   KC operand: rows of K contiguous values (A [M][K], B [N][K])
//   MC operand: K rows of contiguous values (A [K][M], B [K][N])
//
// C may have two panels of columns with a B of their own (DUAL: up and gate, or
// their gradients), and K may run over two pairs of operands in turn (dX = dU
// W_up^T + dG W_gate^T).
//
// bf16 (BfCore): K stages of 64 go from global memory straight into a ring of
// LDS slots (16 bytes per lane). KC operands lie there as rows of 128 bytes and
// are read by ds_read_b128, MC operands as K rows of a panel of up to 128
// columns and are read transposed (ds_read_b64_tr_b16); both with the chunk
// orders that the MoE layer's tile core measured free of bank conflicts. The MFMA
// takes B's fragment as its first operand, so a lane ends up with 4 consecutive
// columns of one row and loads and stores them as one access.
//
// The operands are addressed from a base that moves along K with the stages
// (scalar arithmetic), so an array may exceed the 4 GiB of a buffer's range;
// out-of-range rows, columns and K values read as zeros.
//
// fp32 (F32Core): the same interface on v_mfma_f32_16x16x4_f32; the 32x slower
// matrix rate leaves time for staging through registers.
#pragma once

#include "ffn_common.h"
#include "gemm_direct.h"

namespace moe {

struct GemmArgs {
  const void* A[2];       // per pair of operands
  const void* B[2][2];    // per pair, per panel (DUAL)
  int64_t lda, ldb;       // elements from one row (KC) or K row (MC) to the next
  int64_t M, N;           // N: columns of one panel's C
  int64_t K[2];
  int pairs;              // 1 or 2
  int stages;             // K stages of all pairs
  int split_stages;       // K stages per split
  int splits;
  int tiles_m, tiles_n;
  float* part;            // splits > 1: [splits][panels][M][N]
};

constexpr uint32_t kOutOfRange = 0x80000000u;  // above every record count used here

// A buffer descriptor for `left` bytes from base on (none when left <= 0).
__device__ __forceinline__ i32x4_t window_srd(uint64_t base, int64_t left) {
  i32x4_t r;
  r.x = (int)(uint32_t)base;
  r.y = (int)((base >> 32) & 0xFFFFu);
  r.z = left <= 0 ? 0 : left > 0x7FFFFFFF ? 0x7FFFFFFF : (int)left;
  r.w = 0x00020000;
  return r;
}

// One operand (R tile rows or columns in panels of PW, NB bases) in LDS.
template <bool KC, int R, int PW, int BASES, int NW>
struct BfOperand {
  static constexpr int BK = 64;
  static constexpr int BYTES = R * BK * 2;
  static constexpr int INSTR = BYTES / 1024;
  static constexpr int PER_WAVE = (INSTR + NW - 1) / NW;
  static constexpr int PANEL_INSTR = PW * BK * 2 / 1024;
  static_assert(KC || PW == 64 || PW == 128, "panel width");
  static_assert(INSTR % NW == 0 || INSTR < NW, "loads split evenly");
  static_assert(BASES == 1 || (PANEL_INSTR % NW == 0) || KC || PW == 64, "panels");

  uint32_t off[PER_WAVE];
  uint64_t base[BASES];
  int64_t left[BASES];   // bytes from base to the operand's end
  int64_t step;          // bytes per stage

  __device__ __forceinline__ static int swz_kc(int r) { return (r >> 1) & 7; }
  __device__ __forceinline__ static int swz_mc(int k) {
    return PW == 128 ? (k & 3) | (((k >> 3) & 1) << 2) : ((k >> 1) & 1) | (((k >> 3) & 1) << 1);
  }

  // Tile rows (columns) r0 + p * panel_stride .. of panel p; n valid in all.
  __device__ __forceinline__ void setup(int64_t ld, int64_t r0, int64_t n, bool dual) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    step = KC ? BK * 2 : (int64_t)BK * ld * 2;
#pragma unroll
    for (int t = 0; t < PER_WAVE; ++t) {
      const int q = wave + NW * t;
      if constexpr (KC) {
        const int r = q * 8 + (lane >> 3);
        const int c = (lane & 7) ^ swz_kc(r);
        const int rr = dual ? r % PW : r;
        off[t] = r0 + rr < n ? (uint32_t)(rr * ld * 2 + c * 16) : kOutOfRange;
      } else {
        constexpr int CH = PW / 8;  // chunks per K row
        const int kr = (q % PANEL_INSTR) * (64 / CH) + lane / CH;
        const int pc = lane % CH;
        const int c = (((pc >> 1) ^ swz_mc(kr)) << 1) | (pc & 1);
        const int col = (dual ? 0 : q / PANEL_INSTR * PW) + c * 8;
        off[t] = r0 + col < n ? (uint32_t)(kr * ld * 2 + col * 2) : kOutOfRange;
      }
    }
  }
  // Base `b` of an operand at p, of n rows (columns), K values, at K value k0.
  __device__ __forceinline__ void seek(int b, const void* p, int64_t ld, int64_t r0, int64_t n,
                                       int64_t K, int64_t k0) {
    const int64_t at = KC ? (r0 * ld + k0) * 2 : (k0 * ld + r0) * 2;
    base[b] = reinterpret_cast<uint64_t>(p) + (uint64_t)at;
    left[b] = (KC ? n * ld : K * ld) * 2 - at;
  }
  __device__ __forceinline__ void advance() {
#pragma unroll
    for (int b = 0; b < BASES; ++b) {
      base[b] += (uint64_t)step;
      left[b] -= step;
    }
  }
  // This wave's load t of the stage; kleft: K values from the stage's first on.
  __device__ __forceinline__ void issue(char* lds, int t, int kleft) const {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = wave + NW * t;
    if (INSTR % NW != 0 && q >= INSTR) return;
    int b = 0;
    if constexpr (BASES == 2) b = q / PANEL_INSTR;
    const i32x4_t srd = b == 0 ? window_srd(base[0], left[0])
                               : window_srd(base[BASES - 1], left[BASES - 1]);
    uint32_t o = off[t];
    if constexpr (KC) {
      const int c = (lane & 7) ^ swz_kc(q * 8 + (lane >> 3));
      o = c * 8 < kleft ? o : kOutOfRange;
    }
    dma16<true>(srd, o, lds + q * 1024);
  }
  // Fragment of the 16 rows (columns) at r (a multiple of 16) for K step ks of 32.
  __device__ __forceinline__ static uint4 frag(const char* lds, int r, int ks) {
    const int lane = threadIdx.x & 63;
    const int lr = lane & 15, lg = lane >> 4;
    if constexpr (KC) {
      const int row = r + lr;
      return *reinterpret_cast<const uint4*>(lds + row * 128 +
                                             (((ks * 4 + lg) ^ swz_kc(row)) << 4));
    } else {
      i16x4_t h[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int k = ks * 32 + 8 * lg + 4 * hh + (lr >> 2);
        const int n = r + 4 * (lr & 3);
        const int c = (n % PW) >> 3;
        const int pc = (((c >> 1) ^ swz_mc(k)) << 1) | (c & 1);
        const char* p = lds + n / PW * (PW * BK * 2) + k * (PW * 2) + (pc << 4) + ((n & 4) << 1);
        h[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) i16x4_t*)(p));
      }
      return __builtin_bit_cast(uint4, h);
    }
  }
};

// BM x BN tile by WM x WN waves, NP column panels of BN / NP, DUAL: each panel
// has a B and a C of its own. A wave covers the same BN / NP / WN columns of each
// panel. NST: LDS slots.
template <int BM_, int BN_, int NP_, bool DUAL_, bool AKC, bool BKC, int WM, int WN, int NST_>
struct BfCore {
  using elem = bf16_t;
  static constexpr int BM = BM_, BN = BN_, NP = NP_, BK = 64, NST = NST_;
  static constexpr bool DUAL = DUAL_;
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int PWB = BN / NP;
  static constexpr int PWA = AKC ? BM : (BM < 128 ? BM : 128);
  using OpA = BfOperand<AKC, BM, PWA, 1, NW>;
  using OpB = BfOperand<BKC, BN, PWB, DUAL ? 2 : 1, NW>;
  static constexpr int MI = BM / WM / 16;
  static constexpr int NIP = PWB / WN / 16;  // 16-column blocks per wave and panel
  static constexpr int NI = NP * NIP;
  static constexpr int STAGE = OpA::BYTES + OpB::BYTES;
  static constexpr int LDS_BYTES = NST * STAGE;
  // loads every wave issues per stage, at least
  static constexpr int MIN_PW = OpA::INSTR / NW + OpB::INSTR / NW;
  static constexpr int PIECES = OpA::PER_WAVE + OpB::PER_WAVE;
  static_assert(MI >= 1 && NIP >= 1, "tile too small for the waves");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
  static_assert((NST - 1) * PIECES < 64, "vmcnt range");

  f32x4_t acc[MI][NI];
  OpA a;
  OpB b;
  int kleft;      // K values of the current pair from the next stage to issue on
  int pair;

  __device__ __forceinline__ void seek(const GemmArgs& g, int64_t m0, int64_t n0, int64_t k0) {
    a.seek(0, g.A[pair], g.lda, m0, g.M, g.K[pair], k0);
    b.seek(0, g.B[pair][0], g.ldb, n0, g.N, g.K[pair], k0);
    if constexpr (DUAL) b.seek(1, g.B[pair][1], g.ldb, n0, g.N, g.K[pair], k0);
    kleft = (int)(g.K[pair] - k0);
  }
  __device__ __forceinline__ void issue_piece(char* slot, int i) const {
    if (i < OpA::PER_WAVE)
      a.issue(slot, i, kleft);
    else
      b.issue(slot + OpA::BYTES, i - OpA::PER_WAVE, kleft);
  }
  // To the next stage to issue (past the last one: loads give zeros).
  __device__ __forceinline__ void next_stage(const GemmArgs& g, int64_t m0, int64_t n0) {
    kleft -= BK;
    if (kleft <= 0 && pair + 1 < g.pairs) {
      ++pair;
      seek(g, m0, n0, 0);
    } else {
      a.advance();
      b.advance();
    }
  }

  template <typename Between>
  __device__ __forceinline__ void compute(const char* slot, Between between) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm0 = wave / WN * (BM / WM);
    const int wn0 = wave % WN * (PWB / WN);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      uint4 fb[NI], fa[MI];
#pragma unroll
      for (int j = 0; j < NI; ++j)
        fb[j] = OpB::frag(slot + OpA::BYTES, j / NIP * PWB + wn0 + j % NIP * 16, ks);
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[i] = OpA::frag(slot, wm0 + i * 16, ks);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_t, fb[j]), __builtin_bit_cast(bf16x8_t, fa[i]),
              acc[i][j], 0, 0, 0);
        between(ks * MI + i);
      }
    }
  }

  // K stages [s0, s0 + ns) of the tile at (m0, n0).
  __device__ __forceinline__ void run(const GemmArgs& g, char* lds, int64_t m0, int64_t n0,
                                      int s0, int ns) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    a.setup(g.lda, m0, g.M, false);
    b.setup(g.ldb, n0, g.N, DUAL);
    const int first = (int)((g.K[0] + BK - 1) / BK);  // stages of pair 0
    pair = s0 < first ? 0 : 1;
    seek(g, m0, n0, (int64_t)(s0 - (pair ? first : 0)) * BK);
    // issue stages behind the last one as zeros: the window ends there
    int to_issue = ns;
    auto finish = [&] {
      next_stage(g, m0, n0);
      if (--to_issue <= 0) {
        kleft = 0;
        pair = 1 << 20;
        a.left[0] = b.left[0] = 0;
        if constexpr (DUAL) b.left[1] = 0;
      }
    };
#pragma unroll
    for (int s = 0; s + 1 < NST; ++s) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) issue_piece(lds + s * STAGE, i);
      finish();
    }
    int slot = 0, slot_next = NST - 1;
    for (int kt = 0; kt < ns; ++kt) {
      wait_vmcnt<(NST - 2) * MIN_PW>();
      __syncthreads();
      char* nxt = lds + slot_next * STAGE;
      compute(lds + slot * STAGE, [&](int i) {
        if (i < PIECES) issue_piece(nxt, i);
      });
#pragma unroll
      for (int i = 2 * MI; i < PIECES; ++i) issue_piece(nxt, i);
      finish();
      slot = slot + 1 == NST ? 0 : slot + 1;
      slot_next = slot_next + 1 == NST ? 0 : slot_next + 1;
    }
    wait_vmcnt<0>();
  }

  // f(row, column, values of panel 0 .. of 4 consecutive columns): DUAL: one call
  // with both panels' values of the same columns; else v1 is unused.
  template <typename F>
  __device__ __forceinline__ void for_each4(F f) const {
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int row = wave / WN * (BM / WM) + (lane & 15);
    const int col = wave % WN * (PWB / WN) + (lane >> 4) * 4;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if constexpr (DUAL) {
#pragma unroll
        for (int j = 0; j < NIP; ++j)
          f(row + i * 16, col + j * 16, acc[i][j], acc[i][NIP + j]);
      } else {
#pragma unroll
        for (int j = 0; j < NI; ++j)
          f(row + i * 16, j / NIP * PWB + col + j % NIP * 16, acc[i][j], acc[i][j]);
      }
    }
  }
};

// fp32: 4 waves (2 x 2), K stages of 16 through registers into two LDS slots of
// [16][rows + 4] floats per operand.
template <int BM_, int BN_, int NP_, bool DUAL_, bool AKC, bool BKC>
struct F32Core {
  using elem = float;
  static constexpr int BM = BM_, BN = BN_, NP = NP_, BK = 16;
  static constexpr bool DUAL = DUAL_;
  static constexpr int WM = 2, WN = 2, NW = 4, THREADS = 256;
  static constexpr int PWB = BN / NP;
  static constexpr int MI = BM / WM / 16, NIP = PWB / WN / 16, NI = NP * NIP;
  static constexpr int PA = BM + 4, PB = BN + 4;
  static constexpr int STAGE = BK * (PA + PB) * 4;
  static constexpr int LDS_BYTES = 2 * STAGE;
  static constexpr int LA = BM * BK / 4 / THREADS, LB = BN * BK / 4 / THREADS;
  static_assert(LA >= 1 && LB >= 1 && MI >= 1 && NIP >= 1, "tile too small");

  f32x4_t acc[MI][NI];
  f32x4_t ra[LA], rb[LB];
  int pair;
  int64_t k;  // of the next stage to load, within the pair

  template <bool KC, int R>
  __device__ __forceinline__ static f32x4_t load(const float* p, int64_t ld, int64_t r0,
                                                 int64_t n, int64_t K, int64_t k0, int idx) {
    f32x4_t z = {0.f, 0.f, 0.f, 0.f};
    if constexpr (KC) {
      const int64_t r = r0 + idx / 4, kk = k0 + idx % 4 * 4;
      return r < n && kk < K ? load4(p + r * ld + kk) : z;
    } else {
      const int64_t kk = k0 + idx / (R / 4), r = r0 + idx % (R / 4) * 4;
      return r < n && kk < K ? load4(p + kk * ld + r) : z;
    }
  }
  template <bool KC, int R, int P>
  __device__ __forceinline__ static void put(float* lds, int idx, f32x4_t v) {
    if constexpr (KC) {
#pragma unroll
      for (int e = 0; e < 4; ++e) lds[(idx % 4 * 4 + e) * P + idx / 4] = v[e];
    } else {
      store4(lds + idx / (R / 4) * P + idx % (R / 4) * 4, v);
    }
  }
  __device__ __forceinline__ void fetch(const GemmArgs& g, int64_t m0, int64_t n0) {
    const float* A = (const float*)g.A[pair];
#pragma unroll
    for (int t = 0; t < LA; ++t)
      ra[t] = load<AKC, BM>(A, g.lda, m0, g.M, g.K[pair], k, threadIdx.x + t * THREADS);
    // an index of B runs over panels of PWB rows (columns)
#pragma unroll
    for (int t = 0; t < LB; ++t) {
      const int idx = threadIdx.x + t * THREADS;
      constexpr int PER = PWB * BK / 4;
      const int p = idx / PER;
      rb[t] = load<BKC, PWB>((const float*)(DUAL && p ? g.B[pair][1] : g.B[pair][0]), g.ldb,
                             n0 + (DUAL ? 0 : p * PWB), g.N, g.K[pair], k, idx % PER);
    }
    k += BK;
    if (k >= g.K[pair] && pair + 1 < g.pairs) {
      ++pair;
      k = 0;
    }
  }
  __device__ __forceinline__ void stage(float* lds) const {
#pragma unroll
    for (int t = 0; t < LA; ++t) put<AKC, BM, PA>(lds, threadIdx.x + t * THREADS, ra[t]);
#pragma unroll
    for (int t = 0; t < LB; ++t) {
      const int idx = threadIdx.x + t * THREADS;
      constexpr int PER = PWB * BK / 4;
      put<BKC, PWB, PB>(lds + BK * PA + idx / PER * PWB, idx % PER, rb[t]);
    }
  }
  __device__ __forceinline__ void compute(const float* lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lr = lane & 15, lg = lane >> 4;
    const int wm0 = wave / WN * (BM / WM), wn0 = wave % WN * (PWB / WN);
#pragma unroll
    for (int ks = 0; ks < BK / 4; ++ks) {
      float fa[MI], fb[NI];
      const int kk = ks * 4 + lg;
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[i] = lds[kk * PA + wm0 + i * 16 + lr];
#pragma unroll
      for (int j = 0; j < NI; ++j)
        fb[j] = lds[BK * PA + kk * PB + j / NIP * PWB + wn0 + j % NIP * 16 + lr];
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  }
  __device__ __forceinline__ void run(const GemmArgs& g, char* lds, int64_t m0, int64_t n0,
                                      int s0, int ns) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int first = (int)((g.K[0] + BK - 1) / BK);
    pair = s0 < first ? 0 : 1;
    k = (int64_t)(s0 - (pair ? first : 0)) * BK;
    fetch(g, m0, n0);
    for (int kt = 0; kt < ns; ++kt) {
      float* slot = reinterpret_cast<float*>(lds + (kt & 1) * STAGE);
      stage(slot);
      if (kt + 1 < ns) fetch(g, m0, n0);
      __syncthreads();
      compute(slot);
    }
  }
  template <typename F>
  __device__ __forceinline__ void for_each4(F f) const {
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int row = wave / WN * (BM / WM) + (lane & 15);
    const int col = wave % WN * (PWB / WN) + (lane >> 4) * 4;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if constexpr (DUAL) {
#pragma unroll
        for (int j = 0; j < NIP; ++j)
          f(row + i * 16, col + j * 16, acc[i][j], acc[i][NIP + j]);
      } else {
#pragma unroll
        for (int j = 0; j < NI; ++j)
          f(row + i * 16, j / NIP * PWB + col + j % NIP * 16, acc[i][j], acc[i][j]);
      }
    }
  }
};

// Tile of workgroup id: a contiguous range of tiles per XCD (workgroups go to
// the 8 XCDs in turn), in groups of 8 row tiles by all column tiles, so that a
// XCD's L2 holds what its workgroups share.
__device__ __forceinline__ void tile_of(int id, int total, int tiles_m, int tiles_n, int* split,
                                        int* tm, int* tn) {
  const int per = total / kXcds, rem = total % kXcds;
  const int x = id % kXcds, l = id / kXcds;
  int t = x * per + (x < rem ? x : rem) + l;
  const int mn = tiles_m * tiles_n;
  *split = t / mn;
  t %= mn;
  constexpr int GM = 8;
  const int in_group = GM * tiles_n;
  const int g = t / in_group, m0 = g * GM;
  const int gm = tiles_m - m0 < GM ? tiles_m - m0 : GM;
  t -= g * in_group;
  *tm = m0 + t % gm;
  *tn = t / gm;
}

// The product with epilogue EP: ep(row, column, v0, v1) for 4 columns each; with
// splits > 1 the sums go to g.part instead.
template <typename Core, typename EP>
__global__ __launch_bounds__(Core::THREADS) void gemm_kernel(GemmArgs g, EP ep) {
  __shared__ __align__(16) char gemm_lds[Core::LDS_BYTES];
  int split, tm, tn;
  tile_of(blockIdx.x, gridDim.x, g.tiles_m, g.tiles_n, &split, &tm, &tn);
  const int64_t m0 = (int64_t)tm * Core::BM;
  const int64_t n0 = (int64_t)tn * (Core::DUAL ? Core::PWB : Core::BN);
  const int s0 = split * g.split_stages;
  const int ns = g.stages - s0 < g.split_stages ? g.stages - s0 : g.split_stages;
  Core core;
  core.run(g, gemm_lds, m0, n0, s0, ns);
  if (g.splits > 1) {
    float* p0 = g.part + (int64_t)split * (Core::DUAL ? 2 : 1) * g.M * g.N;
    core.for_each4([&](int r, int c, f32x4_t v0, f32x4_t v1) {
      const int64_t m = m0 + r, n = n0 + c;
      if (m >= g.M || n >= g.N) return;
      store4(p0 + m * g.N + n, v0);
      if constexpr (Core::DUAL) store4(p0 + (g.M + m) * g.N + n, v1);
    });
  } else {
    core.for_each4([&](int r, int c, f32x4_t v0, f32x4_t v1) {
      const int64_t m = m0 + r, n = n0 + c;
      if (m < g.M && n < g.N) ep(m, n, v0, v1);
    });
  }
}

// Adds the splits' sums in split order and applies the epilogue.
template <bool DUAL, typename EP>
__global__ __launch_bounds__(256) void gemm_join_kernel(GemmArgs g, EP ep) {
  const int64_t per = (g.N + 3) / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < g.M * per;
       i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per, n = i % per * 4;
    f32x4_t v[2];
#pragma unroll
    for (int p = 0; p < (DUAL ? 2 : 1); ++p) {
      const float* q = g.part + ((int64_t)p * g.M + m) * g.N + n;
      const int64_t stride = (DUAL ? 2 : 1) * g.M * g.N;
      v[p] = load4(q);
      for (int s = 1; s < g.splits; ++s) {
        const f32x4_t w = load4(q + s * stride);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[p][r] += w[r];
      }
    }
    ep(m, n, v[0], DUAL ? v[1] : v[0]);
  }
}

}  // namespace moe
