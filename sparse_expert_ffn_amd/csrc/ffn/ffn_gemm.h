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
// K stages of 128 bytes (64 bf16, 32 fp32) go from global memory straight into a
// ring of LDS slots (16 bytes per lane). KC operands lie there as rows of 128
// bytes and are read 16 bytes per lane, MC operands as K rows of a panel of up to
// 256 bytes and are read transposed (bf16: ds_read_b64_tr_b16; fp32: 4 bytes per
// lane), in the chunk orders that the MoE layer's tile core measured free of
// bank conflicts (fp32 MC: 64-byte units ordered by the lane group).
//   bf16: v_mfma_f32_16x16x32_bf16, a lane's 16 bytes are 8 K values of a row;
//   fp32: four v_mfma_f32_16x16x4_f32, a lane's 16 bytes are 4 K values, one per
//         MFMA: any order of K serves that is the same for both operands.
// The MFMA takes B's fragment as its first operand, so a lane ends up with 4
// consecutive columns of one row and loads and stores them as one access.
//
// The operands are addressed from a base that moves along K with the stages
// (scalar arithmetic), so an array may exceed the 4 GiB of a buffer's range;
// out-of-range rows, columns and K values read as zeros.
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

// One operand (R tile rows or columns in panels of PW, with one or two bases) in LDS.
//
// KC: row r at r * 128 bytes, its 16-byte chunk c in slot c ^ (r / 2) % 8.
// MC: panel by panel, K row k of a panel at k * ROWB bytes; its units (32 bytes in
// bf16, 64 in fp32: 16 columns) u in slot u ^ swz_mc(k).
template <typename T, bool KC, int R, int PW, int BASES, int NW>
struct Operand {
  static constexpr int ES = sizeof(T);
  static constexpr int BK = 128 / ES;          // K values per stage
  static constexpr int BYTES = R * 128;        // per stage
  static constexpr int INSTR = BYTES / 1024;
  static constexpr int PER_WAVE = (INSTR + NW - 1) / NW;
  static constexpr int PANEL = PW * 128;       // bytes per panel and stage
  static constexpr int PANEL_INSTR = PANEL / 1024;
  static constexpr int ROWB = PW * ES;         // MC: bytes per K row of a panel
  static constexpr int CPU = ES;               // MC: 16-byte chunks per 16-column unit
  static_assert(KC || ROWB == 128 || ROWB == 256, "panel width");
  static_assert(INSTR % NW == 0 || INSTR < NW, "loads split evenly");

  int wave;
  uint32_t off[PER_WAVE];
  int chunk_k;           // KC: this lane's K value within a stage, for all its loads
  uint64_t base[BASES];
  int64_t left[BASES];   // bytes from base to the operand's end
  int64_t step;          // bytes per stage
  i32x4_t srd[BASES];    // of the next stage to load
  uint32_t rd[2];        // LDS offset of this lane's fragment reads (KC: per K step)

  __device__ __forceinline__ static int swz_kc(int r) { return (r >> 1) & 7; }
  __device__ __forceinline__ static int swz_mc(int k) {
    if (ES == 4) return (k >> 2) & (ROWB == 256 ? 3 : 1);
    return ROWB == 256 ? (k & 3) | (((k >> 3) & 1) << 2) : ((k >> 1) & 1) | (((k >> 3) & 1) << 1);
  }

  // Tile rows (columns) from r0 on, n valid in all; with two bases each panel
  // covers the same ones. w0: the first row (column) of each panel that this
  // wave's fragments cover.
  __device__ __forceinline__ void setup(int wave_, int64_t ld, int64_t r0, int64_t n, int w0) {
    const int lane = threadIdx.x & 63;
    wave = wave_;
    step = KC ? 128 : (int64_t)BK * ld * ES;
#pragma unroll
    for (int t = 0; t < PER_WAVE; ++t) {
      const int q = wave + NW * t;
      if constexpr (KC) {
        const int r = q * 8 + (lane >> 3);
        // the chunk is the same for every t (rows 8 NW apart, or one load only)
        const int c = (lane & 7) ^ swz_kc(r);
        const int rr = BASES == 2 ? r % PW : r;
        chunk_k = c * (16 / ES);
        off[t] = r0 + rr < n ? (uint32_t)(rr * ld * ES + c * 16) : kOutOfRange;
      } else {
        constexpr int CH = ROWB / 16;  // chunks per K row
        const int kr = (q % PANEL_INSTR) * (64 / CH) + lane / CH;
        const int pc = lane % CH;
        const int c = (pc / CPU ^ swz_mc(kr)) * CPU + pc % CPU;
        const int col = (BASES == 2 ? 0 : q / PANEL_INSTR * PW) + c * (16 / ES);
        off[t] = r0 + col < n ? (uint32_t)(kr * ld * ES + col * ES) : kOutOfRange;
      }
    }
    const int lr = lane & 15, lg = lane >> 4;
    if constexpr (KC) {
      rd[0] = (w0 + lr) * 128 + ((lg ^ swz_kc(lr)) << 4);
      rd[1] = (w0 + lr) * 128 + (((4 + lg) ^ swz_kc(lr)) << 4);
    } else if constexpr (ES == 2) {
      // K row 8 lg + lr / 4 of a step (+ 4 for the second read), 4 columns at
      // 4 (lr % 4) of a 16-column block: block j of the wave at rd ^ (j * 32)
      const int k = 8 * lg + (lr >> 2);
      rd[0] = w0 / PW * PANEL + k * ROWB + ((w0 % PW / 16 ^ swz_mc(k)) << 5) + ((lr & 3) << 3);
    } else {
      // K rows 4 lg .. + 3 of a step, column lr of block j at rd ^ (j * 64)
      rd[0] = w0 / PW * PANEL + 4 * lg * ROWB + ((w0 % PW / 16 ^ swz_mc(4 * lg)) << 6) + lr * 4;
    }
  }
  // Base `b` of an operand at p, of n rows (columns), K values, at K value k0.
  __device__ __forceinline__ void seek(int b, const void* p, int64_t ld, int64_t r0, int64_t n,
                                       int64_t K, int64_t k0) {
    const int64_t at = KC ? (r0 * ld + k0) * ES : (k0 * ld + r0) * ES;
    base[b] = reinterpret_cast<uint64_t>(p) + (uint64_t)at;
    left[b] = (KC ? n * ld : K * ld) * ES - at;
    srd[b] = window_srd(base[b], left[b]);
  }
  __device__ __forceinline__ void advance() {
#pragma unroll
    for (int b = 0; b < BASES; ++b) {
      base[b] += (uint64_t)step;
      left[b] -= step;
      srd[b] = window_srd(base[b], left[b]);
    }
  }
  // From here on loads give zeros.
  __device__ __forceinline__ void close() {
#pragma unroll
    for (int b = 0; b < BASES; ++b) {
      left[b] = 0;
      srd[b].z = 0;
    }
  }
  // This wave's load t of the stage; kleft: K values from the stage's first on.
  __device__ __forceinline__ void issue(char* lds, int t, int kleft) const {
    const int q = wave + NW * t;
    if (INSTR % NW != 0 && q >= INSTR) return;
    int b = 0;
    if constexpr (BASES == 2) b = PANEL_INSTR % NW == 0 ? NW * t / PANEL_INSTR : q / PANEL_INSTR;
    const i32x4_t r = b == 0 ? srd[0] : srd[BASES - 1];
    uint32_t o = off[t];
    if constexpr (KC) o = chunk_k < kleft ? o : kOutOfRange;
    dma16(r, o, lds + q * 1024);
  }
  // Fragment of the wave's 16-row (column) block j of panel p for K step ks. MC: a
  // wave's blocks lie in one panel and start at a multiple of their number, so
  // that the exclusive or adds j.
  __device__ __forceinline__ uint4 frag(const char* lds, int p, int j, int ks) const {
    if constexpr (KC) {
      return *reinterpret_cast<const uint4*>(lds + rd[ks] + (p * PW + j * 16) * 128);
    } else if constexpr (ES == 2) {
      i16x4_t h[2];
      const char* q = lds + (rd[0] ^ (uint32_t)(j << 5)) + p * PANEL + ks * 32 * ROWB;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        h[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) i16x4_t*)(q + 4 * hh * ROWB));
      return __builtin_bit_cast(uint4, h);
    } else {
      const char* q = lds + (rd[0] ^ (uint32_t)(j << 6)) + p * PANEL + ks * 16 * ROWB;
      f32x4_t v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const float*>(q + e * ROWB);
      return __builtin_bit_cast(uint4, v);
    }
  }
};

// BM x BN tile by WM x WN waves, NP column panels of BN / NP, DUAL: each panel
// has a B and a C of its own. A wave covers the same BN / NP / WN columns of each
// panel. NST: LDS slots.
template <typename T, int BM_, int BN_, int NP_, bool DUAL_, bool AKC, bool BKC, int WM, int WN,
          int NST_>
struct TileCore {
  static constexpr int BM = BM_, BN = BN_, NP = NP_, BK = 128 / (int)sizeof(T), NST = NST_;
  static constexpr bool DUAL = DUAL_;
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int PWB = BN / NP;
  static constexpr int PMAX = 256 / (int)sizeof(T);
  static constexpr int PWA = AKC ? BM : (BM < PMAX ? BM : PMAX);
  using OpA = Operand<T, AKC, BM, PWA, 1, NW>;
  using OpB = Operand<T, BKC, BN, PWB, DUAL ? 2 : 1, NW>;
  static constexpr int MI = BM / WM / 16;
  static constexpr int NIP = PWB / WN / 16;  // 16-column blocks per wave and panel
  static constexpr int NI = NP * NIP;
  static constexpr int STAGE = OpA::BYTES + OpB::BYTES;
  static constexpr int LDS_BYTES = NST * STAGE;
  // loads every wave issues per stage, at least
  static constexpr int MIN_PW = OpA::INSTR / NW + OpB::INSTR / NW;
  static constexpr int PIECES = OpA::PER_WAVE + OpB::PER_WAVE;
  static_assert(MI >= 1 && NIP >= 1, "tile too small for the waves");
  static_assert(AKC || (PWA % (BM / WM) == 0 && (MI & (MI - 1)) == 0), "A blocks in one panel");
  static_assert(BKC || (NIP & (NIP - 1)) == 0, "B blocks");
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

  uint4 fa[2][MI], fb[2][NI];  // fragments of two K steps of 32 in turn

  // Fragment n of K step ks (B's column blocks, then A's row blocks) into set `to`.
  __device__ __forceinline__ void read_frag(const char* slot, int ks, int to, int n) {
    if (n < NI)
      fb[to][n] = b.frag(slot + OpA::BYTES, n / NIP, n % NIP, ks);
    else
      fa[to][n - NI] = a.frag(slot, 0, n - NI, ks);
  }

  // The MFMAs of the K step in set `cur`, row block by row block; between them go
  // the LDS reads of the next K step (from rd, into the other set; all of them out
  // two row blocks before the end, so that they have landed when it starts) and,
  // with `issue`, the global loads of a later stage into wr.
  __device__ __forceinline__ void phase(int cur, const char* rd, int rd_ks, char* wr,
                                        bool issue) {
    constexpr int FRAGS = NI + MI;
    constexpr int ROWS = MI > 2 ? MI - 1 : MI;  // row blocks that carry reads
    constexpr int IROWS = MI < 4 ? MI : 4;      // and global loads
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int e = 0; e < (sizeof(T) == 4 ? 4 : 1); ++e)
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          if constexpr (sizeof(T) == 4)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                __builtin_bit_cast(f32x4_t, fb[cur][j])[e],
                __builtin_bit_cast(f32x4_t, fa[cur][i])[e], acc[i][j], 0, 0, 0);
          else
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8_t, fb[cur][j]),
                __builtin_bit_cast(bf16x8_t, fa[cur][i]), acc[i][j], 0, 0, 0);
        }
      if (i < ROWS) {
#pragma unroll
        for (int n = i * FRAGS / ROWS; n < (i + 1) * FRAGS / ROWS; ++n)
          read_frag(rd, rd_ks, cur ^ 1, n);
      }
      if (issue)
#pragma unroll
        for (int n = i * PIECES / IROWS; n < (i + 1) * PIECES / IROWS && n < PIECES; ++n)
          issue_piece(wr, n);
      __builtin_amdgcn_sched_barrier(0);  // the order of the row blocks stands
    }
  }

  // K stages [s0, s0 + ns) of the tile at (m0, n0). All NST slots are in flight.
  // Stage kt: its first K step's fragments were read during the previous phase;
  // phase 0 reads the second K step's; then every wave's reads of the slot are done
  // and stage kt + 1 has landed (one wait and barrier), and phase 1 reads stage
  // kt + 1's first fragments and loads stage kt + NST into stage kt's slot.
  __device__ __forceinline__ void run(const GemmArgs& g, char* lds, int64_t m0, int64_t n0,
                                      int s0, int ns) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    a.setup(wave, g.lda, m0, g.M, wave / WN * (BM / WM));
    b.setup(wave, g.ldb, n0, g.N, wave % WN * (PWB / WN));
    const int first = (int)((g.K[0] + BK - 1) / BK);  // stages of pair 0
    pair = s0 < first ? 0 : 1;
    seek(g, m0, n0, (int64_t)(s0 - (pair ? first : 0)) * BK);
    int to_issue = ns;
    auto finish = [&] {
      next_stage(g, m0, n0);
      if (--to_issue <= 0) {  // stages past the last one load nothing (zeros)
        kleft = 0;
        pair = 2;
        a.close();
        b.close();
      }
    };
#pragma unroll
    for (int s = 0; s < NST; ++s) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) issue_piece(lds + s * STAGE, i);
      finish();
    }
    wait_vmcnt<(NST - 1) * MIN_PW>();
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NI + MI; ++n) read_frag(lds, 0, 0, n);
    int slot = 0;
    for (int kt = 0; kt < ns; ++kt) {
      char* cur = lds + slot * STAGE;
      slot = slot + 1 == NST ? 0 : slot + 1;
      phase(0, cur, 1, nullptr, false);
      wait_vmcnt<(NST - 2) * MIN_PW>();
      __syncthreads();
      __builtin_amdgcn_sched_barrier(0);
      phase(1, lds + slot * STAGE, 0, cur, true);
      finish();
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_vmcnt<0>();
  }

  // Consecutive columns of one row that a lane handles in the epilogue: the MFMA
  // leaves 4; in bf16 two neighbouring blocks swap lane rows to make it 8, one
  // 16-byte access.
  static constexpr int W = sizeof(T) == 2 && NIP % 2 == 0 ? 8 : 4;
  static constexpr int BPG = W / 4;            // blocks per group of W columns
  static constexpr int GROUPS = (DUAL ? NIP : NI) / BPG;  // per row block

  // Tile row and (panel's) column of group q of row block i.
  __device__ __forceinline__ int group_row(int i) const {
    return (threadIdx.x >> 6) / WN * (BM / WM) + i * 16 + (threadIdx.x & 15);
  }
  __device__ __forceinline__ int group_col(int q) const {
    const int lg = (threadIdx.x & 63) >> 4;
    const int j = q * BPG;
    const int c = j / NIP * PWB + (threadIdx.x >> 6) % WN * (PWB / WN) + j % NIP * 16;
    return W == 8 ? c + (lg & 1) * 16 + (lg >> 1) * 8 : c + lg * 4;
  }
  // Its values (of panel 1 with p = 1 in a DUAL tile).
  __device__ __forceinline__ void group_values(int i, int q, int p, float (&v)[W]) {
    const int j = p * NIP + q * BPG;
    if constexpr (W == 8) {
      // lane rows 0..3 hold columns 0, 4, 8, 12 and up of both blocks; after odd rows of
      // the first swapped places with even rows of the second, row 0 holds the first
      // block's columns 0..7, row 1 the second's, row 2 the first's 8..15, row 3 the
      // second's
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[i][j][r]),
                                                        __float_as_uint(acc[i][j + 1][r]),
                                                        false, false);
        v[r] = __uint_as_float(w[0]);
        v[4 + r] = __uint_as_float(w[1]);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = acc[i][j][r];
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

// The product with epilogue EP: ep(row, column, v0, v1, pre) for W columns each (v1:
// the second panel's values in a DUAL tile, else v0 again; pre: what EP::pre read
// for them, one row block ahead so that the loads do not wait for each other); with
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
  constexpr int W = Core::W, Q = Core::GROUPS;
  using Pre = typename EP::template Pre<W>;
  float* p0 = g.part + (int64_t)split * (Core::DUAL ? 2 : 1) * g.M * g.N;
  const bool direct = g.splits == 1;
  Pre pre[2][Q];
  auto fetch = [&](int i) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int64_t m = m0 + core.group_row(i), n = n0 + core.group_col(q);
      if (direct && m < g.M && n < g.N) ep.pre(m, n, pre[i & 1][q]);
    }
  };
  fetch(0);
#pragma unroll
  for (int i = 0; i < Core::MI; ++i) {
    if (i + 1 < Core::MI) fetch(i + 1);
    __builtin_amdgcn_sched_barrier(0);  // one row block's values at a time
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int64_t m = m0 + core.group_row(i), n = n0 + core.group_col(q);
      float v0[W], v1[W];
      core.group_values(i, q, 0, v0);
      if constexpr (Core::DUAL) core.group_values(i, q, 1, v1);
      if (m >= g.M || n >= g.N) continue;
      if (direct) {
        if constexpr (Core::DUAL)
          ep(m, n, v0, v1, pre[i & 1][q]);
        else
          ep(m, n, v0, v0, pre[i & 1][q]);
      } else {
        store_n(p0 + m * g.N + n, v0);
        if constexpr (Core::DUAL) store_n(p0 + (g.M + m) * g.N + n, v1);
      }
    }
  }
}

// Adds the splits' sums in split order and applies the epilogue.
template <bool DUAL, typename EP>
__global__ __launch_bounds__(256) void gemm_join_kernel(GemmArgs g, EP ep) {
  const int64_t per = (g.N + 3) / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < g.M * per;
       i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per, n = i % per * 4;
    typename EP::template Pre<4> pre;
    ep.pre(m, n, pre);
    float v[2][4] = {};
#pragma unroll
    for (int p = 0; p < (DUAL ? 2 : 1); ++p) {
      const float* q = g.part + ((int64_t)p * g.M + m) * g.N + n;
      const int64_t stride = (DUAL ? 2 : 1) * g.M * g.N;
      // 8 splits' loads in flight; the sums are added in split order
      for (int s = 0; s < g.splits; s += 8) {
        f32x4_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = s + e < g.splits ? load4(q + (s + e) * stride) : f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[p][r] += w[e][r];
      }
    }
    ep(m, n, v[0], v[DUAL ? 1 : 0], pre);
  }
}

}  // namespace moe
