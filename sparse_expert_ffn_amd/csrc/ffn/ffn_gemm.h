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
//
// What bounds it (256 x 256 bf16 tile, 16384 x 2048 x 4096): a K stage takes 1.56 us
// where its MFMAs alone take 1.03 at the 2.0 GHz that this load runs at. With the LDS
// reads it is 1.13 us; the rest is the global loads, whose last ones have one stage's
// time at most to land: 160 KB of LDS hold two and a half stages. Issued later in the
// stage they cost 15% more, in one burst after the barrier 2%. Four waves of 128 x
// 128 (a third fewer LDS reads) spilled and were slower, as were K stages of half the
// length with twice the slots (twice the barriers); 32 x 32 x 16 MFMAs run 12% slower
// than 16 x 16 x 32 on their own (1.84 against 2.11 PFLOP/s: the clock gives way).
// Rates: dX 1.30 PFLOP/s, weight gradients 1.20, forward 1.13 with all outputs; fp32
// 124 TFLOP/s (128 x 128) of the 133 that the library reaches.
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
template <typename T, bool KC, int R, int PW, int BASES, int NW, bool ONCE>
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
  static_assert(!KC || BASES == 1, "two bases: a DUAL product's B, K outermost");
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
        chunk_k = c * (16 / ES);
        off[t] = r0 + r < n ? (uint32_t)(r * ld * ES + c * 16) : kOutOfRange;
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
    dma16<false, ONCE>(r, o, lds + q * 1024);
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
// ONCE: B is read once in all (one row of tiles): its loads carry the non-temporal hint
// (64 tokens of 7168 x 2048, cold caches: up and gate 28.6 -> 16.8 us, down 15.7 ->
// 13.1 us; one token 25.8 -> 14.3 and 14.5 -> 8.9 us).
template <typename T, int BM_, int BN_, int NP_, bool DUAL_, bool AKC, bool BKC, int WM, int WN,
          int NST_, bool ONCE = false>
struct TileCore {
  static constexpr int BM = BM_, BN = BN_, NP = NP_, BK = 128 / (int)sizeof(T), NST = NST_;
  static constexpr bool DUAL = DUAL_;
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int PWB = BN / NP;
  static constexpr int PMAX = 256 / (int)sizeof(T);
  static constexpr int PWA = AKC ? BM : (BM < PMAX ? BM : PMAX);
  using OpA = Operand<T, AKC, BM, PWA, 1, NW, false>;
  using OpB = Operand<T, BKC, BN, PWB, DUAL ? 2 : 1, NW, ONCE>;
  static constexpr int MI = BM / WM / 16;
  static constexpr int NIP = PWB / WN / 16;  // 16-column blocks per wave and panel
  static constexpr int NI = NP * NIP;
  static constexpr int STAGE = OpA::BYTES + OpB::BYTES;
  // loads every wave issues per stage, at least
  static constexpr int MIN_PW = OpA::INSTR / NW + OpB::INSTR / NW;
  static constexpr int PIECES = OpA::PER_WAVE + OpB::PER_WAVE;
  static_assert(MI >= 1 && NIP >= 1, "tile too small for the waves");
  static_assert(AKC || (PWA % (BM / WM) == 0 && (MI & (MI - 1)) == 0), "A blocks in one panel");
  static_assert(BKC || (NIP & (NIP - 1)) == 0, "B blocks");
  static_assert((NST - 1) * PIECES < 64, "vmcnt range");

  f32x4_t acc[MI][NI];
  OpA a;
  OpB b;
  // Where an operand's next stage to load lies: its pair, the pair's K values from
  // that stage on, the stages still to load.
  struct Cursor {
    int pair, kleft, stages;
  };
  Cursor ca, cb;

  __device__ __forceinline__ void seek_a(const GemmArgs& g, int64_t m0, int64_t k0) {
    a.seek(0, g.A[ca.pair], g.lda, m0, g.M, g.K[ca.pair], k0);
    ca.kleft = (int)(g.K[ca.pair] - k0);
  }
  __device__ __forceinline__ void seek_b(const GemmArgs& g, int64_t n0, int64_t k0) {
    b.seek(0, g.B[cb.pair][0], g.ldb, n0, g.N, g.K[cb.pair], k0);
    if constexpr (DUAL) b.seek(1, g.B[cb.pair][1], g.ldb, n0, g.N, g.K[cb.pair], k0);
    cb.kleft = (int)(g.K[cb.pair] - k0);
  }
  // To the next stage to load; past the last one loads give zeros.
  template <typename Op, typename Seek>
  __device__ __forceinline__ static void next(Op& op, Cursor& c, int pairs, Seek seek) {
    c.kleft -= BK;
    if (--c.stages <= 0) {
      c.kleft = 0;
      op.close();
    } else if (c.kleft <= 0 && c.pair + 1 < pairs) {
      ++c.pair;
      seek();
    } else {
      op.advance();
    }
  }
  __device__ __forceinline__ void next_a(const GemmArgs& g, int64_t m0) {
    next(a, ca, g.pairs, [&] { seek_a(g, m0, 0); });
  }
  __device__ __forceinline__ void next_b(const GemmArgs& g, int64_t n0) {
    next(b, cb, g.pairs, [&] { seek_b(g, n0, 0); });
  }

  uint4 fa[2][MI], fb[2][NI];  // fragments of two K steps in turn

  // Fragment n of K step ks (B's column blocks, then A's row blocks) into set `to`.
  __device__ __forceinline__ void read_frag(const char* la, const char* lb, int ks, int to,
                                            int n) {
    if (n < NI)
      fb[to][n] = b.frag(lb, n / NIP, n % NIP, ks);
    else
      fa[to][n - NI] = a.frag(la, 0, n - NI, ks);
  }

  // The MFMAs of the K step in set `cur`, row block by row block; between them go
  // the LDS reads of the next K step (from la and lb, into the other set; all of them
  // out a row block before the end, so that they have landed when it starts) and
  // `loads` global loads of a later stage, issue(n), over the first `rows` row blocks.
  template <typename Issue>
  __device__ __forceinline__ void phase(int cur, const char* la, const char* lb, int ks, int loads,
                                        int rows, Issue issue) {
    constexpr int FRAGS = NI + MI;
    constexpr int ROWS = MI > 1 ? MI - 1 : 1;   // row blocks that carry reads
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
          read_frag(la, lb, ks, cur ^ 1, n);
      }
#pragma unroll
      for (int n = i * loads / rows; n < (i + 1) * loads / rows && n < loads; ++n) issue(n);
      __builtin_amdgcn_sched_barrier(0);  // the order of the row blocks stands
    }
  }

  // K stages [s0, s0 + ns) of the tile at (m0, n0).
  //
  // Stage kt: its first K step's fragments were read during the previous phase;
  // phase 0 reads the second K step's; then every wave's reads of the stage's LDS are
  // done and stage kt + 1 has landed (one wait and barrier), and phase 1 reads stage
  // kt + 1's first fragments.
  //
  // Whole slots: all NST are in flight, phase 1 loads stage kt + NST into stage kt's.
  // HALVES (the 256 x 256 tile, whose LDS holds two stages and a half): A and B have
  // slots of their own, five in turn (A0 B0 A1 B1 A2 B2 ..), phase 0 loads A of stage
  // kt + 2 into the one that B of kt - 1 left and phase 1 B of stage kt + 2 into that of
  // A of kt: half the loads in each phase instead of all of them in one.
  static constexpr bool HALVES = OpA::BYTES == OpB::BYTES && 5 * OpA::BYTES <= 160 * 1024 &&
                                 6 * OpA::BYTES > 160 * 1024;
  static constexpr int LDS_BYTES = HALVES ? 5 * OpA::BYTES : NST * STAGE;
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
  static_assert(!HALVES || (OpA::INSTR % NW == 0 && OpB::INSTR % NW == 0), "even loads");

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
    ca.pair = cb.pair = s0 < first ? 0 : 1;
    ca.stages = cb.stages = ns;
    const int64_t k0 = (int64_t)(s0 - (ca.pair ? first : 0)) * BK;
    seek_a(g, m0, k0);
    seek_b(g, n0, k0);
    auto load_a = [&](char* to, int n) { a.issue(to, n, ca.kleft); };
    auto load_b = [&](char* to, int n) { b.issue(to, n, cb.kleft); };
    constexpr int PA = OpA::PER_WAVE, PB = OpB::PER_WAVE;
    if constexpr (HALVES) {
      constexpr int H = OpA::BYTES;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int n = 0; n < PA; ++n) load_a(lds + 2 * s * H, n);
        next_a(g, m0);
#pragma unroll
        for (int n = 0; n < PB; ++n) load_b(lds + (2 * s + 1) * H, n);
        next_b(g, n0);
      }
      wait_vmcnt<PA + PB>();
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NI + MI; ++n) read_frag(lds, lds + H, 0, 0, n);
      int u = 0;  // slot of A of stage kt
      auto at = [&](int d) { return lds + (u + d >= 5 ? u + d - 5 : u + d) * H; };
      for (int kt = 0; kt < ns; ++kt) {
        char* to_a = at(4);
        phase(0, at(0), at(1), 1, PA, 4, [&](int n) { load_a(to_a, n); });
        next_a(g, m0);
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<PA>();
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        char* to_b = at(0);
        phase(1, at(2), at(3), 0, PB, 4, [&](int n) { load_b(to_b, n); });
        next_b(g, n0);
        u = u + 2 >= 5 ? u - 3 : u + 2;
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      // both operands go through K together: one cursor
      auto load = [&](char* to, int n) {
        if (n < PA)
          a.issue(to, n, ca.kleft);
        else
          b.issue(to + OpA::BYTES, n - PA, ca.kleft);
      };
      auto next_ab = [&] {
        ca.kleft -= BK;
        if (--ca.stages <= 0) {
          ca.kleft = 0;
          a.close();
          b.close();
        } else if (ca.kleft <= 0 && ca.pair + 1 < g.pairs) {
          cb.pair = ++ca.pair;
          seek_a(g, m0, 0);
          seek_b(g, n0, 0);
        } else {
          a.advance();
          b.advance();
        }
      };
#pragma unroll
      for (int s = 0; s < NST; ++s) {
#pragma unroll
        for (int n = 0; n < PA + PB; ++n) load(lds + s * STAGE, n);
        next_ab();
      }
      wait_vmcnt<(NST - 1) * MIN_PW>();
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NI + MI; ++n) read_frag(lds, lds + OpA::BYTES, 0, 0, n);
      int slot = 0;
      for (int kt = 0; kt < ns; ++kt) {
        char* cur = lds + slot * STAGE;
        slot = slot + 1 == NST ? 0 : slot + 1;
        const char* nxt = lds + slot * STAGE;
        phase(0, cur, cur + OpA::BYTES, 1, 0, 1, [](int) {});
        wait_vmcnt<(NST - 2) * MIN_PW>();
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        phase(1, nxt, nxt + OpA::BYTES, 0, PA + PB, MI < 4 ? MI : 4,
              [&](int n) { load(cur, n); });
        next_ab();
        __builtin_amdgcn_sched_barrier(0);
      }
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
    constexpr int P = DUAL ? 2 : 1;
    float v[2][4] = {};
    const float* q = g.part + m * g.N + n;
    const int64_t panel = g.M * g.N;
    // 8 splits' loads in flight; the sums are added in split order
    for (int s = 0; s < g.splits; s += 8) {
      f32x4_t w[8][P];
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int p = 0; p < P; ++p)
          w[e][p] = s + e < g.splits ? load4(q + ((s + e) * P + p) * panel)
                                     : f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[p][r] += w[e][p][r];
    }
    ep(m, n, v[0], v[DUAL ? 1 : 0], pre);
  }
}

}  // namespace moe
