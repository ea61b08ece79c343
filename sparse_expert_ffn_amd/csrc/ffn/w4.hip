// Products with 4-bit weights for decode (include/moe_ffn.h).
//
// Decode is bound by the weights' bytes: a weight is read once and meets at most
// 16 rows. One MFMA (16x16x32, bf16) takes 16 rows, so one row or sixteen cost
// the same and the matrix cores idle next to HBM either way; what matters is
// that the codes stream and that unpacking them stays cheap.
//
// Unpacking: a bf16 with the exponent of 16 has steps of 1/8, so its bits
// 3..6 hold a code exactly: 0x4180 | code << 3 = 16 + code. The packed dword
// (8 codes, rotated left by 3) gives two such values with one rotation and one
// and-or per pair. The MFMA sums X (16 + code); what is too much, 24 X, is
// summed by MFMAs with a constant -24 operand into the accumulator that the
// group's product starts from (once for all columns and matrices of a wave),
// which leaves sum X (code - 8). Products are exact in fp32 (8 x 8 bits), and
// the group's sum is scaled in fp32 by the column's scale, so W is never rounded.
// (0x4300 | code = 128 + code would save a rotation and lose 3 more bits.)
//
// Layout: tiles of 16 columns x 128 rows, 1 KB of codes in the order of the
// MFMA operand (lane l: column l % 16, rows 8 (l / 16) .. + 7 of each 32) and
// the scales behind them, a column's together: a wave streams a column tile as
// contiguous memory, 16 bytes of codes and one access of scales per lane and step.
//
// The loads go through buffer descriptors, so that what lies past the end (a K
// that is no multiple of 128, a step past the last one, a row that is not there)
// reads as zero without a branch: x = 0 and a scale of 0 add nothing. X comes from
// the caches into registers with the weights, DEPTH steps ahead. (Staged in LDS
// first, the wait for its rows at the start cost more than its loads: one row of
// 7168 x 2048 8.4 -> 12.5 us, up and gate of one token 35 -> 47 us.)
#include "ffn_common.h"

namespace moe {
namespace {

constexpr int kTileK = 128, kTileN = 16;
constexpr int64_t kMaxDim = 1 << 22;
constexpr int64_t kMaxRows = 4096;
constexpr int64_t kMaxBytes = 0x7FFFFF00;  // of the rows that a product reads
constexpr uint32_t kPastEnd = 0x80000000u;  // above every descriptor's range
constexpr int64_t kMaxExperts = 1 << 16;
constexpr int64_t kMaxTiles = 1 << 25;  // waves of a launch, below 2^32 threads

__host__ __device__ constexpr int tile_bytes(int group) { return 1024 + kTileK / group * 32; }
__host__ __device__ inline int64_t tiles_k(int64_t K) { return (K + kTileK - 1) / kTileK; }
__host__ __device__ inline int64_t tiles_n(int64_t N) { return (N + kTileN - 1) / kTileN; }

bool group_ok(int32_t g) { return g == 32 || g == 64 || g == 128; }

// One thread per column and group, which it reads twice (256 x 2048 x 768 bf16, groups of
// 64: 780 us, 1.6 TB/s; once per weight).
template <typename T>
__global__ void w4_quantize_kernel(const T* W, int64_t E, int64_t K, int64_t N, int group,
                                   uint8_t* codes, bf16_t* scales) {
  const int64_t ng = (K + group - 1) / group;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= E * ng * N) return;
  const int64_t n = i % N, g = i / N % ng, e = i / N / ng;
  const int64_t k0 = g * group, k1 = k0 + group < K ? k0 + group : K;
  const T* w = W + e * K * N + n;
  float top = 0.f;
  for (int64_t k = k0; k < k1; ++k) top = fmaxf(top, fabsf(to_f32<T>(w[k * N])));
  const bf16_t sb = f32_to_bf16(top / 7.0f);
  const float s = bf16_to_f32(sb);
  scales[(e * ng + g) * N + n] = sb;
  for (int64_t k = k0; k < k1; ++k) {
    // s = 0 (a group of zeros, or too small for a bf16 scale): code 8
    const float q = s > 0.f ? rintf(to_f32<T>(w[k * N]) / s) : 0.f;
    codes[(e * K + k) * N + n] = (uint8_t)(int)(fminf(fmaxf(q, -8.f), 7.f) + 8.f);
  }
}

// One workgroup: 128 rows by 128 columns (8 tiles) of codes through LDS, so that they
// are read as 128 consecutive bytes and written as tiles (256 x 2048 x 768, groups of 64:
// 138 us, 4.6 TB/s).
__global__ __launch_bounds__(256) void w4_pack_kernel(const uint8_t* codes, const bf16_t* scales,
                                                      int64_t K, int64_t N, int group,
                                                      char* packed, int64_t blocks) {
  constexpr int PITCH = 128 + 4;
  __shared__ uint8_t lds[kTileK * PITCH];
  const int64_t nt = tiles_n(N), kt = tiles_k(K), ng = (K + group - 1) / group;
  const int64_t nb = (nt + 7) / 8;  // column blocks
  for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const int64_t kk = blk % kt, cb = blk / kt % nb, e = blk / kt / nb;
    for (int i = threadIdx.x; i < kTileK * 16; i += 256) {
      const int64_t k = kk * kTileK + i / 16, n = cb * 128 + i % 16 * 8;
      uint2 v = make_uint2(0x08080808u, 0x08080808u);
      if (k < K && n < N) {  // 8 codes of a row whose length is a multiple of 8
        const uint8_t* q = codes + (e * K + k) * N + n;
        uint8_t c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = q[j];
        v = __builtin_bit_cast(uint2, c);
      }
      uint32_t* at = reinterpret_cast<uint32_t*>(lds + i / 16 * PITCH + i % 16 * 8);
      at[0] = v.x;
      at[1] = v.y;
    }
    __syncthreads();
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    for (int t = threadIdx.x >> 6; t < 8; t += 4) {
      const int64_t ct = cb * 8 + t;
      if (ct >= nt) break;
      char* out = packed + ((e * nt + ct) * kt + kk) * tile_bytes(group);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v |= (lds[(32 * i + 8 * q + j) * PITCH + t * 16 + c] & 15u)
               << (4 * (j / 2) + 16 * (j % 2));
        w[i] = (v << 3) | (v >> 29);
      }
      *reinterpret_cast<uint4*>(out + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      const int ng_t = kTileK / group;
      for (int i = lane; i < ng_t * kTileN; i += 64) {
        const int64_t g = kk * ng_t + i % ng_t, m = ct * kTileN + i / ng_t;
        reinterpret_cast<bf16_t*>(out + 1024)[i] =
            g < ng && m < N ? scales[(e * ng + g) * N + m] : (bf16_t)0;
      }
    }
    __syncthreads();
  }
}

__device__ __forceinline__ f32x4_t mfma(uint4 a, uint4 b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// A constant in a vector register, where an instruction takes no literal.
__device__ __forceinline__ uint32_t in_vgpr(uint32_t c) {
  asm("" : "+v"(c));
  return c;
}

// 8 codes of a packed dword as bf16 values 16 + code, rows ascending: 3 shifts and 4
// and-or (m = 0x00780078, o = 0x41804180, in registers: as literals they take an
// and and an or each, 88 instead of 56 instructions per step of two tiles).
__device__ __forceinline__ uint4 unpack(uint32_t w, uint32_t m, uint32_t o) {
  return make_uint4((w & m) | o, ((w >> 4) & m) | o, ((w >> 8) & m) | o,
                    (__builtin_amdgcn_alignbit(w, w, 12) & m) | o);
}

using rsrc_t = __amdgpu_buffer_rsrc_t;
constexpr int kNonTemporal = 2;  // load hint: weights are read once

__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

// What a wave holds of one 128-row step: its column tiles' codes and scales and
// 16 rows of X (lane l: row l % 16, values 8 (l / 16) .. + 7 of each 32).
template <int G, int NP>
struct Step {
  static constexpr int NG = kTileK / G;
  uint4 a[4];
  uint4 c[NP];
  uint32_t s[NP][NG == 4 ? 2 : 1];

  // step kt of the stream
  __device__ __forceinline__ void load(const rsrc_t (&w)[NP], int kt) {
    const int lane = threadIdx.x & 63;
    const uint32_t o = (uint32_t)kt * tile_bytes(G);
    const uint32_t os = o + 1024 + (lane & 15) * (NG * 2);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      c[p] = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(w[p], o + lane * 16, 0, kNonTemporal));
      if constexpr (NG == 1) {
        s[p][0] = __builtin_amdgcn_raw_buffer_load_b16(w[p], os, 0, kNonTemporal);
      } else if constexpr (NG == 2) {
        s[p][0] = __builtin_amdgcn_raw_buffer_load_b32(w[p], os, 0, kNonTemporal);
      } else {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(w[p], os, 0, kNonTemporal);
        s[p][0] = v[0];
        s[p][1] = v[1];
      }
    }
  }
  __device__ __forceinline__ float scale(int p, int g) const {
    const uint32_t v = s[p][g / 2];
    return __uint_as_float(g & 1 ? v & 0xFFFF0000u : v << 16);
  }

  // xoff: byte offset in x of this lane's row at k = 8 (lane / 16), or past the end;
  // past: for the last step, the top bit (past the end) where its K values are
  __device__ __forceinline__ void load_x(rsrc_t x, uint32_t xoff, const uint32_t (&past)[4],
                                         int kt, int last) {
    // behind the last step every row's offset is past the end (and none wraps around)
    const uint32_t o = xoff + (kt > last ? (uint32_t)kMaxBytes : (uint32_t)kt * (kTileK * 2));
    const uint32_t sel = kt == last ? kPastEnd : 0;  // (not behind it: no sum may wrap)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                           x, ((past[i] & sel) | o) + 64 * i, 0, 0));
  }
  __device__ __forceinline__ void compute(uint32_t m, uint32_t o, f32x4_t (&acc)[NP]) const {
    constexpr uint32_t m24 = 0xC1C0C1C0u;  // -24, -24
    const uint4 bias = make_uint4(m24, m24, m24, m24);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x4_t start = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < G / 32; ++i) start = mfma(a[g * (G / 32) + i], bias, start);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        f32x4_t t = start;
#pragma unroll
        for (int i = 0; i < G / 32; ++i) {
          const int k = g * (G / 32) + i;
          const uint32_t w = k == 0 ? c[p].x : k == 1 ? c[p].y : k == 2 ? c[p].z : c[p].w;
          t = mfma(a[k], unpack(w, m, o), t);
        }
        const float sc = scale(p, g);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[p][r] += sc * t[r];
      }
    }
  }
};

// (Rows with a matrix each, 2048 x 768, 64 matrices, groups of 64: 8 rows 7.3 us; 64 rows
// of 39 matrices 15 us, 2.2 TB/s; 512 rows, 16 of a matrix at a time, 50 us.)
//
// The rows of the workgroup's list (f indexes) that blockIdx's entry stands for:
//   by_row: entry y stands for ids[y]'s expert if no earlier row has it;
//   else:   entry y stands for expert y.
// Fills list (LDS) with the rows whose id is that expert e, in no particular
// order (rows do not meet in the products), and returns their number.
__device__ __forceinline__ int collect_rows(const int32_t* ids, int F, int e, bool by_row, int y,
                                            int* list, int* count) {
  if (threadIdx.x == 0) count[0] = count[1] = 0;
  __syncthreads();
  for (int f = threadIdx.x; f < F; f += blockDim.x)
    if (ids[f] == e) {
      if (by_row && f < y) count[1] = 1;
      list[atomicAdd(&count[0], 1)] = f;
    }
  __syncthreads();
  return count[1] ? 0 : count[0];
}

enum { kMatvec, kUpgate, kDown };

// Products of a wave and the column tiles they cover: up and gate of one tile; two
// tiles of the down projection, which then share X's loads and the -24 MFMAs; one
// where there are few columns.
constexpr int products(int op) { return op == kMatvec ? 1 : 2; }
constexpr int tiles_per_wave(int op) { return op == kDown ? 2 : 1; }
// Steps of loads ahead of a wave's products. Where there are waves enough to a SIMD (5 at
// 80 to 96 registers) one step each hides the latency best: 64 tokens of 2048 x 768,
// 256 experts: up and gate 78 us, down 46 us; 2 steps (4 waves) 78 and 51 us; 3 steps
// (3 waves) 86 and 57 us; 4 steps 94 and 78 us.
constexpr int steps_ahead(int op) { return op == kMatvec ? 2 : 1; }

// h is rounded to bf16, the down product's operand, as the MoE layer's is (64 tokens of
// 2048 x 768: 0.0022 in the outputs, 2-norm against 64 bits, 0.0017 from their own
// rounding alone).
template <int OP>
__device__ __forceinline__ void w4_store(void* out, int64_t o, float v, float v1, int out_f32) {
  if constexpr (OP == kUpgate)
    reinterpret_cast<bf16_t*>(out)[o] = f32_to_bf16(silu_f32(v) * v1);
  else if (OP == kDown || out_f32)
    reinterpret_cast<float*>(out)[o] = v;
  else
    reinterpret_cast<bf16_t*>(out)[o] = f32_to_bf16(v);
}

struct W4Args {
  const bf16_t* X;        // rows of K values
  const char* w[2];       // packed matrices (up and gate, or one)
  const char* ws[2];      // the shared expert's
  const int32_t* ids;     // [F] or null: every row takes matrix 0
  void* out;              // upgate: h [F][N]; matvec: Y [F][N]; down: slots [F][N] fp32
  void* outs;             // the shared expert's rows
  const bf16_t* Xs;       // the shared expert's input rows
  int64_t K, N;           // routed: K values per row, N columns
  int64_t Ks, Ns;         // shared
  int F, E, k, S;         // routed rows, matrices, routed rows per row of X, shared rows
  int by_row, entries;    // collect_rows' entries in use
  int groups, groups_s;   // workgroups per entry (routed, shared)
  int wk;                 // waves that share a column tile's K (then tiles = 1)
  int64_t x_bytes, xs_bytes;
  int out_f32;
};

// Workgroup b: column tiles of one entry. Its waves are wn tiles (or pairs) by wk
// shares of K (every wk-th step); the shares are added in wave order through LDS.
template <int G, int OP>
__global__ __launch_bounds__(512, OP == kMatvec ? 4 : 5) void w4_kernel(W4Args p) {
  constexpr int NP = products(OP);
  constexpr int TPW = tiles_per_wave(OP);
  constexpr int DEPTH = steps_ahead(OP);
  extern __shared__ char smem[];
  __shared__ int count[2];
  const int waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wk = p.wk, wn = waves / wk;
  float* red = reinterpret_cast<float*>(smem);                   // [waves][NP][256]
  int* list = reinterpret_cast<int*>(smem + waves * NP * 1024);  // [F]

  int64_t b = blockIdx.x;
  const int64_t routed = (int64_t)p.entries * p.groups;
  const bool shared = b >= routed;
  const bool listed = !shared && p.ids != nullptr;
  if (shared) b -= routed;
  const int per = shared ? p.groups_s : p.groups;
  const int y = (int)(b / per), grp = (int)(b % per);
  const int64_t K = shared ? p.Ks : p.K, N = shared ? p.Ns : p.N;
  const int e = !listed ? 0 : p.by_row ? p.ids[y] : y;  // the same for every thread
  const int64_t group_tiles = (int64_t)wn * TPW;  // column tiles of the workgroup
  if (e < 0 || e >= p.E) {
    // rows without an expert: zeros, written by the row's own entry, or by the
    // entry behind the experts
    if (OP == kMatvec)
      for (int f = p.by_row ? y : 0; f < (p.by_row ? y + 1 : p.F); ++f) {
        const int id = p.ids[f];
        if (id >= 0 && id < p.E) continue;
        for (int64_t c = grp * group_tiles * kTileN + threadIdx.x;
             c < N && c < (grp + 1) * group_tiles * kTileN; c += blockDim.x) {
          if (p.out_f32)
            reinterpret_cast<float*>(p.out)[f * N + c] = 0.f;
          else
            reinterpret_cast<bf16_t*>(p.out)[f * N + c] = 0;
        }
      }
    return;
  }

  // this wave's column tiles; those past the last one read as zeros
  const int kt_n = (int)tiles_k(K);
  const int64_t col_bytes = (int64_t)kt_n * tile_bytes(G);
  const int64_t ct0 = grp * group_tiles + (int64_t)(wave / wk) * TPW;
  rsrc_t w[NP];
#pragma unroll
  for (int m = 0; m < NP; ++m) {
    const int64_t t = ct0 + (TPW == 2 ? m : 0);
    const bool in = t < tiles_n(N);
    const int mat = OP == kUpgate ? m : 0;
    w[m] = make_rsrc((shared ? p.ws[mat] : p.w[mat]) +
                         ((int64_t)e * tiles_n(N) + (in ? t : 0)) * col_bytes,
                     in ? col_bytes : 0);
  }
  const int w0 = wave % wk;
  Step<G, NP> st[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) st[d].load(w, w0 + d * wk);  // before the rows are known
  int n_rows, row0 = 0;
  if (listed) {
    n_rows = collect_rows(p.ids, p.F, e, p.by_row, y, list, count);
    if (n_rows == 0) return;
  } else {
    row0 = 16 * y;
    const int all = shared ? p.S : p.F;
    n_rows = all - row0 < 16 ? all - row0 : 16;
  }
  const rsrc_t x = make_rsrc(shared ? p.Xs : p.X, shared ? p.xs_bytes : p.x_bytes);
  void* out = shared ? p.outs : p.out;
  auto row_of = [&](int r) { return listed ? list[r] : row0 + r; };
  const int last = kt_n - 1;
  uint32_t past[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    past[i] = (int64_t)last * kTileK + 32 * i + 8 * lg < K ? 0 : kPastEnd;
  const uint32_t um = in_vgpr(0x00780078u), uo = in_vgpr(0x41804180u);

  for (int r0 = 0; r0 < n_rows; r0 += 16) {
    uint32_t xoff = kPastEnd;
    if (r0 + lr < n_rows) {
      const int f = row_of(r0 + lr);
      xoff = (uint32_t)((int64_t)(listed && OP == kUpgate ? f / p.k : f) * K * 2) + lg * 16;
    }
    if (r0)
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) st[d].load(w, w0 + d * wk);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) st[d].load_x(x, xoff, past, w0 + d * wk, last);
    f32x4_t acc[NP];
#pragma unroll
    for (int m = 0; m < NP; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int kt = w0; kt < kt_n;) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d, kt += wk) {
        st[d].compute(um, uo, acc);  // past the last step: scales of 0
        const int next = kt + DEPTH * wk;
        st[d].load(w, next);
        st[d].load_x(x, xoff, past, next, last);
      }
    }
#pragma unroll
    for (int m = 0; m < NP; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[(wave * NP + m) * 256 + (4 * lg + r) * 16 + lr] = acc[m][r];
    __syncthreads();
    for (int i = threadIdx.x; i < wn * TPW * 256; i += blockDim.x) {
      const int t = i >> 8, r = (i >> 4) & 15, c = i & 15;  // t: column tile of the group
      const int64_t n = (grp * group_tiles + t) * kTileN + c;
      if (r0 + r >= n_rows || n >= N) continue;
      // the first wave of the tile, and its place among that wave's products
      const float* q0 = red + (t / TPW * wk * NP + t % TPW) * 256 + (i & 255);
      float v[NP / TPW];
#pragma unroll
      for (int m = 0; m < NP / TPW; ++m) {
        v[m] = q0[m * 256];
        for (int q = 1; q < wk; ++q) v[m] += q0[(q * NP + m) * 256];
      }
      w4_store<OP>(out, (int64_t)row_of(r0 + r) * N + n, v[0], v[NP / TPW - 1], p.out_f32);
    }
    if (r0 + 16 < n_rows) __syncthreads();
  }
}

// O_t = sum_j w_tj slot_tj (+ the shared row), slots without an expert skipped.
template <typename T>
__global__ void w4_combine_kernel(int64_t S, int64_t H, int k, int E, const int32_t* ids,
                                  const float* w, const float* slots, const float* shared,
                                  T* O) {
  const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4;
  if (i >= S * H) return;
  const int64_t t = i / H, c = i % H;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
  // 8 slots' loads at a time, whether they hold an expert's row or not
  for (int j0 = 0; j0 < k; j0 += 8) {
    f32x4_t v[8];
    float wj[8];
    bool in[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int64_t f = t * k + (j0 + q < k ? j0 + q : 0);
      const int id = ids[f];
      in[q] = j0 + q < k && id >= 0 && id < E;
      wj[q] = w[f];
      v[q] = load4(slots + f * H + c);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
#pragma unroll
      for (int r = 0; r < 4; ++r) a[r] = in[q] ? a[r] + wj[q] * v[q][r] : a[r];
  }
  if (shared != nullptr) {
    const f32x4_t v = load4(shared + t * H + c);
#pragma unroll
    for (int r = 0; r < 4; ++r) a[r] += v[r];
  }
  store_n(O + i, a);
}

moe_status enqueued() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Waves that share one column tile's K (wk) and tiles (or pairs) per workgroup:
// waves share K until there are about as many as the chip holds, while each keeps
// min_steps to stream.
void wave_shape(int64_t wave_tiles, int64_t K, int min_steps, int* wk, int* wn) {
  int s = 1;
  while (s < 8 && wave_tiles * s < 4096 && tiles_k(K) >= min_steps * 2 * s) s *= 2;
  *wk = s;
  *wn = s >= 4 ? 1 : 4 / s;
}

template <int OP>
void launch_w4(int group, W4Args& p, int64_t row_blocks, int64_t row_blocks_s, hipStream_t st) {
  int wn;
  const int64_t ct = tiles_n(p.N), cts = row_blocks_s ? tiles_n(p.Ns) : 0;
  constexpr int TPW = tiles_per_wave(OP);
  // (one row of 7168 x 2048: 7.5 us with 7 steps per wave, 8.8 us with 12)
  wave_shape((row_blocks * ct + row_blocks_s * cts) / TPW, p.K, OP == kMatvec ? 3 : 6, &p.wk,
             &wn);
  p.entries = (int)row_blocks;
  p.groups = (int)((ct + wn * TPW - 1) / (wn * TPW));
  p.groups_s = (int)((cts + wn * TPW - 1) / (wn * TPW));
  const int waves = p.wk * wn;
  const size_t lds = (size_t)waves * products(OP) * 1024 +
                     (p.ids != nullptr ? (size_t)p.F * sizeof(int) : 0);
  const unsigned grid = (unsigned)(row_blocks * p.groups + row_blocks_s * p.groups_s);
  if (group == 32)
    w4_kernel<32, OP><<<grid, 64 * waves, lds, st>>>(p);
  else if (group == 64)
    w4_kernel<64, OP><<<grid, 64 * waves, lds, st>>>(p);
  else
    w4_kernel<128, OP><<<grid, 64 * waves, lds, st>>>(p);
}

moe_status check_w4(int64_t E, int64_t K, int64_t N, int32_t group) {
  if (E < 1 || K < 1 || N < 1 || !group_ok(group)) return MOE_ERR_INVALID_ARGUMENT;
  if (K % 8 || N % 8 || K >= kMaxDim || N >= kMaxDim || E > kMaxExperts)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The workspace of moe_w4_forward: h rows, slots, the shared expert's.
struct W4Ws {
  size_t h, hs, y, ys, total;
};
W4Ws w4_ws(const moe_shape* s) {
  W4Ws w;
  const size_t F = (size_t)(s->S * s->k);
  size_t o = 0;
  auto take = [&](size_t n) {
    const size_t at = o;
    o += ffn_round_up(n, 256);
    return at;
  };
  w.h = take(F * s->D * 2);
  w.y = take(F * s->H * 4);
  w.hs = take((size_t)(s->S * s->D_shared) * 2);
  w.ys = take(s->D_shared ? (size_t)(s->S * s->H) * 4 : 0);
  w.total = o ? o : 256;
  return w;
}

moe_status check_w4_layer(const moe_shape* s) {
  if (s == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16 && s->dtype != MOE_MXFP8)
    return MOE_ERR_INVALID_ARGUMENT;
  if (s->S < 0 || s->H < 1 || s->D < 1 || s->E < 1 || s->k < 1 || s->k > s->E ||
      s->D_shared < 0 || s->capacity < 0)
    return MOE_ERR_INVALID_ARGUMENT;
  if (s->dtype != MOE_BF16 || s->capacity != 0 || (s->flags & ~MOE_OUTPUT_F32) != 0)
    return MOE_ERR_UNSUPPORTED;
  if (s->H % 8 || s->D % 8 || s->D_shared % 8 || s->H >= kMaxDim || s->D >= kMaxDim ||
      s->D_shared >= kMaxDim || s->E > 1024 || s->k > 32 || s->S > kMaxRows ||
      s->S * s->k > kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  if (s->S * s->H * 2 >= kMaxBytes || s->S * s->k * s->D * 2 >= kMaxBytes ||
      s->S * s->D_shared * 2 >= kMaxBytes)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_w4_weight_bytes(int64_t E, int64_t K, int64_t N, int32_t group) {
  if (check_w4(E, K, N, group) != MOE_OK) return 0;
  return (size_t)E * tiles_n(N) * tiles_k(K) * tile_bytes(group);
}

extern "C" moe_status moe_quantize_w4(const void* W, int64_t E, int64_t K, int64_t N,
                                      int32_t dtype, int32_t group, uint8_t* codes, void* scales,
                                      void* stream) {
  const moe_status st = check_w4(E, K, N, group);
  if (st != MOE_OK) return st;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (W == nullptr || codes == nullptr || scales == nullptr || ffn_shared({codes, scales}, {W}))
    return MOE_ERR_INVALID_ARGUMENT;
  const int es = dtype == MOE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(W) % es || reinterpret_cast<uintptr_t>(scales) % 2)
    return MOE_ERR_UNSUPPORTED;
  const int64_t n = E * ((K + group - 1) / group) * N;
  if ((n + 255) / 256 >= (1 << 24)) return MOE_ERR_UNSUPPORTED;  // a launch's 2^32 threads
  const unsigned grid = (unsigned)((n + 255) / 256);
  if (dtype == MOE_F32)
    w4_quantize_kernel<<<grid, 256, 0, (hipStream_t)stream>>>((const float*)W, E, K, N, group,
                                                              codes, (bf16_t*)scales);
  else
    w4_quantize_kernel<<<grid, 256, 0, (hipStream_t)stream>>>((const bf16_t*)W, E, K, N, group,
                                                              codes, (bf16_t*)scales);
  return enqueued();
}

extern "C" moe_status moe_pack_w4_weights(const uint8_t* codes, const void* scales, int64_t E,
                                          int64_t K, int64_t N, int32_t group, void* packed,
                                          void* stream) {
  const moe_status st = check_w4(E, K, N, group);
  if (st != MOE_OK) return st;
  if (codes == nullptr || scales == nullptr || packed == nullptr ||
      ffn_shared({packed, scales}, {codes}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!ffn_aligned16(packed) || reinterpret_cast<uintptr_t>(scales) % 2)
    return MOE_ERR_UNSUPPORTED;
  const int64_t blocks = E * ((tiles_n(N) + 7) / 8) * tiles_k(K);
  w4_pack_kernel<<<(unsigned)(blocks < (1 << 20) ? blocks : 1 << 20), 256, 0,
                   (hipStream_t)stream>>>(codes, (const bf16_t*)scales, K, N, group,
                                          (char*)packed, blocks);
  return enqueued();
}

extern "C" moe_status moe_w4_matvec(int64_t S, int64_t K, int64_t N, int64_t E, int32_t group,
                                    int32_t flags, const void* X, const void* W,
                                    const int32_t* expert_ids, void* Y, void* stream) {
  if (S < 0 || (flags & ~MOE_OUTPUT_F32) != 0) return MOE_ERR_INVALID_ARGUMENT;
  const moe_status st = check_w4(E, K, N, group);
  if (st != MOE_OK) return st;
  if (S > kMaxRows || S * K * 2 >= kMaxBytes) return MOE_ERR_UNSUPPORTED;
  if (S == 0) return MOE_OK;
  if (X == nullptr || W == nullptr || Y == nullptr || ffn_shared({Y}, {X, W, expert_ids}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!ffn_aligned16(X) || !ffn_aligned16(W) || !ffn_aligned16(Y) ||
      reinterpret_cast<uintptr_t>(expert_ids) % 4)
    return MOE_ERR_UNSUPPORTED;
  W4Args p = {};
  p.X = (const bf16_t*)X;
  p.w[0] = (const char*)W;
  p.ids = expert_ids;
  p.out = Y;
  p.K = K;
  p.N = N;
  p.F = (int)S;
  p.E = (int)E;
  p.k = 1;
  p.by_row = S <= E;
  p.x_bytes = S * K * 2;
  p.out_f32 = (flags & MOE_OUTPUT_F32) != 0;
  const int64_t entries = expert_ids == nullptr ? (S + 15) / 16 : p.by_row ? S : E + 1;
  if (entries * tiles_n(N) >= kMaxTiles) return MOE_ERR_UNSUPPORTED;
  launch_w4<kMatvec>(group, p, entries, 0, (hipStream_t)stream);
  return enqueued();
}

extern "C" size_t moe_w4_forward_workspace_bytes(const moe_shape* shape) {
  return check_w4_layer(shape) == MOE_OK ? w4_ws(shape).total : 0;
}

extern "C" moe_status moe_w4_forward(const moe_shape* s, int32_t group, const void* A,
                                     const void* W_up, const void* W_gate, const void* W_down,
                                     const void* Ws_up, const void* Ws_gate, const void* Ws_down,
                                     const int32_t* topk_ids, const float* topk_weights, void* O,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  const moe_status st = check_w4_layer(s);
  if (st != MOE_OK) return st;
  if (!group_ok(group)) return MOE_ERR_INVALID_ARGUMENT;
  if (s->S == 0) return MOE_OK;
  if (A == nullptr || W_up == nullptr || W_gate == nullptr || W_down == nullptr ||
      topk_ids == nullptr || topk_weights == nullptr || O == nullptr ||
      ffn_shared({O, workspace}, {A, W_up, W_gate, W_down, Ws_up, Ws_gate, Ws_down, topk_ids,
                                  topk_weights}))
    return MOE_ERR_INVALID_ARGUMENT;
  const bool sh = s->D_shared > 0;
  if ((Ws_up != nullptr) != sh || (Ws_gate != nullptr) != sh || (Ws_down != nullptr) != sh)
    return MOE_ERR_INVALID_ARGUMENT;
  for (const void* q : {A, W_up, W_gate, W_down, Ws_up, Ws_gate, Ws_down, (const void*)O,
                        (const void*)workspace})
    if (!ffn_aligned16(q)) return MOE_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(topk_ids) % 4 || reinterpret_cast<uintptr_t>(topk_weights) % 4)
    return MOE_ERR_UNSUPPORTED;
  const W4Ws ws = w4_ws(s);
  if (workspace == nullptr || workspace_bytes < ws.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  char* base = (char*)workspace;
  hipStream_t stq = (hipStream_t)stream;
  W4Args p = {};
  p.F = (int)(s->S * s->k);
  p.E = (int)s->E;
  p.k = (int)s->k;
  p.S = sh ? (int)s->S : 0;
  p.ids = topk_ids;
  p.by_row = p.F <= p.E;
  const int64_t entries = p.by_row ? p.F : p.E, blocks_s = (p.S + 15) / 16;
  const int64_t cols = tiles_n(s->D > s->H ? s->D : s->H);
  const int64_t cols_s = tiles_n(s->D_shared > s->H ? s->D_shared : s->H);
  if (entries * cols + blocks_s * cols_s >= kMaxTiles) return MOE_ERR_UNSUPPORTED;
  // up, gate and SwiGLU
  p.X = p.Xs = (const bf16_t*)A;
  p.w[0] = (const char*)W_up;
  p.w[1] = (const char*)W_gate;
  p.ws[0] = (const char*)Ws_up;
  p.ws[1] = (const char*)Ws_gate;
  p.out = base + ws.h;
  p.outs = base + ws.hs;
  p.x_bytes = p.xs_bytes = s->S * s->H * 2;
  p.K = p.Ks = s->H;
  p.N = s->D;
  p.Ns = s->D_shared;
  launch_w4<kUpgate>(group, p, entries, blocks_s, stq);
  // down
  p.X = (const bf16_t*)(base + ws.h);
  p.Xs = (const bf16_t*)(base + ws.hs);
  p.w[0] = (const char*)W_down;
  p.ws[0] = (const char*)Ws_down;
  p.out = base + ws.y;
  p.outs = base + ws.ys;
  p.x_bytes = p.F * s->D * 2;
  p.xs_bytes = s->S * s->D_shared * 2;
  p.K = s->D;
  p.Ks = s->D_shared;
  p.N = p.Ns = s->H;
  launch_w4<kDown>(group, p, entries, blocks_s, stq);
  const float* y = (const float*)(base + ws.y);
  const float* ys = sh ? (const float*)(base + ws.ys) : nullptr;
  const unsigned grid = (unsigned)((s->S * s->H / 4 + 63) / 64);
  if (s->flags & MOE_OUTPUT_F32)
    w4_combine_kernel<<<grid, 64, 0, stq>>>(s->S, s->H, p.k, p.E, topk_ids, topk_weights, y, ys,
                                             (float*)O);
  else
    w4_combine_kernel<<<grid, 64, 0, stq>>>(s->S, s->H, p.k, p.E, topk_ids, topk_weights, y, ys,
                                             (bf16_t*)O);
  return enqueued();
}
