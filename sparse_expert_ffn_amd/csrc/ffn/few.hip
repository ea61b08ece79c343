// The whole MoE layer for a few tokens in two launches (include/moe_ffn.h).
//
// Decode is bound by the chosen experts' bytes, and at one token by how many times the
// device has to start and finish something.
//   route    (512 rows of H, 64 experts, 16 tokens)  the router's partial scores; clears
//            what the next launch counts with
//   experts  (entry, 64 or 128 columns of D)  h = SiLU(a Wu) * (a Wg) for its columns, then
//            at once their share of the down product, y = h Wd over all of H
// An entry is an expert with its rows, or the shared expert with 16 tokens. A workgroup of
// the second launch needs no other's h: what it would have to wait for is summed instead.
// The last of an entry's workgroups to arrive adds their shares, the last of a token's
// entries forms the token's output. Nothing waits: whatever else runs on the device, and in
// whatever order workgroups start, each runs to its end. (As one grid of tasks that waited
// for each other's h, with claims from counters, a token took 87 us: a wait, a claim or a
// count is 1 to 2 us of memory latency, and there were eight in a row.)
//
// Up to 8 tokens every workgroup sums the scores and selects the top-k for itself; beyond,
// a launch of its own does it (one wave per token). With 8-bit weights h's row scale needs
// the whole row: the experts' launch becomes two, up/gate and down.
//
// Weights go from memory into registers, rows of 128 bytes to 16 lanes, and become MFMA
// operands there: no LDS on their way. 8 waves: up or gate, 64 columns each, shares of K
// added through LDS; then 64 columns of H each.
//   bf16: a lane holds 2 x 8 rows of 4 columns; byte permutes give the operands (8 rows of a
//         column) of v_mfma_f32_16x16x32_bf16
//   fp32: 2 x 4 rows of 4 columns, v_mfma_f32_16x16x4_f32 (K in an order that suits)
//   int8: packed in operand order, v_mfma_i32_16x16x64_i8
#include "gemm_direct.h"
#include "i8.h"
#include "topk.h"

namespace moe {
namespace {

using rsrc_t = __amdgpu_buffer_rsrc_t;
constexpr uint32_t kPastEnd = 0x80000000u;  // above every descriptor's range
constexpr int64_t kMaxMatrix = 0x7F000000;
constexpr int kNonTemporal = 2;      // load hint: weights are read once
constexpr int64_t kMaxTokens = 128;
constexpr int64_t kMaxSize = 65536;  // H, D, D_shared
constexpr int kMaxRows = (int)kMaxTokens * 32;  // assignments
constexpr int kThreads = 512, kWaves = 8;
constexpr int kCols = 64;            // columns of a wave
constexpr int kRouteRows = 512;      // K rows of a router workgroup, 64 to a wave
constexpr int kOwnRoute = 8;         // tokens that each workgroup routes for itself

struct FewArgs {
  const void* A;
  const void* Wr;
  const float* bias;
  const char* w[3];    // up, gate, down
  const char* ws[3];   // the shared expert's
  int32_t* ids;        // [S][k], written when Wr is given
  float* tw;
  void* O;
  float* score;        // [route splits][S][E]
  int* entry_done;     // [entries + shared] arrived column groups
  int* token_done;     // [S] arrived entries
  uint32_t* top;       // int8: [F + S] abs_bits of the largest h
  int n_words;         // of these three
  int8_t* xc;          // int8: codes and scales of the tokens
  float* xs;
  float* h;            // int8: [F][D], then [S][Ds]
  float* y;            // [slices][F + S][H]
  int S, H, D, Ds, E, k, F;
  int by_row, entries; // an entry per assignment (the first of its expert), or per expert
  int shared;          // shared entries
  int slices, slices_s;  // column groups of D
  int route_splits, renormalize, out_f32;
  int routed;          // ids and tw are there (given, or by a launch before)
};

// A value that is the same in all lanes, in a scalar register (the compiler leaves quotients
// and loaded values in vector ones, and then takes a loop around every descriptor load).
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint64_t u =
      ((uint64_t)(uint32_t)uniform((int)(a >> 32)) << 32) | (uint32_t)uniform((int)a);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(u), 0, uniform((int)bytes),
                                           0x00020000);
}
__device__ __forceinline__ uint4 load16(rsrc_t r, uint32_t o) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// What workgroups of one launch exchange goes through accesses of device scope: stores are
// written through to memory, loads pass the caches that another XCD's stores do not reach.
// Then a count needs no cache written back or invalidated before it.
constexpr int kDevice = 16;  // the sc1 bit of a buffer access
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ f32x4_t load_shared(rsrc_t r, uint32_t o) {
  return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, kDevice));
}
__device__ __forceinline__ void store_shared(rsrc_t r, uint32_t o, f32x4_t v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), r, o, 0, kDevice);
}
__device__ __forceinline__ int count_up(int* p) {
  return __hip_atomic_fetch_add(p, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Every wave has to be here before a count that others read: its stores are in memory.
__device__ __forceinline__ void stores_done() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

// ------------------------------------------------------------ streaming a weight

enum { kBf16, kF32, kI8 };
template <int P>
struct Kind;
template <>
struct Kind<kBf16> {
  using T = bf16_t;     // activations
  using Val = float;
  using Acc = f32x4_t;
  static constexpr int ES = 2, STEP = 64, NX = 2;  // bytes of a weight, K rows per step
};
template <>
struct Kind<kF32> {
  using T = float;
  using Val = float;
  using Acc = f32x4_t;
  static constexpr int ES = 4, STEP = 32, NX = 2;
};
template <>
struct Kind<kI8> {
  using T = bf16_t;
  using Val = int;
  using Acc = i32x4_t;
  static constexpr int NX = 1;
};

// 64 columns of a matrix [K][N] from n0 on; K values from k0 on.
template <int P>
struct Columns {
  rsrc_t r;
  uint32_t off, row, step;

  __device__ __forceinline__ Columns() {}
  __device__ __forceinline__ Columns(const char* matrix, int K, int N, int n0, int k0 = 0) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    if constexpr (P == kI8) {
      const uint32_t kt = (uint32_t)i8_tiles_k(K);
      r = make_rsrc(matrix, n0 < N ? i8_code_bytes(K, N) : 0);
      off = (uint32_t)((n0 / 16) * kt + k0 / 64) * 1024 + lane * 16;
      row = kt * 1024;
      step = 1024;
    } else {
      constexpr int ES = Kind<P>::ES;
      r = make_rsrc(matrix, (int64_t)K * N * ES);
      off = n0 + 4 * c < N
                ? (uint32_t)((k0 + (P == kBf16 ? 8 : 4) * g) * N + n0 + 4 * c) * ES
                : kPastEnd;
      row = (uint32_t)N * ES;
      step = row * Kind<P>::STEP;
    }
  }
};

template <int P>
struct Step {
  using Acc = typename Kind<P>::Acc;
  static constexpr int NX = Kind<P>::NX;
  uint4 w[P == kI8 ? 4 : 8];  // bf16: two rows of 8 bytes each

  __device__ __forceinline__ void load(const Columns<P>& m, uint32_t o) {
    if constexpr (P == kI8) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                             m.r, o + j * m.row, 0, kNonTemporal));
    } else if constexpr (P == kBf16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t at = o + (uint32_t)(i / 4 * 32 + i % 4 * 2) * m.row;
        const auto a = __builtin_amdgcn_raw_buffer_load_b64(m.r, at, 0, kNonTemporal);
        const auto b = __builtin_amdgcn_raw_buffer_load_b64(m.r, at + m.row, 0, kNonTemporal);
        w[i] = make_uint4(a[0], a[1], b[0], b[1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = __builtin_bit_cast(
            uint4, __builtin_amdgcn_raw_buffer_load_b128(
                       m.r, o + (uint32_t)(i / 4 * 16 + i % 4) * m.row, 0, kNonTemporal));
    }
  }
  // Step s of the columns; behind the last one (steps): zeros.
  __device__ __forceinline__ void load(const Columns<P>& m, int s, int steps) {
    load(m, s < steps ? m.off + (uint32_t)s * m.step : kPastEnd);
  }
  __device__ __forceinline__ void compute(const uint4 (&x)[NX], Acc (&acc)[4]) const {
    if constexpr (P == kBf16) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bf16x8_t a = __builtin_bit_cast(bf16x8_t, x[h]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // column j of the lane's 4: rows 2 i and 2 i + 1 in dword i
          const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
          uint32_t d[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            d[i] = __builtin_amdgcn_perm(word(w[4 * h + i], 2 + j / 2), word(w[4 * h + i], j / 2),
                                         sel);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              a, __builtin_bit_cast(bf16x8_t, make_uint4(d[0], d[1], d[2], d[3])), acc[j], 0, 0,
              0);
        }
      }
    } else if constexpr (P == kF32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = __uint_as_float(word(x[i / 4], i % 4));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, __uint_as_float(word(w[i], j)), acc[j],
                                                        0, 0, 0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, x[0]),
                                                       __builtin_bit_cast(i32x4_t, w[j]), acc[j],
                                                       0, 0, 0);
    }
  }
};

// 16 rows of the other operand, 64 NX bytes of each per step (lane l: row l % 16, 16 bytes at
// 16 (l / 16) of every 64); rows that are not there and what lies behind a row's end read
// as zeros.
struct Rows {
  rsrc_t r;
  uint32_t off;    // of this lane's row
  uint32_t bytes;  // of a row
  template <int NX>
  __device__ __forceinline__ void load(int s, uint4 (&x)[NX]) const {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const uint32_t at = (uint32_t)(s * NX + i) * 64 + ((threadIdx.x & 63) >> 4) * 16;
      x[i] = load16(r, at < bytes ? off + at : kPastEnd);
    }
  }
};
// int8's h: fp32 rows, quantised as they are read.
struct QuantRows {
  rsrc_t r;
  uint32_t off, bytes;
  Quant q;
  struct Raw {
    uint4 v[4];
  };
  __device__ __forceinline__ void load(int s, Raw& x) const {
    const uint32_t at = ((uint32_t)s * 64 + ((threadIdx.x & 63) >> 4) * 16) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = load16(r, at < bytes ? off + at + 16 * i : kPastEnd);
  }
  __device__ __forceinline__ void codes(const Raw& x, uint4 (&c)[1]) const {
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d[i] = q.pack4(__uint_as_float(x.v[i].x), __uint_as_float(x.v[i].y),
                     __uint_as_float(x.v[i].z), __uint_as_float(x.v[i].w));
    c[0] = make_uint4(d[0], d[1], d[2], d[3]);
  }
};

// Rows 4 (l / 16) + r and columns of the accumulators that a lane holds: 4 c .. + 3 (int8: c,
// 16 + c, ..) of the wave's 64.
template <int P>
__device__ __forceinline__ void put_sums(const typename Kind<P>::Acc (&acc)[4],
                                         typename Kind<P>::Val* to, int n) {
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (4 * g + r >= n) continue;
    typename Kind<P>::Val* row = to + (4 * g + r) * kCols;
    if constexpr (P == kI8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) row[16 * j + c] = acc[j][r];
    } else {
      *reinterpret_cast<typename Kind<P>::Acc*>(row + 4 * c) =
          typename Kind<P>::Acc{acc[0][r], acc[1][r], acc[2][r], acc[3][r]};
    }
  }
}

// ------------------------------------------------------------ router

// E that is no whole number of 16-byte vectors: element by element.
template <int P>
__device__ __forceinline__ void load_router(Step<P>& st, const Columns<P>& m, int s, int K, int N,
                                            int n0) {
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  auto at = [&](int k, int n) {
    return k < K && n < N ? (uint32_t)(k * N + n) * Kind<P>::ES : kPastEnd;
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t d[4];
    if constexpr (P == kBf16) {
#pragma unroll
      for (int v = 0; v < 8; ++v) {  // two rows of 4
        const int k = s * 64 + i / 4 * 32 + 8 * g + i % 4 * 2 + v / 4;
        const uint32_t b =
            __builtin_amdgcn_raw_buffer_load_b16(m.r, at(k, n0 + 4 * c + v % 4), 0, 0);
        d[v / 2] = v & 1 ? d[v / 2] | b << 16 : b;
      }
    } else {
      const int k = s * 32 + i / 4 * 16 + 4 * g + i % 4;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        d[v] = __builtin_amdgcn_raw_buffer_load_b32(m.r, at(k, n0 + 4 * c + v), 0, 0);
    }
    st.w[i] = make_uint4(d[0], d[1], d[2], d[3]);
  }
}

// Router workgroups, then one for each token to quantise (int8); all clear the counters and
// O (a token without an expert has no one else to do it).
template <int P, bool VEC>
__global__ __launch_bounds__(kThreads) void few_route_kernel(FewArgs p, int blocks, int i8) {
  using T = typename Kind<P>::T;
  __shared__ __align__(16) float red[kWaves][16][kCols];
  __shared__ uint32_t tops[kWaves];
  const int64_t gid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t all = (int64_t)gridDim.x * kThreads;
  for (int64_t i = gid; i < p.n_words; i += all) p.entry_done[i] = 0;
  const int64_t words = (int64_t)p.S * p.H / (p.out_f32 ? 1 : 2);
  for (int64_t i = gid; i < words; i += all) reinterpret_cast<uint32_t*>(p.O)[i] = 0;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if ((int)blockIdx.x < blocks) {
    const int tiles = (p.E + kCols - 1) / kCols, toks = (p.S + 15) / 16;
    const int b = blockIdx.x, split = uniform(b / (tiles * toks));
    const int tile = uniform(b / toks) - split * tiles, tb = b - (split * tiles + tile) * toks;
    const int n0 = tile * kCols;
    constexpr int STEPS = kRouteRows / kWaves / Kind<P>::STEP;
    const int s0 = (split * kWaves + wave) * STEPS;
    const int steps = (p.H + Kind<P>::STEP - 1) / Kind<P>::STEP;
    const Columns<P> m((const char*)p.Wr, p.H, p.E, n0);
    const int row = 16 * tb + (lane & 15);
    const uint32_t bytes = (uint32_t)p.H * Kind<P>::ES;
    const Rows a = {make_rsrc(p.A, (int64_t)p.S * bytes), row < p.S ? row * bytes : kPastEnd,
                    bytes};
    Step<P> st[STEPS];
    uint4 x[STEPS][Kind<P>::NX];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if constexpr (VEC)
        st[s].load(m, s0 + s, steps);
      else
        load_router<P>(st[s], m, s0 + s, p.H, p.E, n0);
      a.load(s0 + s, x[s]);
    }
    f32x4_t acc[4] = {};
#pragma unroll
    for (int s = 0; s < STEPS; ++s) st[s].compute(x[s], acc);
    const int n = p.S - 16 * tb < 16 ? p.S - 16 * tb : 16;
    put_sums<P>(acc, &red[wave][0][0], n);
    __syncthreads();
    for (int i = threadIdx.x; i < n * kCols; i += kThreads) {
      const int r = i / kCols, c = i % kCols;
      float v = red[0][r][c];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += red[w][r][c];
      if (n0 + c < p.E) p.score[((int64_t)split * p.S + 16 * tb + r) * p.E + n0 + c] = v;
    }
  } else if (i8 && (int)blockIdx.x < blocks + p.S) {
    // a token's codes: every thread reads its values twice (the second time from the caches)
    const int t = blockIdx.x - blocks;
    const T* x = (const T*)p.A + (int64_t)t * p.H;
    uint32_t top = 0;
    for (int c = threadIdx.x; c < p.H / 8; c += kThreads) {
      Pack<T, 8> v;
      v.load(x + c * 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t q = abs_bits(v.get(i));
        top = top > q ? top : q;
      }
    }
    top = wave_max_u32(top);
    if (lane == 0) tops[wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) top = top > tops[i] ? top : tops[i];
    const Quant q(top);
    if (threadIdx.x == 0) p.xs[t] = q.scale;
    for (int c = threadIdx.x; c < p.H / 8; c += kThreads) {
      Pack<T, 8> v;
      v.load(x + c * 8);
      *reinterpret_cast<uint2*>(p.xc + (int64_t)t * p.H + c * 8) =
          make_uint2(q.pack4(v.get(0), v.get(1), v.get(2), v.get(3)),
                     q.pack4(v.get(4), v.get(5), v.get(6), v.get(7)));
    }
  }
}

// Scores of `tokens` tokens from t0 on into g [tokens][E] (LDS): the router's parts in double,
// rounded once, plus the bias. `n` threads; their loads overlap in batches of 4 x 4.
__device__ __forceinline__ void sum_scores(const FewArgs& p, int t0, int tokens, int tid, int n,
                                           float* g) {
  const int64_t step = (int64_t)p.S * p.E;
  const float* part = p.score + (int64_t)t0 * p.E;
  const int all = tokens * p.E;
  for (int i0 = tid; i0 < all; i0 += 4 * n) {
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (int q0 = 0; q0 < p.route_splits; q0 += 4) {
      float v[4][4];
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          v[a][b] = q0 + b < p.route_splits && i0 + a * n < all
                        ? part[(q0 + b) * step + i0 + a * n]
                        : 0.f;
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) s[a] += (double)v[a][b];
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int i = i0 + a * n;
      if (i < all) g[i] = p.bias != nullptr ? (float)s[a] + p.bias[i % p.E] : (float)s[a];
    }
  }
}

// More than kOwnRoute tokens: a workgroup for each.
__global__ __launch_bounds__(256) void few_topk_kernel(FewArgs p) {
  __shared__ float g[1024];
  const int t = blockIdx.x;
  sum_scores(p, t, 1, threadIdx.x, 256, g);
  __syncthreads();
  if (threadIdx.x < 64)
    topk_one(g, p.E, p.k, p.renormalize, p.ids + (int64_t)t * p.k, p.tw + (int64_t)t * p.k,
             threadIdx.x);
}

// ------------------------------------------------------------ experts

// What a workgroup knows of its entry: an expert's matrix and its rows.
struct Work {
  int n;           // rows
  int expert;      // -1: shared
  int count[2];
  int done[16];    // tokens complete
  uint16_t rows[kMaxRows];       // assignments (shared: tokens)
  int ids[kOwnRoute * 32];       // of the tokens that this workgroup has routed for itself
  float tw[kOwnRoute * 32];
};

// Routes where that is this workgroup's to do, and finds entry y's expert and rows; false:
// nothing to do. lds: kOwnRoute x 1024 floats.
__device__ __forceinline__ bool find_work(const FewArgs& p, int y, bool shared, float* lds,
                                          Work& w) {
  const int tid = threadIdx.x;
  if (!p.routed) {
    sum_scores(p, 0, p.S, tid, kThreads, lds);
    __syncthreads();
    const int t = uniform(tid >> 6);
    if (t < p.S)
      topk_one(lds + t * p.E, p.E, p.k, p.renormalize, w.ids + t * p.k, w.tw + t * p.k, tid & 63);
    __syncthreads();
    if (blockIdx.x == 0 && tid < p.F) {
      p.ids[tid] = w.ids[tid];
      p.tw[tid] = w.tw[tid];
    }
  } else if (p.F <= kOwnRoute * 32) {
    if (tid < p.F) {
      w.ids[tid] = p.ids[tid];
      w.tw[tid] = p.tw[tid];
    }
    __syncthreads();
  }
  if (shared) {
    const int n = p.S - 16 * y < 16 ? p.S - 16 * y : 16;
    if (tid < n) w.rows[tid] = (uint16_t)(16 * y + tid);
    if (tid == 0) {
      w.n = n;
      w.expert = -1;
    }
    __syncthreads();
    return true;
  }
  const bool here = p.F <= kOwnRoute * 32;
  const int e = uniform(!p.by_row ? y : here ? w.ids[y] : p.ids[y]);
  if (e < 0 || e >= p.E) return false;
  if (tid == 0) w.count[0] = w.count[1] = 0;
  __syncthreads();
  // in no particular order: rows do not meet in the products
  for (int f = tid; f < p.F; f += kThreads)
    if ((here ? w.ids[f] : p.ids[f]) == e) {
      if (p.by_row && f < y) w.count[1] = 1;  // an earlier entry's
      w.rows[atomicAdd(&w.count[0], 1)] = (uint16_t)f;
    }
  if (tid == 0) w.expert = e;
  __syncthreads();
  if (tid == 0) w.n = w.count[0];
  const bool mine = uniform(w.count[1]) == 0 && uniform(w.count[0]) > 0;
  __syncthreads();
  return mine;
}

__device__ __forceinline__ bool valid_slot(const FewArgs& p, const Work& w, int f) {
  const int id = p.F <= kOwnRoute * 32 ? w.ids[f] : p.ids[f];
  return id >= 0 && id < p.E;
}

// The tokens that this workgroup's entry completes: O_t = sum_j w_tj y_tj (+ the shared row),
// slots without an expert left out. The entry's rows of y are in memory.
__device__ __forceinline__ void combine(const FewArgs& p, Work& w) {
  const int tid = threadIdx.x;
  const int n = uniform(w.n);
  const bool shared = uniform(w.expert) < 0;
  const rsrc_t y = make_rsrc(p.y, (int64_t)(p.F + p.S) * p.H * 4);
  for (int r0 = 0; r0 < n; r0 += 16) {
    if (tid < 16) {
      int t = -1;
      if (r0 + tid < n) {
        const int f = w.rows[r0 + tid], tok = shared ? f : f / p.k;
        int need = p.shared ? 1 : 0;
        for (int j = 0; j < p.k; ++j) need += valid_slot(p, w, tok * p.k + j);
        if (count_up(p.token_done + tok) == need - 1) t = tok;
      }
      w.done[tid] = t;
    }
    __syncthreads();
    for (int i = 0; i < 16; ++i) {
      const int t = uniform(w.done[i]);
      if (t < 0) continue;
      for (int c = tid * 4; c < p.H; c += kThreads * 4) {
        f32x4_t a = {0.f, 0.f, 0.f, 0.f};
        // 8 slots' loads at a time
        for (int j0 = 0; j0 < p.k; j0 += 8) {
          f32x4_t v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[j] = load_shared(
                y, j0 + j < p.k ? (uint32_t)((t * p.k + j0 + j) * p.H + c) * 4 : kPastEnd);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int f = t * p.k + (j0 + j < p.k ? j0 + j : 0);
            const float wt = p.F <= kOwnRoute * 32 ? w.tw[f] : p.tw[f];
            const bool in = j0 + j < p.k && valid_slot(p, w, f);
#pragma unroll
            for (int q = 0; q < 4; ++q) a[q] = in ? a[q] + wt * v[j][q] : a[q];
          }
        }
        if (p.shared) {
          const f32x4_t v = load_shared(y, (uint32_t)((p.F + t) * p.H + c) * 4);
#pragma unroll
          for (int q = 0; q < 4; ++q) a[q] += v[q];
        }
        const float o[4] = {a[0], a[1], a[2], a[3]};
        if (p.out_f32)
          store_n(reinterpret_cast<float*>(p.O) + (int64_t)t * p.H + c, o);
        else
          store_n(reinterpret_cast<bf16_t*>(p.O) + (int64_t)t * p.H + c, o);
      }
    }
    __syncthreads();
  }
}

// This wave's share of K: every shares-th of `steps` steps from `first` on.
template <int P>
__device__ __forceinline__ void stream(const Columns<P>& m, const Rows& a, int first, int shares,
                                       int steps, typename Kind<P>::Acc (&acc)[4]) {
  constexpr int DEPTH = P == kI8 ? 3 : 2;
  constexpr int NX = Kind<P>::NX;
  Step<P> st[DEPTH];
  uint4 x[DEPTH][NX];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) {
    st[d].load(m, first + d * shares, steps);
    a.load(first + d * shares, x[d]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = typename Kind<P>::Acc{};
  for (int s = first; s < steps;) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d, s += shares) {
      st[d].compute(x[d], acc);
      st[d].load(m, s + DEPTH * shares, steps);
      a.load(s + DEPTH * shares, x[d]);
      __builtin_amdgcn_sched_barrier(0);  // the loads go out here, not behind the next step
    }
  }
}

// Workgroup (entry, column group of CG x 64): up and gate of its columns (waves: 2 matrices x CG
// x 4 / CG shares of K), h, and their share of the down product (waves: 64 columns of H).
// Which entry comes first does not matter; a group's neighbours run at about the same time.
template <int P, int CG>
__global__ __launch_bounds__(kThreads, 4) void few_expert_kernel(FewArgs p) {
  using Acc = typename Kind<P>::Acc;
  constexpr int NX = Kind<P>::NX, STEP = Kind<P>::STEP, ES = Kind<P>::ES;
  constexpr int SHARES = 4 / CG, W = CG * kCols;
  constexpr int PITCH = W * ES + 16;  // bytes of a row of h: 16 rows' 16 bytes in all banks
  __shared__ __align__(16) float red[kWaves * 16 * kCols];
  __shared__ __align__(16) char hbuf[16 * PITCH];
  __shared__ Work w;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int64_t routed = (int64_t)p.entries * p.slices;
  const bool shared = blockIdx.x >= routed;
  const int slices = shared ? p.slices_s : p.slices;
  const int b = shared ? (int)(blockIdx.x - routed) : (int)blockIdx.x;
  const int entry = uniform(b / slices), slice = b - entry * slices;
  if (!find_work(p, entry, shared, red, w)) return;
  const int n = uniform(w.n), e = shared ? 0 : uniform(w.expert);
  const int D = shared ? p.Ds : p.D;
  const int64_t size = (int64_t)p.H * D * ES;
  const char* const* mats = shared ? p.ws : p.w;
  const int mat = wave / 4, part = wave % 4;
  const int d0 = slice * W;
  const int steps = (p.H + STEP - 1) / STEP;
  Columns<P> m(mats[mat] + e * size, p.H, D, d0 + part / SHARES * kCols);
  const rsrc_t y = make_rsrc(p.y + (int64_t)slice * (p.F + p.S) * p.H,
                             (int64_t)(p.F + p.S) * p.H * 4);
  for (int r0 = 0; r0 < n; r0 += 16) {
    const int rows = n - r0 < 16 ? n - r0 : 16;
    const int lr = lane & 15, f = lr < rows ? w.rows[r0 + lr] : 0;
    const uint32_t bytes = (uint32_t)p.H * ES;
    const Rows a = {make_rsrc(p.A, (int64_t)p.S * bytes),
                    lr < rows ? (shared ? f : f / p.k) * bytes : kPastEnd, bytes};
    // (the loads' addresses are formed in each round of 16 rows: kept, they spill)
    int zero = 0;
    asm volatile("" : "+v"(m.off));
    asm volatile("" : "+s"(zero));
    Acc acc[4];
    stream<P>(m, a, part % SHARES, SHARES, steps, acc);
    // the down product's steps: 64 columns of H, the group's rows of D in turn
    constexpr int KS = W / STEP;
    const int tiles = (p.H + kCols - 1) / kCols;
    Step<P> st[2];
    auto columns = [&](int tile) {
      return Columns<P>(mats[2] + e * size, D, p.H, tile * kCols, d0 + zero);
    };
    Columns<P> next = columns(wave);
    int nt = wave, nk = 0;
    auto load = [&](Step<P>& to) {
      to.load(next, nt < tiles ? next.off + nk * next.step : kPastEnd);
      if (++nk == KS) {
        nk = 0;
        nt += kWaves;
        if (nt < tiles) next = columns(nt);
      }
    };
    load(st[0]);
    load(st[1]);
    put_sums<P>(acc, red + wave * 16 * kCols, rows);
    __syncthreads();
    // thread: 4 columns of a row; the shares of K in their order
    for (int i = tid; i < rows * (W / 4); i += kThreads) {
      const int r = i / (W / 4), c = i % (W / 4) * 4;
      f32x4_t v[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float* q = red + ((t * 4 + c / kCols * SHARES) * 16 + r) * kCols + c % kCols;
        v[t] = load4(q);
#pragma unroll
        for (int s = 1; s < SHARES; ++s) v[t] += load4(q + s * 16 * kCols);
      }
      float h[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) h[q] = silu_f32(v[0][q]) * v[1][q];
      // in bf16 rounded once, as the layer's h
      store_n(reinterpret_cast<typename Kind<P>::T*>(hbuf + r * PITCH) + c, h);
    }
    __syncthreads();
    const char* hrow = hbuf + lr * PITCH + (lane >> 4) * 16;
    const int g = lane >> 4, c = lane & 15;
    for (int t = wave; t < tiles; t += kWaves) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = Acc{};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint4 x[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i)
          x[i] = *reinterpret_cast<const uint4*>(hrow + (ks * NX + i) * 64);
        if (KS % 2 == 0) {
          st[ks & 1].compute(x, acc);
          load(st[ks & 1]);
        } else {  // one step to a tile: the two in turn by moving
          st[0].compute(x, acc);
          st[0] = st[1];
          load(st[1]);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 4 * g + r, col = t * kCols + 4 * c;
        if (row >= rows || col >= p.H) continue;
        const int at = (shared ? p.F : 0) + w.rows[r0 + row];
        store_shared(y, (uint32_t)(at * p.H + col) * 4,
                     f32x4_t{acc[0][r], acc[1][r], acc[2][r], acc[3][r]});
      }
    }
    if (r0 + 16 < n) __syncthreads();
  }
  // the last of the entry's column groups adds their rows, in order, into the first's
  stores_done();
  if (slices > 1) {
    if (tid == 0) w.count[0] = count_up(p.entry_done + (shared ? p.entries : 0) + entry);
    __syncthreads();
    if (uniform(w.count[0]) != slices - 1) return;
    const uint32_t one = (uint32_t)(p.F + p.S) * p.H * 4;
    const rsrc_t all = make_rsrc(p.y, (int64_t)slices * one);
    const int quads = p.H / 4;
    for (int i = tid; i < n * quads; i += kThreads) {
      const int r = i / quads, c = (i - r * quads) * 4;
      const uint32_t o = (uint32_t)(((shared ? p.F : 0) + w.rows[r]) * p.H + c) * 4;
      f32x4_t a = {0.f, 0.f, 0.f, 0.f};
      for (int s0 = 0; s0 < slices; s0 += 8) {
        f32x4_t v[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
          v[s] = load_shared(all, s0 + s < slices ? o + (s0 + s) * one : kPastEnd);
#pragma unroll
        for (int s = 0; s < 8; ++s) a += v[s];
      }
      store_shared(all, o, a);
    }
    stores_done();
  }
  combine(p, w);
}

// 8-bit weights, up and gate: workgroup (entry, 64 columns), 4 shares of K each.
__global__ __launch_bounds__(kThreads, 4) void few_up_i8_kernel(FewArgs p) {
  __shared__ __align__(16) int red[kWaves * 16 * kCols];
  __shared__ uint32_t tops[16];
  __shared__ Work w;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int64_t routed = (int64_t)p.entries * p.slices;
  const bool shared = blockIdx.x >= routed;
  const int slices = shared ? p.slices_s : p.slices;
  const int b = shared ? (int)(blockIdx.x - routed) : (int)blockIdx.x;
  const int entry = uniform(b / slices), slice = b - entry * slices;
  if (!find_work(p, entry, shared, reinterpret_cast<float*>(red), w)) return;
  const int n = uniform(w.n), e = shared ? 0 : uniform(w.expert);
  const int D = shared ? p.Ds : p.D, d0 = slice * kCols;
  const int64_t size = i8_matrix_bytes(p.H, D), scales = i8_code_bytes(p.H, D);
  const char* const* mats = shared ? p.ws : p.w;
  const Columns<kI8> m(mats[wave / 4] + e * size, p.H, D, d0);
  float* out = shared ? p.h + (int64_t)p.F * p.D : p.h;
  for (int r0 = 0; r0 < n; r0 += 16) {
    const int rows = n - r0 < 16 ? n - r0 : 16;
    const int lr = lane & 15, f = lr < rows ? w.rows[r0 + lr] : 0;
    const Rows a = {make_rsrc(p.xc, (int64_t)p.S * p.H),
                    lr < rows ? (uint32_t)(shared ? f : f / p.k) * p.H : kPastEnd, (uint32_t)p.H};
    if (tid < 16) tops[tid] = 0;
    i32x4_t acc[4];
    stream<kI8>(m, a, wave % 4, 4, (int)i8_tiles_k(p.H), acc);
    put_sums<kI8>(acc, red + wave * 16 * kCols, rows);
    __syncthreads();
    const int r = tid / 16, c = tid % 16 * 4;
    if (r < rows && d0 + c < D) {
      i32x4_t v[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int* q = red + (t * 4 * 16 + r) * kCols + c;
        v[t] = *reinterpret_cast<const i32x4_t*>(q);
#pragma unroll
        for (int s = 1; s < 4; ++s) v[t] += *reinterpret_cast<const i32x4_t*>(q + s * 16 * kCols);
      }
      const int row = w.rows[r0 + r];
      const float x = p.xs[shared ? row : row / p.k];
      const f32x4_t su = load4(reinterpret_cast<const float*>(mats[0] + e * size + scales) + d0 + c);
      const f32x4_t sg = load4(reinterpret_cast<const float*>(mats[1] + e * size + scales) + d0 + c);
      float h[4];
      uint32_t top = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        h[q] = silu_f32((float)v[0][q] * x * su[q]) * ((float)v[1][q] * x * sg[q]);
        const uint32_t bits = abs_bits(h[q]);
        top = top > bits ? top : bits;
      }
      store_n(out + (int64_t)row * D + d0 + c, h);
      atomicMax(&tops[r], top);
    }
    __syncthreads();
    if (tid < rows)
      atomicMax(p.top + (shared ? p.F : 0) + w.rows[r0 + tid], tops[tid]);
  }
}

// 8-bit weights, down: workgroup (entry, 128 columns of H), 2 x 4 shares of D; h's rows are
// quantised on their way.
__global__ __launch_bounds__(kThreads, 4) void few_down_i8_kernel(FewArgs p, int groups) {
  __shared__ __align__(16) int red[kWaves * 16 * kCols];
  __shared__ Work w;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int all = uniform((int)blockIdx.x / groups), group = blockIdx.x - all * groups;
  const bool shared = all >= p.entries;
  const int entry = shared ? all - p.entries : all;
  if (!find_work(p, entry, shared, nullptr, w)) return;
  const int n = uniform(w.n), e = shared ? 0 : uniform(w.expert);
  const int D = shared ? p.Ds : p.D;
  const char* matrix = (shared ? p.ws[2] : p.w[2]) + e * i8_matrix_bytes(D, p.H);
  const int n0 = group * 2 * kCols;
  const Columns<kI8> m(matrix, D, p.H, n0 + wave / 4 * kCols);
  const int steps = (int)i8_tiles_k(D);
  const uint32_t* tops = p.top + (shared ? p.F : 0);
  const float* in = shared ? p.h + (int64_t)p.F * p.D : p.h;
  const rsrc_t y = make_rsrc(p.y + (shared ? (int64_t)p.F * p.H : 0),
                             (int64_t)(shared ? p.S : p.F) * p.H * 4);
  for (int r0 = 0; r0 < n; r0 += 16) {
    const int rows = n - r0 < 16 ? n - r0 : 16;
    const int lr = lane & 15, f = lr < rows ? w.rows[r0 + lr] : 0;
    const uint32_t bytes = (uint32_t)D * 4;
    const QuantRows a = {make_rsrc(in, (int64_t)(shared ? p.S : p.F) * bytes),
                         lr < rows ? f * bytes : kPastEnd, bytes, Quant(lr < rows ? tops[f] : 0)};
    constexpr int DEPTH = 2;
    Step<kI8> st[DEPTH];
    QuantRows::Raw x[DEPTH];
    const int first = wave % 4;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      st[d].load(m, first + d * 4, steps);
      a.load(first + d * 4, x[d]);
    }
    i32x4_t acc[4] = {};
    for (int s = first; s < steps;) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d, s += 4) {
        uint4 codes[1];
        a.codes(x[d], codes);
        st[d].compute(codes, acc);
        st[d].load(m, s + DEPTH * 4, steps);
        a.load(s + DEPTH * 4, x[d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    put_sums<kI8>(acc, red + wave * 16 * kCols, rows);
    __syncthreads();
    const int half = tid / 256, r = tid / 16 % 16, c = tid % 16 * 4;
    const int col = n0 + half * kCols + c;
    if (r < rows && col < p.H) {
      const int* q = red + (half * 4 * 16 + r) * kCols + c;
      i32x4_t v = *reinterpret_cast<const i32x4_t*>(q);
#pragma unroll
      for (int s = 1; s < 4; ++s) v += *reinterpret_cast<const i32x4_t*>(q + s * 16 * kCols);
      const int row = w.rows[r0 + r];
      const float xs = Quant(tops[row]).scale;
      const f32x4_t sw = load4(reinterpret_cast<const float*>(matrix + i8_code_bytes(D, p.H)) + col);
      f32x4_t o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = (float)v[i] * xs * sw[i];
      store_shared(y, (uint32_t)(row * p.H + col) * 4, o);
    }
    if (r0 + 16 < n) __syncthreads();
  }
  stores_done();
  if (groups > 1) {
    if (tid == 0) w.count[0] = count_up(p.entry_done + (shared ? p.entries : 0) + entry);
    __syncthreads();
    if (uniform(w.count[0]) != groups - 1) return;
  }
  combine(p, w);
}

// ------------------------------------------------------------ host

moe_status check_few(const moe_shape* s, bool i8) {
  if (s == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16 && s->dtype != MOE_MXFP8)
    return MOE_ERR_INVALID_ARGUMENT;
  if (s->S < 0 || s->H < 1 || s->D < 1 || s->E < 1 || s->k < 1 || s->k > s->E ||
      s->D_shared < 0 || s->capacity < 0)
    return MOE_ERR_INVALID_ARGUMENT;
  if (s->dtype == MOE_MXFP8 || (i8 && s->dtype != MOE_BF16) || s->capacity != 0 ||
      (s->flags & ~MOE_OUTPUT_F32) != 0)
    return MOE_ERR_UNSUPPORTED;
  const int64_t m = i8 ? 16 : 8;
  if (s->H % m || s->D % m || s->D_shared % m || s->H > kMaxSize || s->D > kMaxSize ||
      s->D_shared > kMaxSize || s->E > 1024 || s->k > 32 || s->S > kMaxTokens)
    return MOE_ERR_UNSUPPORTED;
  const int64_t widest = s->D > s->D_shared ? s->D : s->D_shared;
  const int64_t es = i8 ? 1 : s->dtype == MOE_F32 ? 4 : 2;
  if ((s->H + 64) * (widest + 64) * es >= kMaxMatrix) return MOE_ERR_UNSUPPORTED;
  // the column groups' rows of y, addressed from one base
  const int64_t groups = i8 ? 1 : (widest + kCols - 1) / kCols;
  if (groups * (s->S * s->k + s->S) * s->H * 4 >= kMaxMatrix) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Columns of D to a workgroup: 64 while there are few (at one token every workgroup counts),
// 128 beyond.
int column_group(const moe_shape* s) { return s->S * s->k >= 256 ? 2 : 1; }

struct FewWs {
  size_t words, score, xc, xs, h, y, total;
  int entries, by_row, shared, slices, slices_s, route_splits;
  int token_done, top, n_words;  // ints from words on
};
FewWs few_ws(const moe_shape* s, bool i8) {
  FewWs w = {};
  const int64_t F = s->S * s->k;
  auto up = [](int64_t a, int64_t b) { return (int)((a + b - 1) / b); };
  w.by_row = F <= s->E;
  w.entries = (int)(w.by_row ? F : s->E);
  w.shared = s->D_shared ? up(s->S, 16) : 0;
  const int cols = i8 ? kCols : column_group(s) * kCols;
  w.slices = up(s->D, cols);
  w.slices_s = s->D_shared ? up(s->D_shared, cols) : 0;
  w.route_splits = up(s->H, kRouteRows);
  w.token_done = w.entries + w.shared;
  w.top = w.token_done + (int)s->S;
  w.n_words = w.top + (i8 ? (int)(F + s->S) : 0);
  size_t o = 0;
  auto take = [&](size_t n) {
    const size_t at = o;
    o += ffn_round_up(n, 256);
    return at;
  };
  const int most = w.slices > w.slices_s ? w.slices : w.slices_s;
  w.words = take((size_t)w.n_words * 4);
  w.score = take((size_t)w.route_splits * s->S * s->E * 4);
  w.xc = take(i8 ? (size_t)s->S * s->H : 0);
  w.xs = take(i8 ? (size_t)s->S * 4 : 0);
  w.h = take(i8 ? (size_t)(F * s->D + s->S * s->D_shared) * 4 : 0);
  w.y = take((size_t)(i8 ? 1 : most) * (F + s->S) * s->H * 4);
  w.total = o ? o : 256;
  return w;
}

template <int P>
void launch_experts(const FewArgs& p, int cg, hipStream_t st) {
  const unsigned grid = (unsigned)(p.entries * p.slices + p.shared * p.slices_s);
  if (cg == 1)
    few_expert_kernel<P, 1><<<grid, kThreads, 0, st>>>(p);
  else
    few_expert_kernel<P, 2><<<grid, kThreads, 0, st>>>(p);
}

template <int R>
void launch_route(const FewArgs& p, bool i8, hipStream_t st) {
  const int blocks =
      p.Wr == nullptr ? 0 : p.route_splits * ((p.E + kCols - 1) / kCols) * ((p.S + 15) / 16);
  int grid = blocks + (i8 ? p.S : 0);
  if (grid < 8) grid = 8;
  if (p.E % 8 == 0)
    few_route_kernel<R, true><<<grid, kThreads, 0, st>>>(p, blocks, i8);
  else
    few_route_kernel<R, false><<<grid, kThreads, 0, st>>>(p, blocks, i8);
}

moe_status few_forward(const moe_shape* s, bool i8, const void* A, const void* W_router,
                       const float* bias, const void* const (&w)[3], const void* const (&sw)[3],
                       int32_t* ids, float* tw, void* O, void* workspace, size_t bytes,
                       hipStream_t st) {
  const moe_status bad = check_few(s, i8);
  if (bad != MOE_OK) return bad;
  if (s->S == 0) return MOE_OK;
  if (A == nullptr || w[0] == nullptr || w[1] == nullptr || w[2] == nullptr || ids == nullptr ||
      tw == nullptr || O == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (W_router == nullptr && bias != nullptr) return MOE_ERR_INVALID_ARGUMENT;
  const bool sh = s->D_shared > 0;
  if ((sw[0] != nullptr) != sh || (sw[1] != nullptr) != sh || (sw[2] != nullptr) != sh)
    return MOE_ERR_INVALID_ARGUMENT;
  // with a router the ids and weights are outputs
  const void* in[] = {A, W_router, bias, w[0], w[1], w[2], sw[0], sw[1], sw[2], ids, tw};
  for (int i = 0; i < 11; ++i) {
    if (in[i] != nullptr && (in[i] == O || in[i] == workspace)) return MOE_ERR_INVALID_ARGUMENT;
    if (W_router != nullptr && i < 9 && in[i] != nullptr && (in[i] == ids || in[i] == tw))
      return MOE_ERR_INVALID_ARGUMENT;
  }
  if (O == workspace || (const void*)ids == (const void*)tw) return MOE_ERR_INVALID_ARGUMENT;
  for (const void* q : {A, W_router, w[0], w[1], w[2], sw[0], sw[1], sw[2], (const void*)O,
                        (const void*)workspace})
    if (!ffn_aligned16(q)) return MOE_ERR_UNSUPPORTED;
  for (const void* q : {(const void*)bias, (const void*)ids, (const void*)tw})
    if (reinterpret_cast<uintptr_t>(q) % 4) return MOE_ERR_UNSUPPORTED;
  const FewWs z = few_ws(s, i8);
  if (workspace == nullptr || bytes < z.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  char* ws = (char*)workspace;
  FewArgs p = {};
  p.A = A;
  p.Wr = W_router;
  p.bias = bias;
  for (int i = 0; i < 3; ++i) {
    p.w[i] = (const char*)w[i];
    p.ws[i] = (const char*)sw[i];
  }
  p.ids = ids;
  p.tw = tw;
  p.O = O;
  p.score = (float*)(ws + z.score);
  p.entry_done = (int*)(ws + z.words);
  p.token_done = p.entry_done + z.token_done;
  p.top = (uint32_t*)(p.entry_done + z.top);
  p.n_words = z.n_words;
  p.xc = (int8_t*)(ws + z.xc);
  p.xs = (float*)(ws + z.xs);
  p.h = (float*)(ws + z.h);
  p.y = (float*)(ws + z.y);
  p.S = (int)s->S;
  p.H = (int)s->H;
  p.D = (int)s->D;
  p.Ds = (int)s->D_shared;
  p.E = (int)s->E;
  p.k = (int)s->k;
  p.F = p.S * p.k;
  p.by_row = z.by_row;
  p.entries = z.entries;
  p.shared = z.shared;
  p.slices = z.slices;
  p.slices_s = z.slices_s;
  p.route_splits = z.route_splits;
  p.renormalize = s->renormalize;
  p.out_f32 = s->dtype == MOE_F32 || (s->flags & MOE_OUTPUT_F32) != 0;
  if (s->dtype == MOE_F32)
    launch_route<kF32>(p, i8, st);
  else
    launch_route<kBf16>(p, i8, st);
  p.routed = W_router == nullptr;
  if (W_router != nullptr && p.S > kOwnRoute) {
    few_topk_kernel<<<(unsigned)p.S, 256, 0, st>>>(p);
    p.routed = 1;
  }
  if (i8) {
    few_up_i8_kernel<<<(unsigned)(p.entries * p.slices + p.shared * p.slices_s), kThreads, 0,
                       st>>>(p);
    p.routed = 1;
    const int groups = (p.H + 2 * kCols - 1) / (2 * kCols);
    few_down_i8_kernel<<<(unsigned)((p.entries + p.shared) * groups), kThreads, 0, st>>>(p,
                                                                                         groups);
  } else if (s->dtype == MOE_F32) {
    launch_experts<kF32>(p, column_group(s), st);
  } else {
    launch_experts<kBf16>(p, column_group(s), st);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_few_workspace_bytes(const moe_shape* shape) {
  return check_few(shape, false) == MOE_OK ? few_ws(shape, false).total : 0;
}

extern "C" moe_status moe_few_forward(const moe_shape* shape, const void* A, const void* W_router,
                                      const float* router_bias, const void* W_up,
                                      const void* W_gate, const void* W_down, const void* Ws_up,
                                      const void* Ws_gate, const void* Ws_down, int32_t* topk_ids,
                                      float* topk_weights, void* O, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  return few_forward(shape, false, A, W_router, router_bias, {W_up, W_gate, W_down},
                     {Ws_up, Ws_gate, Ws_down}, topk_ids, topk_weights, O, workspace,
                     workspace_bytes, (hipStream_t)stream);
}

extern "C" size_t moe_few_i8_workspace_bytes(const moe_shape* shape) {
  return check_few(shape, true) == MOE_OK ? few_ws(shape, true).total : 0;
}

extern "C" moe_status moe_few_i8_forward(const moe_shape* shape, const void* A,
                                         const void* W_router, const float* router_bias,
                                         const void* W_up, const void* W_gate,
                                         const void* W_down, const void* Ws_up,
                                         const void* Ws_gate, const void* Ws_down,
                                         int32_t* topk_ids, float* topk_weights, void* O,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  return few_forward(shape, true, A, W_router, router_bias, {W_up, W_gate, W_down},
                     {Ws_up, Ws_gate, Ws_down}, topk_ids, topk_weights, O, workspace,
                     workspace_bytes, (hipStream_t)stream);
}
