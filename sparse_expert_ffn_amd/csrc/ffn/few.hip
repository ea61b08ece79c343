// The whole MoE layer for a few tokens in three launches (include/moe_ffn.h).
//
// Decode is bound by the chosen experts' bytes, and at one token by how many times the
// device has to start and finish something.
//   route   (512 rows of H, 128 experts, 16 tokens)  the router's partial scores; clears what
//           the next launches count with
//   up      (entry, 128 columns of D, part of H)     h = SiLU(a Wu) * (a Wg)
//   down    (entry, 128 or 256 columns of H)         y = h Wd, and O for the tokens that it
//           completes
// An entry is an expert with its rows, or the shared expert with 16 tokens. Up to 8 tokens
// every workgroup of `up` sums the scores and selects the top-k for itself; beyond, a launch
// of its own does it (one workgroup per token), which also lists the experts' rows where
// there are too many assignments for every workgroup to look through.
//
// Within a launch nothing waits: where there are few columns, H is cut in parts, and the last
// of them to arrive adds the sums; the last of a token's entries to arrive at a column
// group of H forms the token's output there.
//
// Fewer launches were slower (one token, 256 experts of 2048 x 768 top-8; 64 tokens): one grid
// of tasks that wait for each other's h, claimed from counters: 87 and 507 us, since a claim,
// a wait or a count is 1 to 2 us of memory latency and there were eight in a row; up and
// down in one workgroup, each adding its columns' share of y: 47 and 440 us, since at one
// token 48 workgroups held all of the down product, and with many the last round of long
// workgroups left the chip half empty.
//
// Weights go from memory into registers and become MFMA operands there (stream.h). 4 waves: up
// or gate, half of H each; or 1 or 2 column tiles of H, a quarter or half of D each (8 waves
// an eighth where there are few workgroups); added through LDS. With 8-bit weights h's row
// scale needs the whole row: the last of an entry's workgroups quantises its rows.
#include "i8.h"
#include "stream.h"
#include "topk.h"

namespace moe {
namespace {

constexpr int64_t kMaxTokens = 128;
constexpr int64_t kMaxSize = 65536;  // H, D, D_shared
constexpr int kMaxRows = (int)kMaxTokens * 32;  // assignments
constexpr int kThreads = 512, kWaves = 8;  // router
constexpr int kExpertThreads = 256;
constexpr int kMaxSplits = 8;        // parts of H
constexpr int kWanted = 512;         // workgroups: as many as the chip holds
constexpr int kRouteRows = 512;      // K rows of a router workgroup, 64 to a wave
constexpr int kOwnRoute = 8;         // tokens that each workgroup routes for itself
constexpr int kOwnList = kOwnRoute * 32;  // assignments up to which it looks for its own rows

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
  int* entry_done;     // [entries + shared] int8: arrived column groups of each 16 rows
  int* split_done;     // [column groups of D][rounds] arrived parts of H
  int* token_done;     // [S][column groups of H] arrived entries
  int* expert_rows;    // [E] rows of each expert in `list` (more than kOwnList assignments)
  int n_words;         // of these
  uint16_t* list;      // [E][F]
  int8_t* xc;          // int8: codes and scales of the tokens
  float* xs;
  char* h;             // [F][D], then [S][Ds] (fp32 with 8-bit weights)
  int8_t* hc;          // int8: its codes and scales
  float* hs;
  char* part;          // [splits][F + S][2][D or Ds]
  float* y;            // [F + S][H]
  int S, H, D, Ds, E, k, F;
  int by_row, entries; // an entry per assignment (the first of its expert), or per expert
  int shared;          // shared entries
  int slices, slices_s;  // column groups of D
  int splits, rounds;  // parts of H; rounds of 16 rows at most
  int blocks;          // workgroups that share an entry's rounds
  int cols;            // column groups of H
  int route_splits, renormalize, out_f32;
  int routed;          // ids and tw are there (given, or by a launch before)
};

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
      const int k = s * 32 + 8 * g + i;
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const uint32_t b = __builtin_amdgcn_raw_buffer_load_b16(m.r, at(k, n0 + 8 * c + v), 0, 0);
        d[v / 2] = v & 1 ? d[v / 2] | b << 16 : b;
      }
    } else {
      const int k = s * 16 + 4 * g + i / 2;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        d[v] = __builtin_amdgcn_raw_buffer_load_b32(m.r, at(k, n0 + 64 * (i & 1) + 4 * c + v), 0,
                                                    0);
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
    uint4 x[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if constexpr (VEC)
        st[s].load(m, s0 + s, steps);
      else
        load_router<P>(st[s], m, s0 + s, p.H, p.E, n0);
      x[s] = a.load(s0 + s, steps);
    }
    f32x4_t acc[8] = {};
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

// A workgroup for each token: more than kOwnRoute tokens are routed here; of more than kOwnList
// assignments the experts' rows are listed, in the order in which they come (rows do not
// meet in the products; every workgroup of the next launches sees the same list).
__global__ __launch_bounds__(256) void few_topk_kernel(FewArgs p) {
  __shared__ float g[1024];
  const int t = blockIdx.x, lane = threadIdx.x;
  int32_t* ids = p.ids + (int64_t)t * p.k;
  if (p.Wr != nullptr) {
    sum_scores(p, t, 1, threadIdx.x, 256, g);
    __syncthreads();
    if (lane < 64)
      topk_one(g, p.E, p.k, p.renormalize, ids, p.tw + (int64_t)t * p.k, lane);
  }
  if (p.F > kOwnList && lane < p.k) {
    const int id = ids[lane];  // this thread's own store, or given
    if (id >= 0 && id < p.E)
      p.list[(int64_t)id * p.F + count_up(p.expert_rows + id)] = (uint16_t)(t * p.k + lane);
  }
}

// ------------------------------------------------------------ experts

// What a workgroup knows of its entry: an expert's matrix and its rows.
struct Work {
  int n;           // rows
  int expert;      // -1: shared
  int count;
  int part[8];
  int done[64];    // tokens complete
  uint16_t rows[kMaxRows];       // assignments (shared: tokens)
  int ids[kOwnList];       // of the tokens that this workgroup has routed for itself
  float tw[kOwnList];
};

// Entry y's expert e (routed first where that is this workgroup's to do); false: there is none.
// lds: kOwnRoute x 1024 floats.
template <int THREADS>
__device__ __forceinline__ bool find_expert(const FewArgs& p, int y, bool shared, float* lds,
                                            Work& w, int& e) {
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  e = 0;
  if (shared) return true;
  if (!p.routed) {
    sum_scores(p, 0, p.S, tid, THREADS, lds);
    __syncthreads();
    for (int t = wave; t < p.S; t += THREADS / 64) {
      float score, top;
      int id;
      topk_select(lds + t * p.E, p.E, p.k, lane, score, id, top);
      if (lane < p.k) w.ids[t * p.k + lane] = id;
    }
    __syncthreads();
    if (blockIdx.x == 0)  // the weights are the next launch's
      for (int t = wave; t < p.S; t += THREADS / 64)
        topk_one(lds + t * p.E, p.E, p.k, p.renormalize, p.ids + t * p.k, p.tw + t * p.k, lane);
  }
  e = p.by_row ? uniform(p.routed ? p.ids[y] : w.ids[y]) : y;
  return e >= 0 && e < p.E;
}

// Its rows; false: there are none, or they are an earlier entry's.
template <int THREADS>
__device__ __forceinline__ bool find_rows(const FewArgs& p, int y, bool shared, int e, Work& w) {
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  static_assert(THREADS >= kOwnList, "a thread for each assignment");
  const bool own = p.F <= kOwnList;
  if (own && p.routed) {
    if (tid < p.F) {
      w.ids[tid] = p.ids[tid];
      w.tw[tid] = p.tw[tid];
    }
    __syncthreads();
  }
  int n;
  if (shared) {
    n = p.S - 16 * y < 16 ? p.S - 16 * y : 16;
    if (tid < n) w.rows[tid] = (uint16_t)(16 * y + tid);
  } else if (own) {
    const bool mine = tid < p.F && w.ids[tid] == e;
    const uint64_t b = __ballot(mine);
    if (lane == 0) w.part[wave] = (int)__popcll(b);
    __syncthreads();
    int at = 0;
    n = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) {
      if (i < wave) at += w.part[i];
      n += w.part[i];
    }
    if (mine) w.rows[at + __popcll(b & ((1ull << lane) - 1))] = (uint16_t)tid;
  } else {
    n = p.expert_rows[e];
    for (int i = tid; i < n; i += THREADS) w.rows[i] = p.list[(int64_t)e * p.F + i];
  }
  n = uniform(n);
  if (tid == 0) {
    w.n = n;
    w.expert = shared ? -1 : e;
  }
  __syncthreads();
  return n > 0 && (shared || !p.by_row || uniform(w.rows[0]) == y);
}

__device__ __forceinline__ bool valid_slot(const FewArgs& p, const Work& w, int f) {
  const int id = p.F <= kOwnList ? w.ids[f] : p.ids[f];
  return id >= 0 && id < p.E;
}

// The tokens whose columns n0 .. + width - 1 this workgroup completes: O_t = sum_j w_tj y_tj (+
// the shared row), slots without an expert left out. Its own rows of y are in memory.
template <int THREADS>
__device__ __forceinline__ void combine(const FewArgs& p, Work& w, int block, int blocks, int group,
                                        int n0, int width) {
  const int tid = threadIdx.x;
  const int n = uniform(w.n);
  const bool shared = uniform(w.expert) < 0;
  const rsrc_t y = make_rsrc(p.y, (int64_t)(p.F + p.S) * p.H * 4);
  const int quads = (p.H - n0 < width ? p.H - n0 : width) / 4;
  // 4 of this workgroup's rounds at a time
  for (int r0 = 16 * block; r0 < n; r0 += 64 * blocks) {
    if (tid < 64) {
      bool last = false;
      int tok = 0;
      const int r = r0 + tid / 16 * 16 * blocks + tid % 16;
      if (r < n) {
        const int f = w.rows[r];
        tok = shared ? f : f / p.k;
        int need = p.shared ? 1 : 0;
        for (int j = 0; j < p.k; ++j) need += valid_slot(p, w, tok * p.k + j);
        last = count_up(p.token_done + tok * p.cols + group) == need - 1;
      }
      const uint64_t b = __ballot(last);
      if (last) w.done[__popcll(b & ((1ull << tid) - 1))] = tok;
      if (tid == 0) w.count = __popcll(b);
    }
    __syncthreads();
    const int all = uniform(w.count) * quads;
    for (int i = tid; i < all; i += THREADS) {
      const int d = i / quads, c = n0 + (i - d * quads) * 4, t = w.done[d];
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
          const float wt = p.F <= kOwnList ? w.tw[f] : p.tw[f];
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
    __syncthreads();
  }
}

// Row f's codes and scale from its fp32 values, by one wave (twice read).
__device__ __forceinline__ void quantize_row(rsrc_t h, uint32_t row, int D, int8_t* codes,
                                             float* scale) {
  const int lane = threadIdx.x & 63;
  uint32_t top = 0;
  for (int c = lane * 4; c < D; c += 256) {
    const f32x4_t v = load_shared(h, row + c * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = abs_bits(v[i]);
      top = top > b ? top : b;
    }
  }
  const Quant q(wave_max_u32(top));
  if (lane == 0) *scale = q.scale;
  for (int c = lane * 4; c < D; c += 256) {
    const f32x4_t v = load_shared(h, row + c * 4);
    *reinterpret_cast<uint32_t*>(codes + c) = q.pack4(v[0], v[1], v[2], v[3]);
  }
}

// Workgroup (entry, columns of D, part of H): waves 2 matrices x 2 shares of K.
template <int P>
__global__ __launch_bounds__(kExpertThreads, 2) void few_up_kernel(FewArgs p) {
  using Val = typename Kind<P>::Val;
  using Acc = typename Kind<P>::Acc;
  constexpr bool I8 = P == kI8;
  // a thread's 4 columns of two rows of a round: rows r1 and r1 + STRIDE
  constexpr int PER_ROW = kCols / 4, N = 16 * PER_ROW / kExpertThreads, STRIDE = 16 / N;
  constexpr int STEP = Kind<P>::STEP, SHARES = 2, HS = P == kBf16 ? 2 : 4;
  __shared__ __align__(16) Val red[4 * 16 * kCols];
  __shared__ Work w;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  // blocks of an entry's rounds (the shared expert's have one) outermost, then entries, their
  // column groups, parts of H
  const int64_t routed = (int64_t)p.blocks * p.entries * p.slices * p.splits;
  const bool shared = blockIdx.x >= routed;
  const int slices = shared ? p.slices_s : p.slices;
  const int b = shared ? (int)(blockIdx.x - routed) : (int)blockIdx.x;
  const int g0 = uniform(b / p.splits), split = b - g0 * p.splits;
  const int e0 = uniform(g0 / slices), d0 = (g0 - e0 * slices) * kCols;
  const int block = shared ? 0 : uniform(e0 / p.entries), entry = e0 - block * p.entries;
  const int blocks = shared ? 1 : p.blocks;
  int e;
  if (!find_expert<kExpertThreads>(p, entry, shared, reinterpret_cast<float*>(red), w, e)) return;
  const int D = shared ? p.Ds : p.D;
  const int64_t size = I8 ? i8_matrix_bytes(p.H, D) : (int64_t)p.H * D * Kind<P>::ES;
  const char* const* mats = shared ? p.ws : p.w;
  const int steps = (p.H + STEP - 1) / STEP, per = uniform((steps + p.splits - 1) / p.splits);
  const int end = (split + 1) * per < steps ? (split + 1) * per : steps;
  Columns<P> m(mats[wave / SHARES] + e * size, p.H, D, d0);
  const int first = split * per + wave % SHARES;
  Stream<P, SHARES> sm;
  sm.start(m, first, end);
  if (!find_rows<kExpertThreads>(p, entry, shared, e, w)) return;
  const int n = uniform(w.n);
  const int base = shared ? p.F : 0;
  const int at = shared ? p.entries * p.slices + g0 : g0 - block * p.entries * p.slices;
  const rsrc_t h = make_rsrc(p.h + (shared ? (int64_t)p.F * p.D * HS : 0),
                             (int64_t)(shared ? p.S : p.F) * D * HS);
  // the shared expert's rows of sums behind the others'
  const int64_t routed_part = (int64_t)p.splits * p.F * 2 * p.D * 4;
  const uint32_t one = (uint32_t)(shared ? p.S : p.F) * 2 * D * 4;
  const rsrc_t part = make_rsrc(p.part + (shared ? routed_part : 0), (int64_t)p.splits * one);
  const int r1 = tid / PER_ROW, c = tid % PER_ROW * 4;
  for (int r0 = 16 * block; r0 < n; r0 += 16 * blocks) {
    const int rows = n - r0 < 16 ? n - r0 : 16;
    const int lr = lane & 15, f = lr < rows ? w.rows[r0 + lr] : 0;
    const uint32_t bytes = (uint32_t)p.H * Kind<P>::ES;
    const Rows a = {make_rsrc(I8 ? (const void*)p.xc : p.A, (int64_t)p.S * bytes),
                    lr < rows ? (shared ? f : f / p.k) * bytes : kPastEnd, bytes};
    asm volatile("" : "+v"(m.off));  // (addresses kept over the rounds spill)
    Acc acc[8];
    if (r0 > 16 * block) sm.start(m, first, end);
    sm.run(m, a, first, end, acc);
    put_sums<P>(acc, red + wave * 16 * kCols, rows);
    __syncthreads();
    // the shares of K in their order, then the parts
    Acc v[N][2];
    uint32_t o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = r1 + i * STRIDE;
      o[i] = kPastEnd;
      v[i][0] = v[i][1] = Acc{};
      if (r >= rows) continue;
      if (d0 + c < D) o[i] = (uint32_t)(w.rows[r0 + r] * 2 * D + d0 + c) * 4;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const Val* q = red + (t * SHARES * 16 + r) * kCols + c;
        v[i][t] = *reinterpret_cast<const Acc*>(q) +
                  *reinterpret_cast<const Acc*>(q + 16 * kCols);
      }
    }
    if (p.splits > 1) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          store_shared(part, o[i] + split * one + t * D * 4,
                       __builtin_bit_cast(f32x4_t, v[i][t]));
      stores_done();
      if (tid == 0) w.count = count_up(p.split_done + at * p.rounds + r0 / 16);
      __syncthreads();
      const bool last = uniform(w.count) == p.splits - 1;
      __syncthreads();
      if (!last) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        Acc q[kMaxSplits][2];
#pragma unroll
        for (int s = 0; s < kMaxSplits; ++s)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            q[s][t] = __builtin_bit_cast(
                Acc, load_shared(part, s < p.splits ? o[i] + s * one + t * D * 4 : kPastEnd));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          v[i][t] = q[0][t];
#pragma unroll
          for (int s = 1; s < kMaxSplits; ++s) v[i][t] += q[s][t];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = r1 + i * STRIDE;
      if (r >= rows || d0 + c >= D) continue;
      const int row = w.rows[r0 + r];
      float u[4], g[4], hv[4];
      if constexpr (I8) {
        const float x = p.xs[shared ? row : row / p.k];
        const int64_t sc = e * size + i8_code_bytes(p.H, D);
        const f32x4_t su = load4(reinterpret_cast<const float*>(mats[0] + sc) + d0 + c);
        const f32x4_t sg = load4(reinterpret_cast<const float*>(mats[1] + sc) + d0 + c);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          u[q] = scaled(v[i][0][q], x, su[q]);
          g[q] = scaled(v[i][1][q], x, sg[q]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) u[q] = v[i][0][q], g[q] = v[i][1][q];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) hv[q] = silu_f32(u[q]) * g[q];
      const int64_t to = (int64_t)row * D + d0 + c;
      // bf16: the down product's operand, rounded once as the layer's h is (2-norm error of O
      // against 64 bits 0.0023 so, 0.0017 from O's own rounding alone)
      if constexpr (P == kBf16)
        store_n(reinterpret_cast<bf16_t*>(p.h) + (shared ? (int64_t)p.F * p.D : 0) + to, hv);
      else
        store_shared(h, (uint32_t)to * 4, f32x4_t{hv[0], hv[1], hv[2], hv[3]});
    }
    if constexpr (I8) {
      // the entry's last column group: codes of its rows
      stores_done();
      if (tid == 0) w.count = count_up(p.entry_done + (shared ? p.entries : 0) + entry);
      __syncthreads();
      const bool last = uniform(w.count) == slices * ((n + 15) / 16) - 1;
      __syncthreads();
      if (last)
        for (int r = wave; r < n; r += 4) {
          const int row = w.rows[r];
          quantize_row(h, (uint32_t)row * D * 4, D,
                       p.hc + (shared ? (int64_t)p.F * p.D : 0) + (int64_t)row * D,
                       p.hs + base + row);
        }
    } else if (r0 + 16 * blocks < n) {
      __syncthreads();
    }
  }
}

// Workgroup (entry, CT column tiles of H): waves CT x SHARES of D.
template <int P, int CT, int SHARES>
__global__ __launch_bounds__(64 * CT * SHARES, 2) void few_down_kernel(FewArgs p) {
  using Val = typename Kind<P>::Val;
  using Acc = typename Kind<P>::Acc;
  constexpr bool I8 = P == kI8;
  constexpr int PER_ROW = kCols / 4;
  constexpr int STEP = Kind<P>::STEP, THREADS = 64 * CT * SHARES;
  constexpr int HS = P == kBf16 ? 2 : P == kF32 ? 4 : 1;  // bytes of the operand
  __shared__ __align__(16) Val red[CT * SHARES * 16 * kCols];
  __shared__ Work w;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int all = uniform((int)blockIdx.x / p.cols), group = blockIdx.x - all * p.cols;
  const bool shared = all >= p.blocks * p.entries;
  const int block = shared ? 0 : uniform(all / p.entries);
  const int entry = all - (shared ? p.blocks : block) * p.entries;
  const int blocks = shared ? 1 : p.blocks;
  int e;
  if (!find_expert<THREADS>(p, entry, shared, nullptr, w, e)) return;
  const int D = shared ? p.Ds : p.D, base = shared ? p.F : 0;
  const int64_t size = I8 ? i8_matrix_bytes(D, p.H) : (int64_t)D * p.H * Kind<P>::ES;
  const char* matrix = (shared ? p.ws[2] : p.w[2]) + e * size;
  const int n0 = group * CT * kCols;
  Columns<P> m(matrix, D, p.H, n0 + wave / SHARES * kCols);
  const int steps = (D + STEP - 1) / STEP;
  Stream<P, SHARES> sm;
  sm.start(m, wave % SHARES, steps);
  if (!find_rows<THREADS>(p, entry, shared, e, w)) return;
  const int n = uniform(w.n);
  const char* in = (I8 ? (const char*)p.hc : p.h) + (shared ? (int64_t)p.F * p.D * HS : 0);
  const uint32_t bytes = (uint32_t)D * HS;
  const rsrc_t y = make_rsrc(p.y, (int64_t)(p.F + p.S) * p.H * 4);
  for (int r0 = 16 * block; r0 < n; r0 += 16 * blocks) {
    const int rows = n - r0 < 16 ? n - r0 : 16;
    const int lr = lane & 15, f = lr < rows ? w.rows[r0 + lr] : 0;
    const Rows a = {make_rsrc(in, (int64_t)(shared ? p.S : p.F) * bytes),
                    lr < rows ? f * bytes : kPastEnd, bytes};
    asm volatile("" : "+v"(m.off));
    Acc acc[8];
    if (r0 > 16 * block) sm.start(m, wave % SHARES, steps);
    sm.run(m, a, wave % SHARES, steps, acc);
    put_sums<P>(acc, red + wave * 16 * kCols, rows);
    __syncthreads();
    for (int i = tid; i < rows * CT * PER_ROW; i += THREADS) {
      const int r = i / (CT * PER_ROW), tile = i / PER_ROW % CT, c = i % PER_ROW * 4;
      const int col = n0 + tile * kCols + c;
      if (col >= p.H) continue;
      const Val* q = red + (tile * SHARES * 16 + r) * kCols + c;
      Acc v = *reinterpret_cast<const Acc*>(q);
#pragma unroll
      for (int s = 1; s < SHARES; ++s) v += *reinterpret_cast<const Acc*>(q + s * 16 * kCols);
      const int row = base + w.rows[r0 + r];
      f32x4_t o;
      if constexpr (I8) {
        const float hs = p.hs[row];
        const f32x4_t sw =
            load4(reinterpret_cast<const float*>(matrix + i8_code_bytes(D, p.H)) + col);
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = scaled(v[q], hs, sw[q]);
      } else {
        o = v;
      }
      store_shared(y, (uint32_t)(row * p.H + col) * 4, o);
    }
    if (r0 + 16 * blocks < n) __syncthreads();
  }
  stores_done();
  combine<THREADS>(p, w, block, blocks, group, n0, CT * kCols);
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
  return MOE_OK;
}

struct FewWs {
  size_t words, list, score, xc, xs, h, hc, hs, part, y, total;
  int entries, by_row, shared, slices, slices_s, splits, rounds, blocks, route_splits,
      tiles, shares, cols;
  int split_done, token_done, expert_rows, n_words;  // ints from words on
};
FewWs few_ws(const moe_shape* s, bool i8) {
  FewWs w = {};
  w.total = 256;
  if (s->S == 0) return w;  // no entries to divide workgroups among
  const int64_t F = s->S * s->k;
  auto up = [](int64_t a, int64_t b) { return (int)((a + b - 1) / b); };
  w.by_row = F <= s->E && F <= kOwnList;
  w.entries = (int)(w.by_row ? F : s->E);
  w.shared = s->D_shared ? up(s->S, 16) : 0;
  w.slices = up(s->D, kCols);
  w.slices_s = s->D_shared ? up(s->D_shared, kCols) : 0;
  w.route_splits = up(s->H, kRouteRows);
  // workgroups that share an expert's rounds of 16 rows where it has several as a rule
  w.blocks = F > 8 * s->E ? (up(s->S, 16) < 8 ? up(s->S, 16) : 8) : 1;
  // H in parts until there are kWanted workgroups (of entries that at least some have)
  const int groups = w.entries * w.slices + w.shared * w.slices_s;
  int64_t splits = kWanted / ((int64_t)groups * w.blocks);
  const int64_t most = up(s->H, 2 * 64);  // two steps of bf16 for each wave
  if (splits > most) splits = most;
  if (splits > kMaxSplits) splits = kMaxSplits;
  w.splits = splits < 1 ? 1 : (int)splits;
  w.rounds = up(F > s->S ? F : s->S, 16);
  // two column tiles of H to a workgroup where that leaves enough of them
  const int64_t all = (int64_t)w.blocks * w.entries + w.shared;
  w.tiles = all * up(s->H, 2 * kCols) >= 1024 ? 2 : 1;
  w.shares = all * up(s->H, kCols) <= 512 ? 8 : 4 / w.tiles;
  w.cols = up(s->H, w.tiles * kCols);
  w.split_done = w.entries + w.shared;
  w.token_done = w.split_done + (w.splits > 1 ? groups * w.rounds : 0);
  w.expert_rows = w.token_done + (int)s->S * w.cols;
  w.n_words = w.expert_rows + (F > kOwnList ? (int)s->E : 0);
  size_t o = 0;
  auto take = [&](size_t n) {
    const size_t at = o;
    o += ffn_round_up(n, 256);
    return at;
  };
  const size_t n_h = (size_t)(F * s->D + s->S * s->D_shared);
  w.words = take((size_t)w.n_words * 4);
  w.list = take(F > kOwnList ? (size_t)(s->E * F) * 2 : 0);
  w.score = take((size_t)w.route_splits * s->S * s->E * 4);
  w.xc = take(i8 ? (size_t)s->S * s->H : 0);
  w.xs = take(i8 ? (size_t)s->S * 4 : 0);
  w.h = take(n_h * (!i8 && s->dtype == MOE_BF16 ? 2 : 4));
  w.hc = take(i8 ? n_h : 0);
  w.hs = take(i8 ? (size_t)(F + s->S) * 4 : 0);
  w.part = take(w.splits > 1 ? n_h * w.splits * 2 * 4 : 0);
  w.y = take((size_t)(F + s->S) * s->H * 4);
  w.total = o;
  return w;
}

template <int P, int CT, int SHARES>
void launch_down(const FewArgs& p, hipStream_t st) {
  const unsigned grid = (unsigned)((p.blocks * p.entries + p.shared) * p.cols);
  few_down_kernel<P, CT, SHARES><<<grid, 64 * CT * SHARES, 0, st>>>(p);
}

template <int P>
void launch_experts(FewArgs p, const FewWs& z, hipStream_t st) {
  const unsigned groups =
      (unsigned)(p.blocks * p.entries * p.slices + p.shared * p.slices_s);
  few_up_kernel<P><<<groups * p.splits, kExpertThreads, 0, st>>>(p);
  p.routed = 1;
  if (z.tiles == 2)
    launch_down<P, 2, 2>(p, st);
  else if (z.shares == 8)
    launch_down<P, 1, 8>(p, st);
  else
    launch_down<P, 1, 4>(p, st);
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

// The launches of a call whose arguments are in order.
hipError_t run_few(const moe_shape* s, bool i8, const FewWs& z, const void* A,
                   const void* W_router, const float* bias, const void* const (&w)[3],
                   const void* const (&sw)[3], int32_t* ids, float* tw, void* O, char* ws,
                   hipStream_t st) {
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
  p.split_done = p.entry_done + z.split_done;
  p.token_done = p.entry_done + z.token_done;
  p.expert_rows = p.entry_done + z.expert_rows;
  p.n_words = z.n_words;
  p.list = (uint16_t*)(ws + z.list);
  p.xc = (int8_t*)(ws + z.xc);
  p.xs = (float*)(ws + z.xs);
  p.h = ws + z.h;
  p.hc = (int8_t*)(ws + z.hc);
  p.hs = (float*)(ws + z.hs);
  p.part = ws + z.part;
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
  p.splits = z.splits;
  p.rounds = z.rounds;
  p.blocks = z.blocks;
  p.cols = z.cols;
  p.route_splits = z.route_splits;
  p.renormalize = s->renormalize;
  p.out_f32 = s->dtype == MOE_F32 || (s->flags & MOE_OUTPUT_F32) != 0;
  if (s->dtype == MOE_F32)
    launch_route<kF32>(p, i8, st);
  else
    launch_route<kBf16>(p, i8, st);
  p.routed = W_router == nullptr || p.S > kOwnRoute;
  if ((W_router != nullptr && p.S > kOwnRoute) || p.F > kOwnList)
    few_topk_kernel<<<(unsigned)p.S, 256, 0, st>>>(p);
  if (i8)
    launch_experts<kI8>(p, z, st);
  else if (s->dtype == MOE_F32)
    launch_experts<kF32>(p, z, st);
  else
    launch_experts<kBf16>(p, z, st);
  return hipGetLastError();
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
  return run_few(s, i8, z, A, W_router, bias, w, sw, ids, tw, O, (char*)workspace, st) ==
                 hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
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
