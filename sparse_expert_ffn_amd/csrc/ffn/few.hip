// The whole MoE layer for a few tokens in two launches (include/moe_ffn.h).
//
// Decode is bound by the chosen experts' bytes, and at one token by how many times the
// device has to start and finish something. The first launch forms the router's partial
// scores (and clears what the second one counts with). The second is one grid that works
// through a list of tasks:
//   route    (token)                 scores summed, top-k; the last one lists the experts
//   upgate   (entry, 128 columns of D, part of K)    h = SiLU(a Wu) * (a Wg)
//   down     (entry, 256 columns of H, part of D)    y = h Wd, a row per (token, slot)
//   combine  (256 columns of H, 8 tokens)            O = sum w y
// An entry is an expert with up to 16 of its rows (one MFMA's); the shared expert has an
// entry for every 16 tokens. A workgroup takes the next task's number from a counter; a
// task waits only for tasks of smaller numbers, which running workgroups hold: no wait
// depends on a workgroup that has not started, whatever else runs on the device. (As a
// guard each wait is bounded all the same, and the first launch fills O with NaN.)
//
// Weights go from memory into registers, 16 bytes per lane, whole rows of 256 bytes, and
// become MFMA operands there: no LDS on their way. A wave streams 128 columns; 4 waves
// share K and add their sums through LDS.
//   bf16: a lane holds 8 rows of 8 columns; 32 byte permutes give the operands of 8
//         columns (8 rows each), one v_mfma_f32_16x16x32_bf16 per column block
//   fp32: 4 rows of 2 x 4 columns, v_mfma_f32_16x16x4_f32 (K in an order that suits)
//   int8: packed in operand order, v_mfma_i32_16x16x64_i8
// The first steps of a down task's weights are on their way before it waits for h.
#include "gemm_direct.h"
#include "i8.h"
#include "topk.h"

namespace moe {
namespace {

using rsrc_t = __amdgpu_buffer_rsrc_t;
constexpr uint32_t kPastEnd = 0x80000000u;  // above every descriptor's range
constexpr int64_t kMaxMatrix = 0x7F000000;
constexpr int kNonTemporal = 2;  // load hint: weights are read once
constexpr int64_t kMaxTokens = 128;
constexpr int64_t kMaxSize = 65536;  // H, D, D_shared
constexpr int kCols = 128;           // columns of a wave
constexpr int kShares = 4;           // waves that share K
constexpr int kThreads = 512;
constexpr int kGrid = 512;           // workgroups of the second launch: two to a CU
constexpr int kMaxSplits = 8;
constexpr int kRouteRows = 256;      // K rows of a router workgroup, 64 to a wave
constexpr uint64_t kWaitTicks = (uint64_t)1 << 28;  // about 2.7 s at 100 MHz

// Control words, cleared by the first launch.
enum { kTicket, kRouted, kPlanned, kGaveUp, kWords = 64 };
// The plan, written by the last route task.
struct FewPlan {
  int routed;      // entries of routed experts
  int splits;      // upgate: parts of K
  int slices;      // down: parts of D
  int slices_s;    // the shared expert's
};
struct Entry {
  int expert;      // -1: shared
  int row0, n;     // its rows in the list (shared: tokens)
  int pad;
};

struct FewArgs {
  const void* A;
  const void* Wr;
  const float* bias;
  const char* w[3];    // up, gate, down
  const char* ws[3];
  int32_t* ids;        // [S][k], written when Wr is given
  float* tw;
  void* O;
  int* words;          // control words, then counters
  int* entry_done;     // [max entries] finished column tiles of h
  int* split_done;     // [kGrid] arrived parts of an upgate tile
  int* tile_done;      // [H / 256] finished down tasks
  uint32_t* top;       // int8: [F + S] abs_bits of the largest h
  int n_words;         // of all of these
  FewPlan* plan;
  Entry* entries;
  int* rows;           // [F] assignments by entry
  float* score;        // [route splits][S][E]
  int8_t* xc;          // int8: codes and scales of the tokens
  float* xs;
  char* part;          // [upgate tasks with splits][2][part_rows][128]
  char* h;             // [F][D]
  char* hs;            // [S][Ds]
  float* y;            // [slices][F + S][H]
  int S, H, D, Ds, E, k, F;
  int t1, t1s, t2;     // column tiles
  int shared;          // shared entries
  int part_rows;       // min(S, 16)
  int max_slices;
  int route_splits, renormalize, out_f32;
};

// A value that is the same in all lanes, in a scalar register (the compiler leaves quotients
// and loaded values in vector ones, and then takes a loop around every descriptor load).
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint64_t u = ((uint64_t)(uint32_t)uniform((int)(a >> 32)) << 32) | (uint32_t)uniform((int)a);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(u), 0, uniform((int)bytes),
                                           0x00020000);
}
__device__ __forceinline__ uint4 load16(rsrc_t r, uint32_t o) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0));
}
__device__ __forceinline__ uint4 load16_once(rsrc_t r, uint32_t o) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, kNonTemporal));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
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
  static constexpr int ES = 2, STEP = 32;  // bytes of a weight, K rows per step
};
template <>
struct Kind<kF32> {
  using T = float;
  using Val = float;
  using Acc = f32x4_t;
  static constexpr int ES = 4, STEP = 16;
};
template <>
struct Kind<kI8> {
  using T = bf16_t;
  using Val = int;
  using Acc = i32x4_t;
  static constexpr int ES = 1, STEP = 64;
};

// 128 columns of a matrix from n0 on: 8 loads per step.
template <int P>
struct Columns {
  rsrc_t r;
  uint32_t off, row, step;
  int steps;

  __device__ __forceinline__ Columns() {}
  __device__ __forceinline__ Columns(int tid, const char* matrix, int K, int N, int n0, bool in) {
    const int lane = tid & 63, c = lane & 15, g = lane >> 4;
    steps = (K + Kind<P>::STEP - 1) / Kind<P>::STEP;
    if constexpr (P == kI8) {
      const uint32_t kt = (uint32_t)i8_tiles_k(K);
      r = make_rsrc(matrix, in ? i8_code_bytes(K, N) : 0);
      off = (uint32_t)(n0 / 16) * kt * 1024 + lane * 16;
      row = kt * 1024;
      step = 1024;
    } else if constexpr (P == kBf16) {
      r = make_rsrc(matrix, in ? (int64_t)K * N * 2 : 0);
      off = n0 + 8 * c < N ? (uint32_t)(8 * g * N + n0 + 8 * c) * 2 : kPastEnd;
      row = (uint32_t)N * 2;
      step = (uint32_t)N * 64;
    } else {
      r = make_rsrc(matrix, in ? (int64_t)K * N * 4 : 0);
      // two halves of 64 columns, which end at N each on their own
      off = (uint32_t)(4 * g * N + n0 + 4 * c) * 4;
      row = (uint32_t)N * 4;
      step = (uint32_t)N * 64;
      past[0] = n0 + 4 * c < N ? 0 : kPastEnd;
      past[1] = n0 + 64 + 4 * c < N ? 0 : kPastEnd;
    }
  }
  uint32_t past[P == kF32 ? 2 : 1];
  __device__ __forceinline__ uint4 load(uint32_t o, int i) const {
    if constexpr (P == kF32)
      return load16_once(r, (o + (i >> 1) * row + (i & 1) * 256) | past[i & 1]);
    else
      return load16_once(r, o + i * row);
  }
};

// 16 rows of the other operand, 64 bytes of each per step (lane l: row l % 16, bytes 16 (l
// / 16) .. + 15); rows that are not there and K values behind the end read as zeros.
struct Rows {
  rsrc_t r;
  uint32_t off;    // of this lane's row
  uint32_t bytes;  // of a row
  __device__ __forceinline__ uint4 load(int tid, int s) const {
    const uint32_t g = (tid & 63) >> 4, at = (uint32_t)s * 64 + g * 16;
    return load16(r, at < bytes ? off + at : kPastEnd);
  }
};

template <int P, bool QUANT>
struct Step {
  using Acc = typename Kind<P>::Acc;
  uint4 w[8];
  uint4 x[QUANT ? 4 : 1];

  __device__ __forceinline__ void load_w(const Columns<P>& m, int s) {
    const uint32_t o = s < m.steps ? m.off + (uint32_t)s * m.step : kPastEnd;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = m.load(o, i);
  }
  // QUANT: rows of fp32, of which the step's 16 values are 64 bytes
  __device__ __forceinline__ void load_x(int tid, const Rows& a, int s) {
    if constexpr (QUANT) {
      const uint32_t g = (tid & 63) >> 4, at = ((uint32_t)s * 64 + g * 16) * 4;
      const uint32_t o = at < a.bytes ? a.off + at : kPastEnd;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = load16(a.r, o + 16 * i);
    } else {
      x[0] = a.load(tid, s);
    }
  }
  __device__ __forceinline__ void compute(Acc (&acc)[8], const Quant& q) const {
    if constexpr (P == kBf16) {
      const bf16x8_t a = __builtin_bit_cast(bf16x8_t, x[0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // column j of the lane's 8: rows 2 i and 2 i + 1 in dword i
        const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
        uint4 b;
        b.x = __builtin_amdgcn_perm(word(w[1], j / 2), word(w[0], j / 2), sel);
        b.y = __builtin_amdgcn_perm(word(w[3], j / 2), word(w[2], j / 2), sel);
        b.z = __builtin_amdgcn_perm(word(w[5], j / 2), word(w[4], j / 2), sel);
        b.w = __builtin_amdgcn_perm(word(w[7], j / 2), word(w[6], j / 2), sel);
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, b),
                                                         acc[j], 0, 0, 0);
      }
    } else if constexpr (P == kF32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(word(x[0], i));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
              a, __uint_as_float(word(w[2 * i + j / 4], j % 4)), acc[j], 0, 0, 0);
      }
    } else {
      i32x4_t a;
      if constexpr (QUANT) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = (int)q.pack4(__uint_as_float(x[i].x), __uint_as_float(x[i].y),
                              __uint_as_float(x[i].z), __uint_as_float(x[i].w));
      } else {
        a = __builtin_bit_cast(i32x4_t, x[0]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, __builtin_bit_cast(i32x4_t, w[j]),
                                                       acc[j], 0, 0, 0);
    }
  }
};

// This lane's sums into LDS as rows of 128 columns: rows 4 (l / 16) .. + 3 below n.
template <int P>
__device__ __forceinline__ void put_sums(int tid, const typename Kind<P>::Acc (&acc)[8],
                                         typename Kind<P>::Val* to, int n) {
  using Acc = typename Kind<P>::Acc;
  const int lane = tid & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (4 * g + r >= n) continue;
    typename Kind<P>::Val* row = to + (4 * g + r) * kCols;
    if constexpr (P == kI8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) row[16 * j + c] = acc[j][r];
    } else {
      const int at0 = P == kBf16 ? 8 * c : 4 * c, at1 = P == kBf16 ? 8 * c + 4 : 64 + 4 * c;
      *reinterpret_cast<Acc*>(row + at0) = Acc{acc[0][r], acc[1][r], acc[2][r], acc[3][r]};
      *reinterpret_cast<Acc*>(row + at1) = Acc{acc[4][r], acc[5][r], acc[6][r], acc[7][r]};
    }
  }
}

// ------------------------------------------------------------ first launch

// E that is no whole number of 16-byte vectors: element by element.
template <int P>
__device__ __forceinline__ void load_router(Step<P, false>& st, const Columns<P>& m, int s, int K,
                                            int N, int n0) {
  constexpr int V = 16 / Kind<P>::ES;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = s * Kind<P>::STEP + (P == kBf16 ? 8 * g + i : 4 * g + i / 2);
    const int n = P == kBf16 ? n0 + 8 * c : n0 + 64 * (i & 1) + 4 * c;
    uint32_t d[4];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t o =
          k < K && n + v < N ? (uint32_t)(k * N + n + v) * Kind<P>::ES : kPastEnd;
      if constexpr (P == kBf16) {
        const uint32_t b = __builtin_amdgcn_raw_buffer_load_b16(m.r, o, 0, 0);
        d[v / 2] = v & 1 ? d[v / 2] | b << 16 : b;
      } else {
        d[v] = __builtin_amdgcn_raw_buffer_load_b32(m.r, o, 0, 0);
      }
    }
    st.w[i] = make_uint4(d[0], d[1], d[2], d[3]);
  }
}

// Router workgroups (256 rows of K, 128 experts, 16 tokens each), then one for each
// token to quantise (int8); all clear the counters and fill O with NaN.
template <int P, bool VEC>
__global__ __launch_bounds__(256) void few_route_kernel(FewArgs p, int blocks, int i8) {
  using T = typename Kind<P>::T;
  __shared__ __align__(16) float red[4][16][kCols];
  __shared__ uint32_t tops[4];
  const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)gridDim.x * 256;
  for (int64_t i = gid; i < p.n_words; i += all) p.words[i] = 0;
  if (p.out_f32)
    for (int64_t i = gid; i < (int64_t)p.S * p.H; i += all)
      reinterpret_cast<uint32_t*>(p.O)[i] = 0x7FC00000u;
  else
    for (int64_t i = gid; i < (int64_t)p.S * p.H / 2; i += all)
      reinterpret_cast<uint32_t*>(p.O)[i] = 0x7FC07FC0u;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if ((int)blockIdx.x < blocks) {
    const int tiles = (p.E + kCols - 1) / kCols, toks = (p.S + 15) / 16;
    const int b = blockIdx.x, split = uniform(b / (tiles * toks));
    const int tile = uniform(b / toks) - split * tiles, tb = b - (split * tiles + tile) * toks;
    const int n0 = tile * kCols;
    constexpr int STEPS = kRouteRows / 4 / Kind<P>::STEP;
    const int s0 = (split * 4 + wave) * STEPS;
    const Columns<P> m(threadIdx.x, (const char*)p.Wr, p.H, p.E, n0, true);
    const int row = 16 * tb + (lane & 15);
    const uint32_t bytes = (uint32_t)p.H * Kind<P>::ES;
    const Rows a = {make_rsrc(p.A, (int64_t)p.S * bytes), row < p.S ? row * bytes : kPastEnd,
                    bytes};
    Step<P, false> st[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if constexpr (VEC)
        st[s].load_w(m, s0 + s);
      else
        load_router<P>(st[s], m, s0 + s, p.H, p.E, n0);
      st[s].load_x(threadIdx.x, a, s0 + s);
    }
    f32x4_t acc[8] = {};
    const Quant none(0);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) st[s].compute(acc, none);
    const int n = p.S - 16 * tb < 16 ? p.S - 16 * tb : 16;
    put_sums<P>(threadIdx.x, acc, &red[wave][0][0], n);
    __syncthreads();
    for (int i = threadIdx.x; i < n * kCols; i += 256) {
      const int r = i / kCols, c = i % kCols;
      if (n0 + c < p.E)
        p.score[((int64_t)split * p.S + 16 * tb + r) * p.E + n0 + c] =
            (red[0][r][c] + red[1][r][c]) + (red[2][r][c] + red[3][r][c]);
    }
  } else if (i8 && (int)blockIdx.x < blocks + p.S) {
    // a token's codes: every thread reads its chunks of 8 values twice (the second time
    // from the caches)
    const int t = blockIdx.x - blocks;
    const T* x = (const T*)p.A + (int64_t)t * p.H;
    uint32_t top = 0;
    for (int c = threadIdx.x; c < p.H / 8; c += 256) {
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
    for (int i = 0; i < 4; ++i) top = top > tops[i] ? top : tops[i];
    const Quant q(top);
    if (threadIdx.x == 0) p.xs[t] = q.scale;
    for (int c = threadIdx.x; c < p.H / 8; c += 256) {
      Pack<T, 8> v;
      v.load(x + c * 8);
      *reinterpret_cast<uint2*>(p.xc + (int64_t)t * p.H + c * 8) =
          make_uint2(q.pack4(v.get(0), v.get(1), v.get(2), v.get(3)),
                     q.pack4(v.get(4), v.get(5), v.get(6), v.get(7)));
    }
  }
}

// ------------------------------------------------------------ second launch

struct Shared {
  int ticket, ok, old;
  int row[16];
  uint32_t top[16];
};

__device__ __forceinline__ Entry entry_at(const FewArgs& p, int i) {
  return Entry{uniform(p.entries[i].expert), uniform(p.entries[i].row0), uniform(p.entries[i].n), 0};
}

// Everything that this workgroup has stored is visible to whoever sees the count (see the
// one-launch kernel of the layer: each wave waits for its stores, one thread releases).
// The count before, in every thread, where `want`.
__device__ __forceinline__ int publish(int tid, int* count, Shared& sh, bool want) {
  wait_vmcnt<0>();
  __syncthreads();
  if (tid == 0) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
    const int old = __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (want) {
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      sh.old = old;
    }
  }
  if (!want) return 0;
  __syncthreads();
  return uniform(sh.old);
}

// Until *count reaches need; false: gave up.
__device__ __forceinline__ bool wait_for(int tid, const int* count, int need, int* words, Shared& sh) {
  if (tid == 0) {
    const uint64_t t0 = wall_clock64();
    int ok = 1;
    while (__hip_atomic_load(count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < need) {
      __builtin_amdgcn_s_sleep(1);
      if (wall_clock64() - t0 > kWaitTicks) {
        __hip_atomic_store(words + kGaveUp, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        ok = 0;
        break;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    sh.ok = ok;
  }
  __syncthreads();
  return uniform(sh.ok) != 0;
}

// One token's scores (the router's parts in double, rounded once, plus the bias) and top-k.
__device__ __forceinline__ void route_token(int tid, const FewArgs& p, int t, char* lds) {
  const int lane = tid & 63;
  float* g = reinterpret_cast<float*>(lds);                  // [E], up to 1024
  // thread (share, expert): shares of the parts where there are fewer experts than threads
  const int cols = p.E < kThreads ? p.E : kThreads, shares = kThreads / cols;
  const int share = tid / cols, col = tid % cols;
  double* sums = reinterpret_cast<double*>(lds + 4096);  // [shares][cols]
  for (int e0 = 0; e0 < p.E; e0 += cols) {
    const int e = e0 + col;
    double s = 0.0;
    if (share < shares && e < p.E)
      for (int q0 = share; q0 < p.route_splits; q0 += 8 * shares) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int q = q0 + i * shares;
          v[i] = q < p.route_splits ? p.score[((int64_t)q * p.S + t) * p.E + e] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s += (double)v[i];
      }
    if (share < shares) sums[share * cols + col] = s;
    __syncthreads();
    if (share == 0 && e < p.E) {
      for (int i = 1; i < shares; ++i) s += sums[i * cols + col];
      g[e] = p.bias != nullptr ? (float)s + p.bias[e] : (float)s;
    }
    __syncthreads();
  }
  if (tid < 64)
    topk_one(g, p.E, p.k, p.renormalize, p.ids + (int64_t)t * p.k, p.tw + (int64_t)t * p.k, lane);
}

// The experts in use, with their rows in blocks of 16, and the split of the products.
template <int P>
__device__ __forceinline__ void list_entries(int tid, const FewArgs& p, char* lds, Shared& sh) {
  int* count = reinterpret_cast<int*>(lds);  // [1024] rows of an expert
  int* first = count + 1024;                 // its first place in the list of rows
  int* block = first + 1024;                 // its first entry
  for (int e = tid; e < p.E; e += kThreads) count[e] = 0;
  __syncthreads();
  for (int f = tid; f < p.F; f += kThreads) {
    const int id = p.ids[f];
    if (id >= 0 && id < p.E) atomicAdd(&count[id], 1);
  }
  __syncthreads();
  if (tid < 64) {
    // lane l: experts l per .. + per - 1
    const int per = (p.E + 63) / 64, e0 = tid * per;
    int rows = 0, blocks = 0;
    for (int i = 0; i < per && e0 + i < p.E; ++i) {
      rows += count[e0 + i];
      blocks += (count[e0 + i] + 15) / 16;
    }
    int r = rows, b = blocks;
    for (int o = 1; o < 64; o *= 2) {
      const int ur = __shfl_up(r, o, 64), ub = __shfl_up(b, o, 64);
      if (tid >= o) {
        r += ur;
        b += ub;
      }
    }
    if (tid == 63) sh.old = b;
    r -= rows;
    b -= blocks;
    for (int i = 0; i < per && e0 + i < p.E; ++i) {
      first[e0 + i] = r;
      block[e0 + i] = b;
      r += count[e0 + i];
      b += (count[e0 + i] + 15) / 16;
    }
  }
  __syncthreads();
  const int routed = uniform(sh.old);
  for (int i = tid; i < p.shared; i += kThreads)
    p.entries[i] = Entry{-1, 16 * i, p.S - 16 * i < 16 ? p.S - 16 * i : 16, 0};
  for (int e = tid; e < p.E; e += kThreads)
    for (int i = 0; i * 16 < count[e]; ++i)
      p.entries[p.shared + block[e] + i] =
          Entry{e, first[e] + 16 * i, count[e] - 16 * i < 16 ? count[e] - 16 * i : 16, 0};
  __syncthreads();
  // the order of an expert's rows does not matter: rows do not meet in the products
  for (int f = tid; f < p.F; f += kThreads) {
    const int id = p.ids[f];
    if (id >= 0 && id < p.E) p.rows[atomicAdd(&first[id], 1)] = f;
  }
  if (tid == 0) {
    // as many parts as there are workgroups for, a step for each wave at least
    auto parts = [](int tiles, int K, int most) {
      const int steps = (K + Kind<P>::STEP - 1) / Kind<P>::STEP;
      int n = tiles ? kGrid / tiles : 1;
      if (n > most) n = most;
      if (n > steps / kShares) n = steps / kShares;
      return n < 1 ? 1 : n;
    };
    FewPlan q;
    q.routed = routed;
    q.splits = parts(routed * p.t1 + p.shared * p.t1s, p.H, kMaxSplits);
    const int tiles = (routed + p.shared) * p.t2;
    q.slices = parts(tiles, p.D, p.max_slices);
    q.slices_s = p.shared ? parts(tiles, p.Ds, p.max_slices) : 1;
    *p.plan = q;
  }
}

// A wave's share of a part [s0, s1) of K: every kShares-th step. `ready` is called after the
// first loads of weights; the rows are loaded after it.
template <int P, bool QUANT, typename Ready, typename RowsOf>
__device__ __forceinline__ bool stream(int tid, const Columns<P>& m, int s0, int s1, int share,
                                       typename Kind<P>::Acc (&acc)[8], Ready ready,
                                       RowsOf rows_of) {
  constexpr int DEPTH = 2;
  Step<P, QUANT> st[DEPTH];
  // a step behind the part's end reads as the one behind the last: zeros
  auto at = [&](int s) { return s < s1 ? s : m.steps + 64; };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) st[d].load_w(m, at(s0 + share + d * kShares));
  if (!ready()) return false;
  Quant q(0);
  const Rows a = rows_of(q);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) st[d].load_x(tid, a, at(s0 + share + d * kShares));
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = typename Kind<P>::Acc{};
  for (int s = s0 + share; s < s1;) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d, s += kShares) {
      st[d].compute(acc, q);
      const int next = at(s + DEPTH * kShares);
      st[d].load_w(m, next);
      st[d].load_x(tid, a, next);
      __builtin_amdgcn_sched_barrier(0);  // the loads go out here, not behind the next step
    }
  }
  return true;
}

template <int P>
__device__ __forceinline__ void store_h(char* to, int64_t o, const float (&v)[4]) {
  if constexpr (P == kBf16)
    store_n(reinterpret_cast<bf16_t*>(to) + o, v);  // rounded once, as the layer's h
  else
    store_n(reinterpret_cast<float*>(to) + o, v);
}

template <int P>
__global__ __launch_bounds__(kThreads, 4) void few_kernel(FewArgs args) {
  using Val = typename Kind<P>::Val;
  using Acc = typename Kind<P>::Acc;
  constexpr bool I8 = P == kI8;
  constexpr int HS = P == kBf16 ? 2 : 4;  // bytes of h
  __shared__ __align__(16) Val red[8 * 16 * kCols];
  __shared__ Shared sh;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int routes = args.Wr != nullptr ? args.S : 1;
  bool planned = false;
  FewPlan plan = {};
  if (threadIdx.x == 0)
    sh.ticket =
        __hip_atomic_fetch_add(args.words + kTicket, 1, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
  for (;;) {
    // what depends on the thread and the sizes is formed again in every task: hoisted out of
    // this loop, the tasks' addresses took twice the registers that there are
    int tid = threadIdx.x, zero = 0;
    asm volatile("" : "+v"(tid));
    asm volatile("" : "+s"(zero));
    FewArgs p = args;
    for (int* n : {&p.S, &p.H, &p.D, &p.Ds, &p.E, &p.k, &p.F, &p.t1, &p.t1s, &p.t2, &p.shared,
                   &p.part_rows})
      *n += zero;
    const int lane = tid & 63;
    __syncthreads();
    const int ticket = uniform(sh.ticket);
    int next = 0;
    if (tid == 0)
      next = __hip_atomic_fetch_add(p.words + kTicket, 1, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT);
    if (ticket < routes) {
      int last = 1;
      if (p.Wr != nullptr) {
        route_token(tid, p, ticket, reinterpret_cast<char*>(red));
        last = publish(tid, p.words + kRouted, sh, true) == routes - 1;
        __syncthreads();
      }
      if (last) {
        list_entries<P>(tid, p, reinterpret_cast<char*>(red), sh);
        publish(tid, p.words + kPlanned, sh, false);
      }
      __syncthreads();
      if (tid == 0) sh.ticket = next;
      continue;
    }
    if (!planned) {
      if (!wait_for(tid, p.words + kPlanned, 1, p.words, sh)) return;
      plan.routed = uniform(p.plan->routed);
      plan.splits = uniform(p.plan->splits);
      plan.slices = uniform(p.plan->slices);
      plan.slices_s = uniform(p.plan->slices_s);
      planned = true;
    }
    int t = ticket - routes;
    const int n1s = p.shared * p.t1s * plan.splits, n1 = n1s + plan.routed * p.t1 * plan.splits;
    const int n2s = p.shared * p.t2 * plan.slices_s;
    const int n2 = n2s + plan.routed * p.t2 * plan.slices;
    const int n3 = p.t2 * ((p.S + 7) / 8);
    if (t < n1) {
      // ------------------------------------------------ up, gate, SwiGLU
      const bool shared = t < n1s;
      const int tiles = shared ? p.t1s : p.t1;
      if (!shared) t -= n1s;
      const int column = uniform(t / plan.splits), split = t - column * plan.splits;
      const int en0 = uniform(column / tiles), tile = column - en0 * tiles;
      const int entry = en0 + (shared ? 0 : p.shared);
      const Entry en = entry_at(p, entry);
      const int N = shared ? p.Ds : p.D, n0 = tile * kCols;
      const int steps = (p.H + Kind<P>::STEP - 1) / Kind<P>::STEP;
      const int per = uniform((steps + plan.splits - 1) / plan.splits);
      const int s0 = split * per, s1 = s0 + per < steps ? s0 + per : steps;
      const int mat = wave / kShares;
      const int64_t size = I8 ? i8_matrix_bytes(p.H, N) : (int64_t)p.H * N * Kind<P>::ES;
      const char* base = (shared ? p.ws[mat] : p.w[mat]) + (shared ? 0 : en.expert) * size;
      const Columns<P> m(tid, base, p.H, N, n0, true);
      if (tid < 16) {
        sh.row[tid] = tid >= en.n ? 0
                              : shared                 ? en.row0 + tid
                                                       : p.rows[en.row0 + tid];
        sh.top[tid] = 0;
      }
      Acc acc[8];
      stream<P, false>(
          tid, m, s0, s1, wave % kShares, acc,
          [&] {
            __syncthreads();
            return true;
          },
          [&](Quant&) {
            const int r = lane & 15, f = sh.row[r];
            const int tok = shared ? f : f / p.k;
            const uint32_t bytes = (uint32_t)p.H * Kind<P>::ES;
            return Rows{make_rsrc(I8 ? (const void*)p.xc : p.A, (int64_t)p.S * bytes),
                        r < en.n ? tok * bytes : kPastEnd, bytes};
          });
      put_sums<P>(tid, acc, red + wave * 16 * kCols, en.n);
      __syncthreads();
      // thread: 4 columns of a row; sums over the waves, then over the parts
      auto finish = [&](int r, int q, const Val (&u)[4], const Val (&g)[4]) {
        if (n0 + 4 * q >= N) return;
        const int f = sh.row[r];
        float v[4], fu[4], fg[4];
        if constexpr (I8) {
          const float x = p.xs[shared ? f : f / p.k];
          const int64_t cb = i8_code_bytes(p.H, N);
          const char* const* w = shared ? p.ws : p.w;
          const int64_t at = (shared ? 0 : en.expert) * size + cb;
          const f32x4_t su = load4(reinterpret_cast<const float*>(w[0] + at) + n0 + 4 * q);
          const f32x4_t sg = load4(reinterpret_cast<const float*>(w[1] + at) + n0 + 4 * q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            fu[i] = (float)u[i] * x * su[i];
            fg[i] = (float)g[i] * x * sg[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) fu[i] = u[i], fg[i] = g[i];
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = silu_f32(fu[i]) * fg[i];
          if constexpr (I8) {
            const uint32_t b = abs_bits(v[i]);
            top = top > b ? top : b;
          }
        }
        store_h<P>(shared ? p.hs : p.h, (int64_t)f * N + n0 + 4 * q, v);
        if constexpr (I8) atomicMax(&sh.top[r], top);
      };
      auto sums = [&](int r, int q, int mt, Val (&v)[4]) {
        const Acc* a = reinterpret_cast<const Acc*>(red + (mt * kShares * 16 + r) * kCols + 4 * q);
        Acc s = a[0];
#pragma unroll
        for (int i = 1; i < kShares; ++i) s += a[i * 16 * kCols / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = s[i];
      };
      bool done = true;
      if (plan.splits == 1) {
        for (int i = tid; i < en.n * 32; i += kThreads) {
          Val u[4], g[4];
          sums(i / 32, i % 32, 0, u);
          sums(i / 32, i % 32, 1, g);
          finish(i / 32, i % 32, u, g);
        }
      } else {
        const int slot = shared ? entry * p.t1s + tile
                                : p.shared * p.t1s + (entry - p.shared) * p.t1 + tile;
        const int64_t one = (int64_t)2 * p.part_rows * kCols;
        Val* part = reinterpret_cast<Val*>(p.part) + (int64_t)slot * plan.splits * one;
        for (int i = tid; i < en.n * 64; i += kThreads) {
          const int mt = i / 32 % 2, r = i / 64, q = i % 32;
          Val v[4];
          sums(r, q, mt, v);
          store_n(part + split * one + (mt * p.part_rows + r) * kCols + 4 * q, v);
        }
        done = publish(tid, p.split_done + slot, sh, true) == plan.splits - 1;
        if (done)
          for (int i = tid; i < en.n * 32; i += kThreads) {
            const int r = i / 32, q = i % 32;
            Acc v[kMaxSplits][2];
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s)
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
                v[s][mt] = s < plan.splits
                               ? *reinterpret_cast<const Acc*>(
                                     part + s * one + (mt * p.part_rows + r) * kCols + 4 * q)
                               : Acc{};
            Val u[4], g[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              u[e] = v[0][0][e];
              g[e] = v[0][1][e];
#pragma unroll
              for (int s = 1; s < kMaxSplits; ++s) {
                u[e] += v[s][0][e];
                g[e] += v[s][1][e];
              }
            }
            finish(r, q, u, g);
          }
      }
      if (done) {
        if constexpr (I8) {
          __syncthreads();
          if (tid < en.n)
            atomicMax(p.top + (shared ? p.F : 0) + sh.row[tid], sh.top[tid]);
        }
        publish(tid, p.entry_done + entry, sh, false);
      }
    } else if (t < n1 + n2) {
      // ------------------------------------------------ down
      t -= n1;
      const bool shared = t < n2s;
      if (!shared) t -= n2s;
      const int slices = shared ? plan.slices_s : plan.slices;
      const int column = uniform(t / slices), slice = t - column * slices;
      const int en0 = uniform(column / p.t2), tile = column - en0 * p.t2;
      const int entry = en0 + (shared ? 0 : p.shared);
      const Entry en = entry_at(p, entry);
      const int K = shared ? p.Ds : p.D, n0 = tile * 2 * kCols + wave / kShares * kCols;
      const int steps = (K + Kind<P>::STEP - 1) / Kind<P>::STEP;
      const int per = uniform((steps + slices - 1) / slices);
      const int s0 = slice * per, s1 = s0 + per < steps ? s0 + per : steps;
      const int64_t size = I8 ? i8_matrix_bytes(K, p.H) : (int64_t)K * p.H * Kind<P>::ES;
      const char* base = (shared ? p.ws[2] : p.w[2]) + (shared ? 0 : en.expert) * size;
      const bool in = n0 < p.H;
      const Columns<P> m(tid, base, K, p.H, in ? n0 : 0, in);
      if (tid < 16)
        sh.row[tid] = tid >= en.n ? 0
                              : shared                 ? en.row0 + tid
                                                       : p.rows[en.row0 + tid];
      Acc acc[8];
      const uint32_t* tops = p.top + (shared ? p.F : 0);
      const bool ok = stream<P, I8>(
          tid, m, s0, s1, wave % kShares, acc,
          [&] {
            return wait_for(tid, p.entry_done + entry, shared ? p.t1s : p.t1, p.words, sh);
          },
          [&](Quant& q) {
            const int r = lane & 15, f = sh.row[r];
            if constexpr (I8) q = Quant(r < en.n ? tops[f] : 0);
            const uint32_t bytes = (uint32_t)K * HS;
            return Rows{make_rsrc(shared ? p.hs : p.h, (int64_t)(shared ? p.S : p.F) * bytes),
                        r < en.n ? f * bytes : kPastEnd, bytes};
          });
      if (!ok) return;
      put_sums<P>(tid, acc, red + wave * 16 * kCols, en.n);
      __syncthreads();
      float* y = p.y + ((int64_t)slice * (p.F + p.S) + (shared ? p.F : 0)) * p.H;
      for (int i = tid; i < en.n * 64; i += kThreads) {
        const int r = i / 64, half = i / 32 % 2, q = i % 32;
        const int n = tile * 2 * kCols + half * kCols + 4 * q;
        if (n >= p.H) continue;
        const Acc* a =
            reinterpret_cast<const Acc*>(red + (half * kShares * 16 + r) * kCols + 4 * q);
        Acc s = a[0];
#pragma unroll
        for (int j = 1; j < kShares; ++j) s += a[j * 16 * kCols / 4];
        float v[4];
        if constexpr (I8) {
          const float x = Quant(tops[sh.row[r]]).scale;
          const f32x4_t sw =
              load4(reinterpret_cast<const float*>(base + i8_code_bytes(K, p.H)) + n);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = (float)s[j] * x * sw[j];
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = s[j];
        }
        store_n(y + (int64_t)sh.row[r] * p.H + n, v);
      }
      publish(tid, p.tile_done + tile, sh, false);
    } else if (t < n1 + n2 + n3) {
      // ------------------------------------------------ combine
      t -= n1 + n2;
      const int group = uniform(t / p.t2), tile = t - group * p.t2, tok = group * 8 + wave;
      if (!wait_for(tid, p.tile_done + tile, plan.routed * plan.slices + p.shared * plan.slices_s,
                    p.words, sh))
        return;
      const int c = tile * 2 * kCols + 4 * lane;
      if (tok < p.S && c < p.H) {
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        const int64_t rows = p.F + p.S;
        auto row = [&](int64_t f, int slices, float w) {
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          const float* y = p.y + f * p.H + c;
          f32x4_t l[kMaxSplits];
#pragma unroll
          for (int s = 0; s < kMaxSplits; ++s)
            l[s] = s < slices ? load4(y + s * rows * p.H) : f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < kMaxSplits; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += l[s][i];
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] += w * v[i];
        };
        for (int j = 0; j < p.k; ++j) {
          const int f = tok * p.k + j, id = p.ids[f];
          if (id >= 0 && id < p.E) row(f, plan.slices, p.tw[f]);
        }
        if (p.shared) row(p.F + tok, plan.slices_s, 1.f);
        if (p.out_f32)
          store_n(reinterpret_cast<float*>(p.O) + (int64_t)tok * p.H + c, a);
        else
          store_n(reinterpret_cast<bf16_t*>(p.O) + (int64_t)tok * p.H + c, a);
      }
    } else {
      return;
    }
    __syncthreads();
    if (tid == 0) sh.ticket = next;
  }
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
  size_t words, plan, entries, rows, score, xc, xs, part, h, hs, y, total;
  int entry_done, split_done, tile_done, top, n_words;  // ints from words on
  int t1, t1s, t2, shared, part_rows, max_slices, route_splits;
};
FewWs few_ws(const moe_shape* s, bool i8) {
  FewWs w = {};
  const int64_t F = s->S * s->k;
  auto up = [](int64_t a, int64_t b) { return (int)((a + b - 1) / b); };
  w.t1 = up(s->D, kCols);
  w.t1s = up(s->D_shared, kCols);
  w.t2 = up(s->H, 2 * kCols);
  w.shared = s->D_shared ? up(s->S, 16) : 0;
  w.part_rows = s->S < 16 ? (int)s->S : 16;
  w.route_splits = up(s->H, kRouteRows);
  // entries at most (an expert's last block may be short), and at least, if every slot has an
  // expert; with fewer the down tasks are split no further
  const int64_t most = F < s->E + F / 16 ? F : s->E + F / 16;
  const int64_t least = up(F, 16) > s->k ? up(F, 16) : s->k;
  int64_t slices = kGrid / ((least + w.shared) * w.t2);
  w.max_slices = (int)(slices < 1 ? 1 : slices > kMaxSplits ? kMaxSplits : slices);
  w.entry_done = kWords;
  w.split_done = w.entry_done + (int)most + w.shared;
  w.tile_done = w.split_done + kGrid;
  w.top = w.tile_done + w.t2;
  w.n_words = w.top + (i8 ? (int)(F + s->S) : 0);
  size_t o = 0;
  auto take = [&](size_t n) {
    const size_t at = o;
    o += ffn_round_up(n, 256);
    return at;
  };
  const size_t hb = !i8 && s->dtype == MOE_BF16 ? 2 : 4;
  w.words = take((size_t)w.n_words * 4);
  w.plan = take(sizeof(FewPlan));
  w.entries = take((size_t)(most + w.shared) * sizeof(Entry));
  w.rows = take((size_t)F * 4);
  w.score = take((size_t)w.route_splits * s->S * s->E * 4);
  w.xc = take(i8 ? (size_t)s->S * s->H : 0);
  w.xs = take(i8 ? (size_t)s->S * 4 : 0);
  w.part = take((size_t)kGrid * 2 * w.part_rows * kCols * 4);
  w.h = take((size_t)F * s->D * hb);
  w.hs = take((size_t)s->S * s->D_shared * hb);
  w.y = take((size_t)w.max_slices * (F + s->S) * s->H * 4);
  w.total = o ? o : 256;
  return w;
}

template <int P, int R>
hipError_t launch_few(const FewArgs& p, bool i8, hipStream_t st) {
  const int blocks =
      p.Wr == nullptr ? 0 : p.route_splits * ((p.E + kCols - 1) / kCols) * ((p.S + 15) / 16);
  int grid = blocks + (i8 ? p.S : 0);
  if (grid == 0) grid = 16;
  constexpr int V = 16 / Kind<R>::ES;
  if (p.E % V == 0)
    few_route_kernel<R, true><<<grid, 256, 0, st>>>(p, blocks, i8);
  else
    few_route_kernel<R, false><<<grid, 256, 0, st>>>(p, blocks, i8);
  few_kernel<P><<<kGrid, kThreads, 0, st>>>(p);
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
  p.words = (int*)(ws + z.words);
  p.entry_done = p.words + z.entry_done;
  p.split_done = p.words + z.split_done;
  p.tile_done = p.words + z.tile_done;
  p.top = (uint32_t*)(p.words + z.top);
  p.n_words = z.n_words;
  p.plan = (FewPlan*)(ws + z.plan);
  p.entries = (Entry*)(ws + z.entries);
  p.rows = (int*)(ws + z.rows);
  p.score = (float*)(ws + z.score);
  p.xc = (int8_t*)(ws + z.xc);
  p.xs = (float*)(ws + z.xs);
  p.part = ws + z.part;
  p.h = ws + z.h;
  p.hs = ws + z.hs;
  p.y = (float*)(ws + z.y);
  p.S = (int)s->S;
  p.H = (int)s->H;
  p.D = (int)s->D;
  p.Ds = (int)s->D_shared;
  p.E = (int)s->E;
  p.k = (int)s->k;
  p.F = p.S * p.k;
  p.t1 = z.t1;
  p.t1s = z.t1s;
  p.t2 = z.t2;
  p.shared = z.shared;
  p.part_rows = z.part_rows;
  p.max_slices = z.max_slices;
  p.route_splits = z.route_splits;
  p.renormalize = s->renormalize;
  p.out_f32 = s->dtype == MOE_F32 || (s->flags & MOE_OUTPUT_F32) != 0;
  const hipError_t e = i8                     ? launch_few<kI8, kBf16>(p, true, st)
                       : s->dtype == MOE_F32 ? launch_few<kF32, kF32>(p, false, st)
                                             : launch_few<kBf16, kBf16>(p, false, st);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
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
