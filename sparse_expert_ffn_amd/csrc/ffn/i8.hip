// Products in 8-bit integers with a scale for each token and channel, and the dense
// gated block in that arithmetic (include/moe_ffn.h).
//
// A row's codes meet a column's in v_mfma_i32_16x16x64_i8, sums are exact in 32 bits and
// scaled once in fp32: twice the operations per MFMA of bf16 and half the bytes.
// Weights are packed once in the MFMA's operand order.
#include "ffn_plan.h"
#include "i8.h"
#include "stream.h"

namespace moe {
namespace {

constexpr int64_t kI8MaxN = 1 << 22;
constexpr int64_t kI8MaxExperts = 1 << 16;

// ------------------------------------------------------------ quantisation

// 16 consecutive values of a row.
template <typename T>
struct Chunk;
template <>
struct Chunk<bf16_t> {
  Pack<bf16_t, 8> v[2];
  __device__ __forceinline__ void load(const bf16_t* p) { v[0].load(p), v[1].load(p + 8); }
  __device__ __forceinline__ float get(int i) const { return v[i / 8].get(i % 8); }
  // abs_bits of the largest magnitude; magnitudes as 16-bit integers, two at a time
  __device__ __forceinline__ uint32_t top() const {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    u16x2_t m = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      m = __builtin_elementwise_max(
          m, __builtin_bit_cast(u16x2_t, v[i / 4].w[i % 4] & 0x7FFF7FFFu));
    return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
  }
};
template <>
struct Chunk<float> {
  Pack<float, 16> v;
  __device__ __forceinline__ void load(const float* p) { v.load(p); }
  __device__ __forceinline__ float get(int i) const { return v.get(i); }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t b = abs_bits(v.get(i));
      m = m > b ? m : b;
    }
    return m;
  }
};

// TPR threads to a row, NC chunks of 16 values each in registers; of a longer row the
// rest is read twice.
template <typename T, int TPR, int NC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void quantize_rows_kernel(
    const T* X, int64_t S, int64_t K, int8_t* codes, float* scales) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  __shared__ uint32_t tops[TPR / 64];
  const int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
  const int lane = threadIdx.x % TPR;
  if (TPR == 64 && row >= S) return;
  const T* x = X + row * K;
  const int chunks = (int)(K / 16);
  Chunk<T> c[NC];
  uint32_t top = 0;
#pragma unroll
  for (int n = 0; n < NC; ++n)
    if (lane + n * TPR < chunks) c[n].load(x + (int64_t)(lane + n * TPR) * 16);
#pragma unroll
  for (int n = 0; n < NC; ++n)
    if (lane + n * TPR < chunks) {
      const uint32_t b = c[n].top();
      top = top > b ? top : b;
    }
  for (int at = lane + NC * TPR; at < chunks; at += TPR) {
    Chunk<T> w;
    w.load(x + (int64_t)at * 16);
    const uint32_t b = w.top();
    top = top > b ? top : b;
  }
  top = wave_max_u32(top);
  if constexpr (TPR > 64) {
    if ((lane & 63) == 0) tops[lane / 64] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) top = top > tops[w] ? top : tops[w];
  }
  const Quant q(top);
  if (lane == 0) scales[row] = q.scale;
  auto put = [&](int at, const Chunk<T>& w) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = w.get(i);
    *reinterpret_cast<uint4*>(codes + row * K + (int64_t)at * 16) = q.pack16(v);
  };
#pragma unroll
  for (int n = 0; n < NC; ++n)
    if (lane + n * TPR < chunks) put(lane + n * TPR, c[n]);
  for (int at = lane + NC * TPR; at < chunks; at += TPR) {
    Chunk<T> w;
    w.load(x + (int64_t)at * 16);
    put(at, w);
  }
}

template <typename T>
void quantize_rows_t(const T* X, int64_t S, int64_t K, int8_t* codes, float* scales,
                     hipStream_t st) {
  if (K <= 64 * 16 * 4)
    quantize_rows_kernel<T, 64, 4><<<(unsigned)((S + 3) / 4), 256, 0, st>>>(X, S, K, codes,
                                                                            scales);
  else if (K <= 256 * 16 * 4)
    quantize_rows_kernel<T, 256, 4><<<(unsigned)S, 256, 0, st>>>(X, S, K, codes, scales);
  else
    quantize_rows_kernel<T, 1024, 2><<<(unsigned)S, 1024, 0, st>>>(X, S, K, codes, scales);
}

// Columns of W [E][K][N]: a workgroup takes 128 columns (16 lanes of 8) of one matrix, its
// 16 lane rows every 16th row; W is read twice, since its maximum comes first. Once per weight:
// 256 matrices of 2048 x 768 bf16 400 us (5.0 TB/s in all), one of 7168 x 2048 470 us, whose 16
// workgroups wait for one load of each lane row after another.
template <typename T>
__global__ __launch_bounds__(256) void quantize_cols_kernel(const T* W, int64_t K, int64_t N,
                                                            int8_t* codes, float* scales) {
  __shared__ uint32_t tops[16][128];
  const int64_t nb = (N + 127) / 128;
  const int64_t e = blockIdx.x / nb, n = blockIdx.x % nb * 128 + threadIdx.x % 16 * 8;
  const int r = threadIdx.x / 16;
  const T* w = W + e * K * N;
  uint32_t top[8] = {};
  if (n < N)
    for (int64_t k = r; k < K; k += 16) {
      Pack<T, 8> v;
      v.load(w + k * N + n);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = abs_bits(v.get(i));
        top[i] = top[i] > b ? top[i] : b;
      }
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) tops[r][threadIdx.x % 16 * 8 + i] = top[i];
  __syncthreads();
  if (n >= N) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    for (int q = 0; q < 16; ++q) {
      const uint32_t b = tops[q][threadIdx.x % 16 * 8 + i];
      top[i] = top[i] > b ? top[i] : b;
    }
  const Quant q[8] = {Quant(top[0]), Quant(top[1]), Quant(top[2]), Quant(top[3]),
                      Quant(top[4]), Quant(top[5]), Quant(top[6]), Quant(top[7])};
  if (r == 0)
#pragma unroll
    for (int i = 0; i < 8; ++i) scales[e * N + n + i] = q[i].scale;
  for (int64_t k = r; k < K; k += 16) {
    Pack<T, 8> v;
    v.load(w + k * N + n);
    uint32_t d[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i / 4] |= ((uint32_t)q[i](v.get(i)) & 255u) << (8 * (i % 4));
    *reinterpret_cast<uint2*>(codes + (e * K + k) * N + n) = make_uint2(d[0], d[1]);
  }
}

// Codes [E][K][N] and scales [E][N] into tiles: a workgroup takes 64 rows by 128 columns (8
// tiles) through LDS. Bound by bytes: 7168 x 2048 7.7 us, 256 x 2048 x 768 169 us (4.8 TB/s).
__global__ __launch_bounds__(256) void i8_pack_kernel(const int8_t* codes, const float* scales,
                                                      int64_t K, int64_t N, char* packed,
                                                      int64_t blocks) {
  constexpr int PITCH = 128 + 4;
  __shared__ __align__(4) uint8_t lds[kI8TileK * PITCH];
  const int64_t nt = i8_tiles_n(N), kt = i8_tiles_k(K), nb = (nt + 7) / 8;
  for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const int64_t kk = blk % kt, cb = blk / kt % nb, e = blk / kt / nb;
    char* matrix = packed + e * i8_matrix_bytes(K, N);
    for (int i = threadIdx.x; i < kI8TileK * 16; i += 256) {
      const int64_t k = kk * kI8TileK + i / 16, n = cb * 128 + i % 16 * 8;
      uint2 v = make_uint2(0, 0);
      if (k < K && n < N) {  // 8 codes of a row whose length is a multiple of 8
        const int8_t* q = codes + (e * K + k) * N + n;
        uint8_t c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = (uint8_t)q[j];
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
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v |= (uint32_t)lds[(16 * q + 4 * i + j) * PITCH + t * 16 + c] << (8 * j);
        w[i] = v;
      }
      *reinterpret_cast<uint4*>(matrix + (ct * kt + kk) * 1024 + lane * 16) =
          make_uint4(w[0], w[1], w[2], w[3]);
      if (kk == 0 && lane < kI8TileN) {
        const int64_t n = ct * kI8TileN + lane;
        reinterpret_cast<float*>(matrix + i8_code_bytes(K, N))[n] =
            n < N ? scales[e * N + n] : 0.f;
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ products

// Y = sum * (row scale) * (column scale), rounded once from fp32.
template <typename T>
struct EpI8Store {
  T* out;
  const float *sx, *sw;
  int64_t ld;
  template <int W>
  struct Pre {
    float x, w[W];
  };
  template <int W>
  __device__ __forceinline__ void pre(int64_t m, int64_t n, Pre<W>& p) const {
    p.x = sx[m];
#pragma unroll
    for (int r = 0; r < W; r += 4)
      *reinterpret_cast<f32x4_t*>(p.w + r) = load4(sw + n + r);
  }
  template <int W>
  __device__ __forceinline__ void operator()(int64_t m, int64_t n, const int (&a)[W],
                                             const int (&)[W], const Pre<W>& p) const {
    float v[W];
#pragma unroll
    for (int r = 0; r < W; ++r) v[r] = scaled(a[r], p.x, p.w[r]);
    store_n(out + m * ld + n, v);
  }
};

// h = SiLU(u) g in fp32: it is quantised by its rows next, and a rounding to bf16 before
// would move one code in a hundred.
struct EpI8Swiglu {
  float* h;
  const float *sx, *su, *sg;
  int64_t ld;
  template <int W>
  struct Pre {
    float x, u[W], g[W];
  };
  template <int W>
  __device__ __forceinline__ void pre(int64_t m, int64_t n, Pre<W>& p) const {
    p.x = sx[m];
#pragma unroll
    for (int r = 0; r < W; r += 4) {
      *reinterpret_cast<f32x4_t*>(p.u + r) = load4(su + n + r);
      *reinterpret_cast<f32x4_t*>(p.g + r) = load4(sg + n + r);
    }
  }
  template <int W>
  __device__ __forceinline__ void operator()(int64_t m, int64_t n, const int (&a)[W],
                                             const int (&b)[W], const Pre<W>& p) const {
    float v[W];
    values(a, b, p, v);
    store_n(h + m * ld + n, v);
  }
  template <int W>
  __device__ __forceinline__ static void values(const int (&a)[W], const int (&b)[W],
                                                const Pre<W>& p, float (&v)[W]) {
#pragma unroll
    for (int r = 0; r < W; ++r)
      v[r] = silu_f32(scaled(a[r], p.x, p.u[r])) * scaled(b[r], p.x, p.g[r]);
  }
};

// Where K was split: a workgroup adds a row's sums, forms h and quantises it at once (as a join
// and the rows' quantisation of their own 8.7 us at 64 x 2048). D up to kJoinCols.
constexpr int kJoinCols = 8192;
__global__ __launch_bounds__(512) void i8_join_kernel(GemmArgs g, EpI8Swiglu ep, int8_t* codes,
                                                      float* scales) {
  constexpr int NC = kJoinCols / 4 / 512;
  __shared__ uint32_t tops[8];
  const int64_t m = blockIdx.x, panel = g.M * g.N;
  const int* part = reinterpret_cast<const int*>(g.part) + m * g.N;
  float h[NC][4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int n = (i * 512 + (int)threadIdx.x) * 4;
    if (n >= g.N) continue;
    EpI8Swiglu::Pre<4> pre;
    ep.pre(m, n, pre);
    int v[2][4] = {};
    for (int s = 0; s < g.splits; s += 4) {
      i32x4_t w[4][2];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int p = 0; p < 2; ++p)
          w[e][p] = s + e < g.splits ? *reinterpret_cast<const i32x4_t*>(
                                           part + ((s + e) * 2 + p) * panel + n)
                                     : i32x4_t{};
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[p][r] += w[e][p][r];
    }
    ep.values(v[0], v[1], pre, h[i]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t b = abs_bits(h[i][r]);
      top = top > b ? top : b;
    }
  }
  top = wave_max_u32(top);
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x / 64] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = top > tops[w] ? top : tops[w];
  const Quant q(top);
  if (threadIdx.x == 0) scales[m] = q.scale;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int n = (i * 512 + (int)threadIdx.x) * 4;
    if (n < g.N)
      *reinterpret_cast<uint32_t*>(codes + m * g.N + n) =
          q.pack4(h[i][0], h[i][1], h[i][2], h[i][3]);
  }
}

template <bool DUAL, typename EP>
void launch_i8(const GemmPlan& p, const GemmArgs& g, const EP& ep, hipStream_t st,
               bool join) {
  constexpr int NP = DUAL ? 2 : 1;
  using T = int8_t;
  if (p.tile == 0)
    launch_tile<TileCore<T, 256, 256, 2, DUAL, true, true, 2, 4, 2>>(g, ep, st, join);
  else if (p.tile == 1)
    launch_tile<TileCore<T, 128, 128, NP, DUAL, true, true, 2, 4, 2>>(g, ep, st, join);
  else if (p.tile == 4)
    launch_tile<TileCore<T, 256, 128, NP, DUAL, true, true, 4, 2, 3>>(g, ep, st, join);
  else if (p.tile == 2 && p.tiles_m == 1)
    launch_tile<TileCore<T, 64, 128, NP, DUAL, true, true, 2, 4, 3, true>>(g, ep, st, join);
  else if (p.tile == 2)
    launch_tile<TileCore<T, 64, 128, NP, DUAL, true, true, 2, 4, 3>>(g, ep, st, join);
  else if (p.tiles_m == 1)
    launch_tile<TileCore<T, 16, 128, NP, DUAL, true, true, 1, 4, 4, true>>(g, ep, st, join);
  else
    launch_tile<TileCore<T, 16, 128, NP, DUAL, true, true, 1, 4, 4>>(g, ep, st, join);
}

// Up to 16 rows in one launch, quantisation included: a workgroup of 8 waves takes 16 columns,
// an eighth of K to each wave. The weight's first loads go out before the rows are read;
// every workgroup quantises the rows for itself into LDS. One row of 7168 x 2048 8.1 us in a
// row, 6.6 of them the kernel's: its latency (quantised by a launch of its own and split over
// K with an arrival count, 14). 16 waves are as fast with one workgroup to a CU (8.3), slower
// with more (13 x 2064 x 5128: 9.7 and 12.7 us).
constexpr int kFewRows = 16;
constexpr int64_t kFewCodes = 128 * 1024;  // bytes of LDS for the rows' codes
struct FewRows {
  const void* X;
  const float* sx;  // given: X holds codes
  const char* W;
  void* Y;
  int S, K, N;
  int per_row;      // waves that quantise a row
};

constexpr int kFewWaves = 8;
template <typename T, typename OUT>
__global__ __launch_bounds__(64 * kFewWaves) void i8_few_kernel(FewRows p) {
  constexpr int DEPTH = 8, WAVES = kFewWaves, THREADS = 64 * WAVES;
  constexpr int NC = 4;  // chunks of a row that a thread keeps between its two passes
  extern __shared__ __align__(16) char codes[];  // [S][K + 16]
  __shared__ __align__(16) int red[WAVES * 16 * 16];
  __shared__ uint32_t tops[WAVES];
  __shared__ float scales[kFewRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int kt = (int)i8_tiles_k(p.K), pitch = p.K + 16, n0 = blockIdx.x * kI8TileN;
  const rsrc_t w = make_rsrc(p.W + (int64_t)blockIdx.x * kt * 1024, (int64_t)kt * 1024);
  auto load = [&](int s) {  // past the last tile: zeros
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                         w, s < kt ? (uint32_t)s * 1024 + lane * 16 : kPastEnd, 0,
                                         kNonTemporal));
  };
  uint4 st[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) st[d] = load(wave + d * WAVES);
  const int chunks = p.K / 16;
  if (p.sx != nullptr) {
    const char* x = (const char*)p.X;
    for (int i = tid; i < p.S * chunks; i += THREADS) {
      const int r = i / chunks, c = i - r * chunks;
      *reinterpret_cast<uint4*>(codes + r * pitch + c * 16) =
          *reinterpret_cast<const uint4*>(x + (int64_t)i * 16);
    }
    if (tid < p.S) scales[tid] = p.sx[tid];
  } else {
    const int stride = p.per_row * 64, c0 = wave % p.per_row * 64 + lane;
    for (int r0 = 0; r0 < p.S; r0 += WAVES / p.per_row) {
      const int row = r0 + wave / p.per_row;
      const bool in = row < p.S;
      const T* x = (const T*)p.X + (int64_t)row * p.K;
      Chunk<T> keep[NC];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (in && c0 + i * stride < chunks) keep[i].load(x + (c0 + i * stride) * 16);
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (in && c0 + i * stride < chunks) {
          const uint32_t b = keep[i].top();
          top = top > b ? top : b;
        }
      if (in)
        for (int c = c0 + NC * stride; c < chunks; c += stride) {
          Chunk<T> v;
          v.load(x + c * 16);
          const uint32_t b = v.top();
          top = top > b ? top : b;
        }
      top = wave_max_u32(top);
      if (p.per_row > 1) {
        if (lane == 0) tops[wave] = top;
        __syncthreads();
        for (int i = 0; i < p.per_row; ++i) {
          const uint32_t b = tops[wave / p.per_row * p.per_row + i];
          top = top > b ? top : b;
        }
      }
      const Quant q(top);
      auto put = [&](const Chunk<T>& v, int c) {
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = v.get(i);
        *reinterpret_cast<uint4*>(codes + row * pitch + c * 16) = q.pack16(f);
      };
      if (in) {
        if (c0 == 0) scales[row] = q.scale;
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (c0 + i * stride < chunks) put(keep[i], c0 + i * stride);
        for (int c = c0 + NC * stride; c < chunks; c += stride) {  // from the caches
          Chunk<T> v;
          v.load(x + c * 16);
          put(v, c);
        }
      }
      if (p.per_row > 1) __syncthreads();
    }
  }
  __syncthreads();
  // rows that are not there take row 0's codes: their sums are not read. K values behind the
  // end meet weights of zero
  const int lr = lane & 15, g = lane >> 4;
  const char* xr = codes + (lr < p.S ? lr : 0) * pitch + g * 16;
  i32x4_t acc = {0, 0, 0, 0};
  for (int s = wave; s < kt;) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d, s += WAVES) {
      if (s < kt) {
        const int at = s * 64 + g * 16 < p.K ? s * 64 : 0;
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
            *reinterpret_cast<const i32x4_t*>(xr + at), __builtin_bit_cast(i32x4_t, st[d]), acc,
            0, 0, 0);
      }
      st[d] = load(s + DEPTH * WAVES);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) red[(wave * 16 + 4 * g + r) * 16 + lr] = acc[r];
  __syncthreads();
  const int r = tid / 16, n = n0 + tid % 16;
  if (tid >= 256 || r >= p.S || n >= p.N) return;
  int sum = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) sum += red[i * 256 + tid];
  const float* sw = reinterpret_cast<const float*>(p.W + i8_code_bytes(p.K, p.N));
  const float y = scaled(sum, scales[r], sw[n]);
  reinterpret_cast<OUT*>(p.Y)[(int64_t)r * p.N + n] = from_f32<OUT>(y);
}

// Against the tiles with the rows' quantisation before them: 1 x 7168 x 2048 8.4 and 16.4 us, 16
// rows 13.7 and 16.7; 1 x 768 x 16384 9.6 and 12.3; 16 x 8192 x 8192 21.5 and 21.7; but 16 x
// 768 x 16384 13.5 and 12.4: each workgroup quantises all rows.
bool few_rows(int64_t S, int64_t K, int64_t N) {
  return S <= kFewRows && S * (K + 16) <= kFewCodes && S * i8_tiles_n(N) <= 8192;
}

template <typename T, typename OUT>
hipError_t launch_few_rows(FewRows p, hipStream_t st) {
  p.per_row = kFewWaves;
  while (p.per_row > 1 && p.per_row * p.S > kFewWaves) p.per_row /= 2;
  const size_t lds = (size_t)p.S * (p.K + 16);
  if (lds > 48 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void*>(i8_few_kernel<T, OUT>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)kFewCodes);
    if (e != hipSuccess) return e;
  }
  i8_few_kernel<T, OUT><<<(unsigned)i8_tiles_n(p.N), 64 * kFewWaves, lds, st>>>(p);
  return hipGetLastError();
}

const float* scales_of(const void* W, int64_t K, int64_t N) {
  return reinterpret_cast<const float*>((const char*)W + i8_code_bytes(K, N));
}

// A product of rows of codes with one packed matrix, or two (DUAL); returns its arguments.
template <bool DUAL, typename EP>
GemmArgs run_i8(const GemmPlan& p, int64_t M, int64_t K, int64_t N, const int8_t* X,
                const void* W0, const void* W1, const EP& ep, void* part, hipStream_t st,
                bool join = true) {
  GemmArgs g = {};
  g.A[0] = X;
  g.B[0][0] = W0;
  g.B[0][1] = W1;
  g.lda = K;
  g.ldb = i8_tiles_k(K);
  g.M = M;
  g.N = N;
  g.K[0] = K;
  g.pairs = 1;
  apply_plan(p, &g, part);
  launch_i8<DUAL>(p, g, ep, st, join);
  return g;
}

GemmPlan plan_i8(bool dual, int64_t M, int64_t N, int64_t K) {
  return plan_gemm(kPlanI8, 31u, dual, M, N, K, 1);
}

struct MatmulWs {
  GemmPlan p;
  bool few;
  size_t codes, scales, part, total;
};
MatmulWs matmul_ws(int64_t S, int64_t K, int64_t N) {
  MatmulWs w = {};
  w.few = few_rows(S, K, N);
  w.total = 256;
  if (w.few) return w;
  w.p = plan_i8(false, S, N, K);
  w.scales = ffn_round_up((size_t)S * K, 256);
  w.part = w.scales + ffn_round_up((size_t)S * 4, 256);
  w.total = w.part + ffn_round_up(w.p.part_bytes, 256);
  return w;
}

struct FfnWs {
  GemmPlan up, down;
  size_t xc, xs, h, hc, hs, part, total;
};
FfnWs ffn_ws(const moe_ffn_shape* s) {
  FfnWs w = {};
  w.up = plan_i8(true, s->S, s->D, s->H);
  w.down = plan_i8(false, s->S, s->H, s->D);
  size_t o = 0;
  auto take = [&](size_t n) {
    const size_t at = o;
    o += ffn_round_up(n, 256);
    return at;
  };
  const size_t S = (size_t)s->S;
  w.xc = take(S * s->H);
  w.xs = take(S * 4);
  w.h = take(S * s->D * 4);
  w.hc = take(S * s->D);
  w.hs = take(S * 4);
  w.part = take(w.up.part_bytes > w.down.part_bytes ? w.up.part_bytes : w.down.part_bytes);
  w.total = o ? o : 256;
  return w;
}

moe_status check_matrix(int64_t E, int64_t K, int64_t N) {
  if (E < 1 || K < 1 || N < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (K % 16 || N % 8 || K > kI8MaxK || N >= kI8MaxN || E > kI8MaxExperts)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Rows and columns of a product: every tile's launch stays below 2^32 threads, as check_ffn's.
moe_status check_rows(int64_t S, int64_t N) {
  if (S < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (S >= INT32_MAX - 256 || (S + 63) / 64 * (N / 64 + 1) >= (1 << 23))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A launch of up to 1024 threads per row, below 2^32 in all.
bool rows_fit(int64_t S, int64_t K) {
  return K <= 64 * 64 ? S < (1 << 26) - 4 : K <= 256 * 64 ? S < 1 << 24 : S < 1 << 22;
}

moe_status check_i8_ffn(const moe_ffn_shape* s) {
  if (s == nullptr || s->S < 0 || s->H < 1 || s->D < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16 && s->dtype != MOE_MXFP8)
    return MOE_ERR_INVALID_ARGUMENT;
  if (s->flags & ~MOE_OUTPUT_F32) return MOE_ERR_INVALID_ARGUMENT;
  if (s->dtype == MOE_MXFP8 || s->H % 16 || s->D % 16 || s->H > kI8MaxK || s->D > kI8MaxK)
    return MOE_ERR_UNSUPPORTED;
  const moe_status st = check_rows(s->S, s->H > s->D ? s->H : s->D);
  if (st != MOE_OK) return st;
  return rows_fit(s->S, s->H) && rows_fit(s->S, s->D) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

moe_status enqueued() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

}  // namespace

hipError_t launch_quantize_rows(const void* X, int64_t S, int64_t K, bool f32, int8_t* codes,
                                float* scales, hipStream_t st) {
  if (f32)
    quantize_rows_t((const float*)X, S, K, codes, scales, st);
  else
    quantize_rows_t((const bf16_t*)X, S, K, codes, scales, st);
  return hipGetLastError();
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_i8_weight_bytes(int64_t E, int64_t K, int64_t N) {
  return check_matrix(E, K, N) == MOE_OK ? (size_t)E * i8_matrix_bytes(K, N) : 0;
}

extern "C" moe_status moe_quantize_i8(const void* W, int64_t E, int64_t K, int64_t N,
                                      int32_t dtype, int8_t* codes, float* scales,
                                      void* stream) {
  const moe_status st = check_matrix(E, K, N);
  if (st != MOE_OK) return st;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (W == nullptr || codes == nullptr || scales == nullptr || ffn_shared({codes, scales}, {W}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!ffn_aligned16(W) || !ffn_aligned16(codes) || !aligned4(scales)) return MOE_ERR_UNSUPPORTED;
  const int64_t grid = E * ((N + 127) / 128);
  if (grid >= 1 << 24) return MOE_ERR_UNSUPPORTED;
  if (dtype == MOE_F32)
    quantize_cols_kernel<<<(unsigned)grid, 256, 0, (hipStream_t)stream>>>((const float*)W, K, N,
                                                                          codes, scales);
  else
    quantize_cols_kernel<<<(unsigned)grid, 256, 0, (hipStream_t)stream>>>((const bf16_t*)W, K, N,
                                                                          codes, scales);
  return enqueued();
}

extern "C" moe_status moe_pack_i8_weights(const int8_t* codes, const float* scales, int64_t E,
                                          int64_t K, int64_t N, void* packed, void* stream) {
  const moe_status st = check_matrix(E, K, N);
  if (st != MOE_OK) return st;
  if (codes == nullptr || scales == nullptr || packed == nullptr ||
      ffn_shared({packed}, {codes, scales}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!ffn_aligned16(packed) || !aligned4(scales)) return MOE_ERR_UNSUPPORTED;
  const int64_t blocks = E * ((i8_tiles_n(N) + 7) / 8) * i8_tiles_k(K);
  i8_pack_kernel<<<(unsigned)(blocks < (1 << 20) ? blocks : 1 << 20), 256, 0,
                   (hipStream_t)stream>>>(codes, scales, K, N, (char*)packed, blocks);
  return enqueued();
}

extern "C" moe_status moe_quantize_i8_rows(const void* X, int64_t S, int64_t K, int32_t dtype,
                                           int8_t* codes, float* scales, void* stream) {
  if (S < 0 || K < 1 || (dtype != MOE_F32 && dtype != MOE_BF16)) return MOE_ERR_INVALID_ARGUMENT;
  if (K % 16 || K > kI8MaxK || !rows_fit(S, K)) return MOE_ERR_UNSUPPORTED;
  if (S == 0) return MOE_OK;
  if (X == nullptr || codes == nullptr || scales == nullptr || ffn_shared({codes, scales}, {X}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!ffn_aligned16(X) || !ffn_aligned16(codes) || !aligned4(scales)) return MOE_ERR_UNSUPPORTED;
  return launch_quantize_rows(X, S, K, dtype == MOE_F32, codes, scales,
                              (hipStream_t)stream) == hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}

extern "C" size_t moe_i8_matmul_workspace_bytes(int64_t S, int64_t K, int64_t N) {
  if (check_matrix(1, K, N) != MOE_OK || check_rows(S, N) != MOE_OK || !rows_fit(S, K)) return 0;
  return matmul_ws(S, K, N).total;
}

extern "C" moe_status moe_i8_matmul(int64_t S, int64_t K, int64_t N, int32_t dtype,
                                    int32_t flags, const void* X, const float* row_scales,
                                    const void* W, void* Y, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (flags & ~MOE_OUTPUT_F32) return MOE_ERR_INVALID_ARGUMENT;
  moe_status st = check_matrix(1, K, N);
  if (st == MOE_OK) st = check_rows(S, N);
  if (st == MOE_OK && !rows_fit(S, K)) st = MOE_ERR_UNSUPPORTED;
  if (st != MOE_OK) return st;
  if (S == 0) return MOE_OK;
  if (X == nullptr || W == nullptr || Y == nullptr ||
      ffn_shared({Y, workspace}, {X, W, row_scales}))
    return MOE_ERR_INVALID_ARGUMENT;
  for (const void* q : {X, W, (const void*)Y, (const void*)workspace})
    if (!ffn_aligned16(q)) return MOE_ERR_UNSUPPORTED;
  if (!aligned4(row_scales)) return MOE_ERR_UNSUPPORTED;
  const MatmulWs w = matmul_ws(S, K, N);
  if (workspace == nullptr || workspace_bytes < w.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  hipStream_t sq = (hipStream_t)stream;
  char* ws = (char*)workspace;
  const int8_t* codes = (const int8_t*)X;
  const bool f32 = dtype == MOE_F32, out_f32 = f32 || (flags & MOE_OUTPUT_F32) != 0;
  if (w.few) {
    const FewRows a = {X, row_scales, (const char*)W, Y, (int)S, (int)K, (int)N, 0};
    const hipError_t e = f32       ? launch_few_rows<float, float>(a, sq)
                         : out_f32 ? launch_few_rows<bf16_t, float>(a, sq)
                                   : launch_few_rows<bf16_t, bf16_t>(a, sq);
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
  }
  if (row_scales == nullptr) {
    codes = (int8_t*)(ws + w.codes);
    row_scales = (float*)(ws + w.scales);
    if (launch_quantize_rows(X, S, K, f32, (int8_t*)(ws + w.codes), (float*)(ws + w.scales),
                             sq) != hipSuccess)
      return MOE_ERR_HIP;
  }
  const float* sw = scales_of(W, K, N);
  if (out_f32)
    run_i8<false>(w.p, S, K, N, codes, W, nullptr,
                  EpI8Store<float>{(float*)Y, row_scales, sw, N}, ws + w.part, sq);
  else
    run_i8<false>(w.p, S, K, N, codes, W, nullptr,
                  EpI8Store<bf16_t>{(bf16_t*)Y, row_scales, sw, N}, ws + w.part, sq);
  return enqueued();
}

extern "C" size_t moe_i8_ffn_workspace_bytes(const moe_ffn_shape* shape) {
  return check_i8_ffn(shape) == MOE_OK ? ffn_ws(shape).total : 0;
}

extern "C" moe_status moe_i8_ffn_forward(const moe_ffn_shape* s, const void* X, const void* W_up,
                                         const void* W_gate, const void* W_down, void* O,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  const moe_status st = check_i8_ffn(s);
  if (st != MOE_OK) return st;
  if (s->S == 0) return MOE_OK;
  if (X == nullptr || W_up == nullptr || W_gate == nullptr || W_down == nullptr || O == nullptr ||
      ffn_shared({O, workspace}, {X, W_up, W_gate, W_down}))
    return MOE_ERR_INVALID_ARGUMENT;
  for (const void* q : {X, W_up, W_gate, W_down, (const void*)O, (const void*)workspace})
    if (!ffn_aligned16(q)) return MOE_ERR_UNSUPPORTED;
  const FfnWs w = ffn_ws(s);
  if (workspace == nullptr || workspace_bytes < w.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  hipStream_t sq = (hipStream_t)stream;
  char* ws = (char*)workspace;
  int8_t *xc = (int8_t*)(ws + w.xc), *hc = (int8_t*)(ws + w.hc);
  float *xs = (float*)(ws + w.xs), *hs = (float*)(ws + w.hs), *h = (float*)(ws + w.h);
  const bool f32 = s->dtype == MOE_F32;
  if (launch_quantize_rows(X, s->S, s->H, f32, xc, xs, sq) != hipSuccess) return MOE_ERR_HIP;
  const EpI8Swiglu swiglu = {h, xs, scales_of(W_up, s->H, s->D), scales_of(W_gate, s->H, s->D),
                             s->D};
  const bool join_here = w.up.splits > 1 && s->D <= kJoinCols;
  const GemmArgs g = run_i8<true>(w.up, s->S, s->H, s->D, xc, W_up, W_gate, swiglu, ws + w.part,
                                  sq, !join_here);
  if (join_here)
    i8_join_kernel<<<(unsigned)s->S, 512, 0, sq>>>(g, swiglu, hc, hs);
  else if (launch_quantize_rows(h, s->S, s->D, true, hc, hs, sq) != hipSuccess)
    return MOE_ERR_HIP;
  const float* sd = scales_of(W_down, s->D, s->H);
  if (f32 || (s->flags & MOE_OUTPUT_F32))
    run_i8<false>(w.down, s->S, s->D, s->H, hc, W_down, nullptr,
                  EpI8Store<float>{(float*)O, hs, sd, s->H}, ws + w.part, sq);
  else
    run_i8<false>(w.down, s->S, s->D, s->H, hc, W_down, nullptr,
                  EpI8Store<bf16_t>{(bf16_t*)O, hs, sd, s->H}, ws + w.part, sq);
  return enqueued();
}
