// Layer norm, forward and backward (include/moe_ffn.h).
//
// Forward: one pass over X. A row is read once into registers, its mean and
// then the mean of its centred squares are summed there (two sums in
// registers: no cancellation as in E[x^2] - E[x]^2), and the result is
// written. Bound by HBM: X once in, Y once out.
//
// Backward: one pass over X and dY. Each workgroup walks over rows; a thread
// keeps the same columns of every row, so it sums its columns' dgamma and
// dbeta in registers (fp32) while it forms dX. The workgroups' sums go to the
// workspace, [workgroups][2][H], and a second kernel adds them in a fixed
// order: no atomics, the same bits on every run.
//
// A row is shared by TPR threads: 16 lanes or a wave where their registers hold the
// row (no barrier then), else a workgroup of 256 or 512. Rows too long for that are
// read again for each sum (they then come from L2). The workgroups walk over the rows,
// a few to a CU, and the next row's loads are out before the sums of the current
// one: what gamma, beta (and their gradients' sums) hold stays in registers.
#include "ffn_common.h"

namespace moe {
namespace {

constexpr int64_t kMaxRow = 1 << 27;
// Workgroups of the reduction, of 1024 threads: a launch has below 2^32 (one for each 64
// of 2 H columns would be 2^22 of them from H = 2^27 - 31 on).
constexpr int64_t kReduceGroups = 1 << 21;
constexpr int kThreads = 256;  // of the kernels that share rows by waves, or re-read them

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xF, 0xF,
                                                         false));
}
// Sum over a wave (N = 64) or each 16 lanes of it, in every lane, without LDS: exchanges
// within quads, half rows and rows of 16 lanes, then between rows and halves.
template <int N>
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0xB1>(v);   // quad_perm 1 0 3 2
  v = dpp_add<0x4E>(v);   // quad_perm 2 3 0 1
  v = dpp_add<0x141>(v);  // row_half_mirror
  v = dpp_add<0x140>(v);  // row_mirror
  if constexpr (N == 16) return v;
  auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(w[0]) + __uint_as_float(w[1]);
  w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(w[0]) + __uint_as_float(w[1]);
}

// Sum over the TPR threads of a row: a wave's by lane exchange, a workgroup's
// through LDS in wave order. `red` has room for 2 x (waves) x NV floats and is
// used in turn (par), so one barrier per sum is enough.
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float* red, int& par) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum<TPR < 64 ? TPR : 64>(v[i]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* r = red + par * W * NV;
    par ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) r[(threadIdx.x >> 6) * NV + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = r[i];
#pragma unroll
      for (int w = 1; w < W; ++w) v[i] += r[w * NV + i];
    }
  }
}

// A sum of many terms that keeps what each addition rounds off (exactly: the two-sum): its
// error does not grow with their number. A thread of a row of 2^24 adds 65536 values; plain
// fp32 sums of equal values were off by 6e-4 of them there, and by 2.5e-3 at 2^26, which
// the centred squares then hold. (Cost: 1 x 20000 fp32 forward 11.8 -> 12.6 us, 512 x 32768
// 40.5 -> 41.5, 4096 x 65536 bf16 328 either way.)
struct LongSum {
  float s = 0.f, c = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = s + v, b = t - s;
    c += (s - (t - b)) + (v - b);
    s = t;
  }
  // not a finite sum: s itself (c is NaN then)
  __device__ __forceinline__ float value() const { return isfinite(s) ? s + c : s; }
};

// 16 bytes of a row as loaded. RAG: rows that are not whole 16-byte vectors, or not
// aligned to them; their vectors are accessed at whatever address they lie (element by
// element: 700 x 9001 fp32 forward 40 -> 15 us, 20000 x 511 bf16 21 -> 10 us).
// Rows are read and written once. Aligned ones both with the non-temporal hint (16384 x
// 7168 bf16, cold caches: forward 119 -> 88 us, backward 169 -> 131 us, 5.4 TB/s; the
// hint on the stores alone made them slower): arrays about as large as the caches, the norm
// alone; what the hint costs whoever reads a small Y next was not timed. The others' vectors share cache lines with
// their neighbours: the hint on the stores only (30000 x 511 bf16 backward: none 28 us,
// stores 24, both 28; 16384 x 7167 forward: 106, 78, 103).
template <typename T>
constexpr int vec_of() { return 16 / (int)sizeof(T); }

// 16 bytes at an element's alignment
typedef float vec_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef float vec_at2 __attribute__((ext_vector_type(4), aligned(2)));
template <typename T>
using vec_at = std::conditional_t<sizeof(T) == 4, vec_at4, vec_at2>;

template <typename T>
struct Raw {
  static constexpr int VEC = vec_of<T>();
  T v[VEC];
  template <bool RAG, bool ONCE>
  __device__ __forceinline__ void load(const T* p, int64_t left) {
    if constexpr (!RAG && ONCE) {
      *this = __builtin_bit_cast(
          Raw, __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p)));
    } else if constexpr (!RAG) {
      *this = __builtin_bit_cast(Raw, *reinterpret_cast<const f32x4_t*>(p));
    } else if (left >= VEC) {
      const vec_at<T> w = *reinterpret_cast<const vec_at<T>*>(p);
      asm volatile("");  // (else merged with the elements' loads below)
      *this = __builtin_bit_cast(Raw, w);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = e < left ? p[e] : T{};
    }
  }
  __device__ __forceinline__ float operator[](int i) const { return to_f32<T>(v[i]); }
};
template <typename T, bool RAG>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[vec_of<T>()], int64_t left) {
  constexpr int VEC = vec_of<T>();
  Raw<T> t;
#pragma unroll
  for (int e = 0; e < VEC; ++e) t.v[e] = from_f32<T>(f[e]);
  if constexpr (!RAG) {
    __builtin_nontemporal_store(__builtin_bit_cast(f32x4_t, t), reinterpret_cast<f32x4_t*>(p));
  } else if (left >= VEC) {
    __builtin_nontemporal_store(__builtin_bit_cast(vec_at<T>, t),
                                reinterpret_cast<vec_at<T>*>(p));
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < left) p[e] = t.v[e];
  }
}

// Column sums of a vector's columns.
template <bool RAG, int VEC>
__device__ __forceinline__ void store_sums(float* p, const float (&f)[VEC], int64_t left) {
  if constexpr (!RAG) {
    store_n(p, f);
  } else if (left >= VEC) {
#pragma unroll
    for (int e = 0; e < VEC; e += 4)
      *reinterpret_cast<vec_at<float>*>(p + e) = vec_at<float>{f[e], f[e + 1], f[e + 2], f[e + 3]};
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < left) p[e] = f[e];
  }
}

// The columns of vector c0 / VEC of a row. RAG: the last vector is moved back to end with
// the row; its first `skip` columns are another thread's too, which computes the same
// for them, so only the row's sums leave them out (a tail of single elements made the
// wave that has it wait for its loads: 20000 x 511 fp32 backward 76 -> 44 us). Rows
// shorter than a vector are read element by element.
template <typename T, bool RAG>
struct Cols {
  static constexpr int VEC = vec_of<T>();
  int at, skip, end;
  bool in;
  __device__ __forceinline__ Cols(int c0, int64_t H) {
    const int h = (int)H;
    in = c0 < h;
    at = RAG && c0 > h - VEC ? (h > VEC ? h - VEC : 0) : c0;
    skip = c0 - at;
    end = h < VEC ? h : VEC;
  }
  // whether column at + e counts in this thread's sums
  __device__ __forceinline__ bool counts(int e) const {
    return in && (!RAG || (e >= skip && e < end));
  }
};

// This thread's vectors of a row (IT of them, TPR apart).
template <typename T, bool RAG, int TPR, int IT, bool ONCE = true>
__device__ __forceinline__ void load_row(const T* row, int64_t H, int t, Raw<T> (&v)[IT]) {
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const Cols<T, RAG> c((i * TPR + t) * vec_of<T>(), H);
    if (c.in) v[i].template load<RAG, ONCE>(row + c.at, TPR > 16 ? vec_of<T>() : H);
  }
}

template <int TPR>
constexpr int group_threads() { return TPR > kThreads ? TPR : kThreads; }

// Rows of at most TPR * VEC * IT elements, held in registers.
template <typename T, bool RAG, int TPR, int IT>
__global__ __launch_bounds__(group_threads<TPR>()) void ln_fwd_kernel(
    int64_t S, int64_t H, const T* X, const T* gamma, const T* beta, float eps, T* Y, float* mean,
    float* rstd) {
  constexpr int RPB = group_threads<TPR>() / TPR, VEC = vec_of<T>();
  __shared__ float red[TPR > 64 ? 2 * (TPR / 64) : 1];
  int par = 0;
  const int t = threadIdx.x % TPR;
  const int64_t stride = (int64_t)gridDim.x * RPB;
  // the same rows for every thread of a row's TPR: barriers stay uniform
  int64_t s = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  Raw<T> g[IT], b[IT], next[IT];
  if (gamma) load_row<T, RAG, TPR, IT, false>(gamma, H, t, g);
  if (beta) load_row<T, RAG, TPR, IT, false>(beta, H, t, b);
  if (s < S) load_row<T, RAG, TPR, IT>(X + s * H, H, t, next);
  for (; s < S; s += stride) {
    float v[IT][VEC];
    float sum[1] = {0.f}, sq[1] = {0.f};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const Cols<T, RAG> c((i * TPR + t) * VEC, H);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] = next[i][e];
        sum[0] += c.counts(e) ? v[i][e] : 0.f;
      }
    }
    if (s + stride < S) load_row<T, RAG, TPR, IT>(X + (s + stride) * H, H, t, next);
    row_sum<TPR, 1>(sum, red, par);
    const float m = sum[0] / (float)H;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const Cols<T, RAG> c((i * TPR + t) * VEC, H);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] -= m;
        sq[0] += c.counts(e) ? v[i][e] * v[i][e] : 0.f;
      }
    }
    row_sum<TPR, 1>(sq, red, par);
    const float r = 1.0f / sqrtf(sq[0] / (float)H + eps);
    T* y = Y + s * H;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const Cols<T, RAG> c((i * TPR + t) * VEC, H);
      if (c.in) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          o[e] = v[i][e] * r * (gamma ? g[i][e] : 1.f) + (beta ? b[i][e] : 0.f);
        store_vec<T, RAG>(y + c.at, o, TPR > 16 ? VEC : H);
      }
    }
    if (mean != nullptr && t == 0) {
      mean[s] = m;
      rstd[s] = r;
    }
  }
}

// Rows of any length: three passes over the row.
template <typename T, bool RAG>
__global__ __launch_bounds__(kThreads) void ln_fwd_long_kernel(int64_t S, int64_t H, const T* X,
                                                               const T* gamma, const T* beta,
                                                               float eps, T* Y, float* mean,
                                                               float* rstd) {
  __shared__ float red[2 * (kThreads / 64)];
  constexpr int VEC = vec_of<T>();
  int par = 0;
  for (int64_t s = blockIdx.x; s < S; s += gridDim.x) {
    const T* x = X + s * H;
    LongSum total, squares;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      Raw<T> v;
      v.template load<RAG, false>(x + c, H - c);
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) part += v[e];
      total.add(part);
    }
    float sum[1] = {total.value()};
    row_sum<kThreads, 1>(sum, red, par);
    const float m = sum[0] / (float)H;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      Raw<T> v;
      v.template load<RAG, false>(x + c, H - c);
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (!RAG || c + e < H) part += (v[e] - m) * (v[e] - m);
      squares.add(part);
    }
    float sq[1] = {squares.value()};
    row_sum<kThreads, 1>(sq, red, par);
    const float r = 1.0f / sqrtf(sq[0] / (float)H + eps);
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      Raw<T> v, g, b;
      v.template load<RAG, false>(x + c, H - c);
      if (gamma) g.template load<RAG, false>(gamma + c, H - c);
      if (beta) b.template load<RAG, false>(beta + c, H - c);
      float o[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        o[e] = (v[e] - m) * r * (gamma ? g[e] : 1.f) + (beta ? b[e] : 0.f);
      store_vec<T, RAG>(Y + s * H + c, o, H - c);
    }
    if (mean != nullptr && threadIdx.x == 0) {
      mean[s] = m;
      rstd[s] = r;
    }
  }
}

// Backward for rows held in registers. part: [gridDim.x][2][H] (dgamma, dbeta
// of this workgroup's rows), or null.
template <typename T, bool RAG, int TPR, int IT>
__global__ __launch_bounds__(group_threads<TPR>()) void ln_bwd_kernel(
    int64_t S, int64_t H, const T* dY, const T* X, const T* gamma, const float* mean,
    const float* rstd, T* dX, float* part) {
  constexpr int RPB = group_threads<TPR>() / TPR, VEC = vec_of<T>();
  __shared__ float red[TPR > 64 ? 2 * 2 * (TPR / 64) : 1];
  int par = 0;
  const int t = threadIdx.x % TPR;
  const int sub = threadIdx.x / TPR;
  Raw<T> g[IT], nx[IT], nd[IT];
  float ag[IT][VEC], ab[IT][VEC];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) ag[i][e] = ab[i][e] = 0.f;
  if (gamma) load_row<T, RAG, TPR, IT, false>(gamma, H, t, g);
  const float inv = 1.0f / (float)H;
  const int64_t stride = (int64_t)gridDim.x * RPB;
  int64_t s = (int64_t)blockIdx.x * RPB + sub;
  float nm = 0.f, nr = 0.f;
  auto fetch = [&](int64_t row) {
    load_row<T, RAG, TPR, IT>(X + row * H, H, t, nx);
    load_row<T, RAG, TPR, IT>(dY + row * H, H, t, nd);
    nm = mean[row];
    nr = rstd[row];
  };
  // the next row ahead; with 8 vectors of fp32 the registers hold one row only, and its
  // n and d are formed again from it instead of kept
  constexpr bool AHEAD = IT <= 6;
  if (AHEAD && s < S) fetch(s);
  for (; s < S; s += stride) {
    if constexpr (!AHEAD) fetch(s);
    const float m = nm, r = nr;
    float n[IT][VEC], d[IT][VEC];
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const Cols<T, RAG> c((i * TPR + t) * VEC, H);
      if (c.in)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          n[i][e] = (nx[i][e] - m) * r;
          d[i][e] = nd[i][e];
          ag[i][e] += d[i][e] * n[i][e];
          ab[i][e] += d[i][e];
          if (gamma) d[i][e] *= g[i][e];
          if (c.counts(e)) {
            sums[0] += d[i][e];
            sums[1] += d[i][e] * n[i][e];
          }
        }
    }
    if (AHEAD && s + stride < S) fetch(s + stride);
    row_sum<TPR, 2>(sums, red, par);
    const float c0 = sums[0] * inv, c1 = sums[1] * inv;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const Cols<T, RAG> c((i * TPR + t) * VEC, H);
      if (c.in) {
        if constexpr (!AHEAD)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float x = nx[i].v[e], y = nd[i].v[e];
            asm volatile("" : "+v"(x), "+v"(y));  // (else kept from above, and spilled)
            n[i][e] = (x - m) * r;
            d[i][e] = gamma ? y * g[i][e] : y;
          }
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[i][e] = r * (d[i][e] - c0 - n[i][e] * c1);
        store_vec<T, RAG>(dX + s * H + c.at, d[i], TPR > 16 ? VEC : H);
      }
    }
  }
  if (part == nullptr) return;
  float* pg = part + (int64_t)blockIdx.x * 2 * H;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const Cols<T, RAG> c((i * TPR + t) * VEC, H);
      if (c.in) {
        store_sums<RAG>(pg + c.at, ag[i], TPR > 16 ? VEC : H);
        store_sums<RAG>(pg + H + c.at, ab[i], TPR > 16 ? VEC : H);
      }
    }
  } else {
    // the waves' columns added in wave order through LDS
    __shared__ float cols[RPB][2][TPR * VEC];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if (i) __syncthreads();
      const Cols<T, RAG> c((i * TPR + t) * VEC, H);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (c.counts(e)) {
          cols[sub][0][t * VEC + e - c.skip] = ag[i][e];
          cols[sub][1][t * VEC + e - c.skip] = ab[i][e];
        }
      __syncthreads();
      for (int j = threadIdx.x; j < 2 * TPR * VEC; j += kThreads) {
        const int w = j / (TPR * VEC), cc = j % (TPR * VEC);
        const int64_t c = (int64_t)i * TPR * VEC + cc;
        if (c < H) {
          float a = cols[0][w][cc];
#pragma unroll
          for (int q = 1; q < RPB; ++q) a += cols[q][w][cc];
          pg[(int64_t)w * H + c] = a;
        }
      }
    }
  }
}

// dX of rows of any length (two passes over the row).
template <typename T, bool RAG>
__global__ __launch_bounds__(kThreads) void ln_bwd_long_kernel(int64_t S, int64_t H, const T* dY,
                                                               const T* X, const T* gamma,
                                                               const float* mean,
                                                               const float* rstd, T* dX) {
  __shared__ float red[2 * 2 * (kThreads / 64)];
  constexpr int VEC = vec_of<T>();
  int par = 0;
  for (int64_t s = blockIdx.x; s < S; s += gridDim.x) {
    const float m = mean[s], r = rstd[s];
    LongSum s0, s1;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      Raw<T> x, d, g;
      x.template load<RAG, false>(X + s * H + c, H - c);
      d.template load<RAG, false>(dY + s * H + c, H - c);
      if (gamma) g.template load<RAG, false>(gamma + c, H - c);
      float p0 = 0.f, p1 = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float dg = gamma ? d[e] * g[e] : d[e];
        p0 += dg;
        p1 += dg * ((x[e] - m) * r);
      }
      s0.add(p0);
      s1.add(p1);
    }
    float sums[2] = {s0.value(), s1.value()};
    row_sum<kThreads, 2>(sums, red, par);
    const float inv = 1.0f / (float)H;
    const float c0 = sums[0] * inv, c1 = sums[1] * inv;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      Raw<T> x, d, g;
      x.template load<RAG, false>(X + s * H + c, H - c);
      d.template load<RAG, false>(dY + s * H + c, H - c);
      if (gamma) g.template load<RAG, false>(gamma + c, H - c);
      float o[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float dg = gamma ? d[e] * g[e] : d[e];
        o[e] = r * (dg - c0 - (x[e] - m) * r * c1);
      }
      store_vec<T, RAG>(dX + s * H + c, o, H - c);
    }
  }
}

// Column sums of rows of any length: one thread per column, a range of rows
// per blockIdx.y, into part [gridDim.y][2][H].
template <typename T>
__global__ __launch_bounds__(kThreads) void ln_cols_kernel(int64_t S, int64_t H, const T* dY,
                                                           const T* X, const float* mean,
                                                           const float* rstd, float* part) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= H) return;
  float a = 0.f, b = 0.f;
  for (int64_t s = blockIdx.y; s < S; s += gridDim.y) {
    const float d = to_f32<T>(dY[s * H + c]);
    a += d * ((to_f32<T>(X[s * H + c]) - mean[s]) * rstd[s]);
    b += d;
  }
  part[(int64_t)blockIdx.y * 2 * H + c] = a;
  part[(int64_t)blockIdx.y * 2 * H + H + c] = b;
}

// dgamma, dbeta: the P partial sums of each of 2 H columns in a fixed order: 64
// columns per workgroup at a time, each of 16 waves a sixteenth of the partials, 8 loads
// at a time. (4 waves with one load at a time took 60 us for P = 512, H = 2048: one
// memory latency after another.)
__global__ __launch_bounds__(1024) void ln_reduce_kernel(int64_t P, int64_t H, const float* part,
                                                         float* dgamma, float* dbeta) {
  constexpr int W = 16, B = 8;
  __shared__ float red[W][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int64_t j0 = (int64_t)blockIdx.x * 64; j0 < 2 * H; j0 += (int64_t)gridDim.x * 64) {
    const int64_t j = j0 + lane;
    float a = 0.f;
    if (j < 2 * H)
      for (int64_t p = w; p < P; p += W * B) {
        float v[B];
#pragma unroll
        for (int e = 0; e < B; ++e) v[e] = p + e * W < P ? part[(p + e * W) * 2 * H + j] : 0.f;
#pragma unroll
        for (int e = 0; e < B; ++e) a += v[e];
      }
    if (j0 != (int64_t)blockIdx.x * 64) __syncthreads();  // the last columns' sums are read
    red[w][lane] = a;
    __syncthreads();
    if (w == 0 && j < 2 * H) {
#pragma unroll
      for (int q = 1; q < W; ++q) a += red[q][lane];
      (j < H ? dgamma[j] : dbeta[j - H]) = a;
    }
  }
}

// Which kernel takes a row: 16 lanes up to 1 vector per lane, a wave up to 2, a workgroup
// of 256 up to 4 vectors per thread, one of 512 up to 32 elements per thread, else the
// re-reading kernels. (16 lanes instead of a wave, 30000 x 64 fp32: forward 8.7 -> 4.6
// us, backward 19 -> 11. A wave instead of 256 threads for 2 vectors per lane, 20000 x
// 511 fp32: 24 -> 18 and 44 -> 31 us; for 4 vectors per lane it is 66 us instead of 58,
// 16384 x 2048 bf16 backward: too few rows in flight at 220 registers. 512 x 16384 fp32
// in registers instead of read again: 18.8 -> 14.3 and 62 -> 35 us; with 1024 threads the
// backward pass spills: 44 us.)
struct LnPlan {
  bool rag;
  int tpr, it;  // it = 0: long rows
};
LnPlan ln_plan(int64_t H, int es, bool aligned) {
  LnPlan p;
  p.rag = !aligned || (H * es) % 16 != 0;
  const int64_t v = 16 / es;
  for (int tpr : {16, 64, 256, 512}) {
    const int64_t it = (H + tpr * v - 1) / (tpr * v);
    if (it > (tpr == 16 ? 1 : tpr == 64 ? 2 : tpr == 256 ? 4 : 32 / v)) continue;
    p.tpr = tpr;
    p.it = (int)(it > 4 ? (it + 1) / 2 * 2 : it);  // compiled for 1, 2, 3, 4, 6 and 8
    return p;
  }
  p.tpr = kThreads;
  p.it = 0;
  return p;
}

// Workgroups of the backward pass, each with partial sums of its own, which go through
// memory twice: at most 512 (1024: dX as fast, the sums' way twice as long), and with
// fewer than 2048 rows one for 4 rows, but 128 at least (500 x 4096 bf16: 512 workgroups
// 13.9 us, 128 11.2; 1000 x 8192 fp32: 32.5 and, with 250, 26.2). The rows' length is not
// weighed: 512 x 16384 fp32 takes 128, half of the CUs, and 39 us, where its bytes take 20.
constexpr int64_t kBwdGroups = 512;
constexpr int64_t kRowGroups = 2048;  // of the forward pass: 8 of 256 threads to a CU

int64_t bwd_groups(int64_t S, const LnPlan& p) {
  const int64_t rpb = p.tpr < kThreads ? kThreads / p.tpr : 1;
  const int64_t n = (S + rpb - 1) / rpb, few = (n + 4 - 1) / 4;
  if (few >= kBwdGroups) return kBwdGroups;
  return few > 128 ? few : n < 128 ? n : 128;
}

template <typename T, typename F>
void dispatch(const LnPlan& p, F f) {
  auto with = [&](auto tpr) {
    auto it = [&](auto n) {
      if (p.tpr == decltype(tpr)::value && p.it == decltype(n)::value) f(tpr, n);
    };
    // what ln_plan can ask for: longer rows begin where the smaller group's end
    constexpr int TPR = decltype(tpr)::value;
    if constexpr (TPR <= 256) it(std::integral_constant<int, 1>{});
    if constexpr (TPR == 64 || TPR == 256) it(std::integral_constant<int, 2>{});
    if constexpr (TPR >= 256) it(std::integral_constant<int, 3>{});
    if constexpr (TPR >= 256) it(std::integral_constant<int, 4>{});
    if constexpr (TPR == 512 && vec_of<T>() == 4) it(std::integral_constant<int, 6>{});
    if constexpr (TPR == 512 && vec_of<T>() == 4) it(std::integral_constant<int, 8>{});
  };
  with(std::integral_constant<int, 16>{});
  with(std::integral_constant<int, 64>{});
  with(std::integral_constant<int, 256>{});
  with(std::integral_constant<int, 512>{});
}

// Workgroups over n rows; the kernels walk over further rows.
unsigned row_grid(int64_t n) { return (unsigned)(n < kRowGroups ? n : kRowGroups); }

template <typename T, bool RAG>
void forward_t(const LnPlan& p, int64_t S, int64_t H, const T* X, const T* gamma, const T* beta,
               float eps, T* Y, float* mean, float* rstd, hipStream_t st) {
  if (p.it == 0) {
    ln_fwd_long_kernel<T, RAG><<<row_grid(S), kThreads, 0, st>>>(S, H, X, gamma, beta, eps, Y,
                                                                mean, rstd);
    return;
  }
  dispatch<T>(p, [&](auto tpr, auto it) {
    constexpr int TPR = decltype(tpr)::value, NT = group_threads<TPR>(), RPB = NT / TPR;
    ln_fwd_kernel<T, RAG, TPR, decltype(it)::value>
        <<<row_grid((S + RPB - 1) / RPB), NT, 0, st>>>(S, H, X, gamma, beta, eps, Y, mean, rstd);
  });
}

template <typename T, bool RAG>
void backward_t(const LnPlan& p, int64_t S, int64_t H, const T* dY, const T* X, const T* gamma,
                const float* mean, const float* rstd, T* dX, float* part, int64_t groups,
                hipStream_t st) {
  if (p.it == 0) {
    ln_bwd_long_kernel<T, RAG>
        <<<row_grid(S), kThreads, 0, st>>>(S, H, dY, X, gamma, mean, rstd, dX);
    if (part)
      ln_cols_kernel<T><<<dim3((unsigned)((H + kThreads - 1) / kThreads), (unsigned)groups),
                          kThreads, 0, st>>>(S, H, dY, X, mean, rstd, part);
    return;
  }
  dispatch<T>(p, [&](auto tpr, auto it) {
    constexpr int TPR = decltype(tpr)::value;
    ln_bwd_kernel<T, RAG, TPR, decltype(it)::value>
        <<<(unsigned)groups, group_threads<TPR>(), 0, st>>>(S, H, dY, X, gamma, mean, rstd, dX,
                                                            part);
  });
}

moe_status check_ln(int64_t S, int64_t H, int32_t dtype) {
  if (S < 0 || H < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (dtype == MOE_MXFP8) return MOE_ERR_UNSUPPORTED;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (S >= INT32_MAX || H >= kMaxRow) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool misaligned(const void* p, int es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }

moe_status enqueued() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_layernorm_forward(int64_t S, int64_t H, int32_t dtype, const void* X,
                                            const void* gamma, const void* beta, float eps,
                                            void* Y, float* mean, float* rstd, void* stream) {
  moe_status st = check_ln(S, H, dtype);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f) || eps > 3.0e38f) return MOE_ERR_INVALID_ARGUMENT;
  if ((mean == nullptr) != (rstd == nullptr)) return MOE_ERR_INVALID_ARGUMENT;
  if (S == 0) return MOE_OK;
  if (X == nullptr || Y == nullptr || ffn_shared({Y, mean, rstd}, {X, gamma, beta}))
    return MOE_ERR_INVALID_ARGUMENT;
  const int es = dtype == MOE_F32 ? 4 : 2;
  if (misaligned(X, es) || misaligned(Y, es) || misaligned(gamma, es) || misaligned(beta, es) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return MOE_ERR_UNSUPPORTED;
  const LnPlan p = ln_plan(H, es, ffn_aligned16(X) && ffn_aligned16(Y) && ffn_aligned16(gamma) &&
                                      ffn_aligned16(beta));
  auto go = [&](auto tag) {
    using T = decltype(tag);
    auto call = [&](auto rag) {
      forward_t<T, decltype(rag)::value>(p, S, H, (const T*)X, (const T*)gamma, (const T*)beta,
                                         eps, (T*)Y, mean, rstd, (hipStream_t)stream);
    };
    if (p.rag)
      call(std::true_type{});
    else
      call(std::false_type{});
  };
  if (dtype == MOE_F32)
    go(float{});
  else
    go(bf16_t{});
  return enqueued();
}

extern "C" size_t moe_layernorm_backward_workspace_bytes(int64_t S, int64_t H, int32_t dtype) {
  if (check_ln(S, H, dtype) != MOE_OK) return 0;
  // for either alignment of the arrays, and never 0
  const int64_t n = S < kBwdGroups ? S : kBwdGroups;
  return (size_t)(n ? n : 1) * 2 * (size_t)H * sizeof(float);
}

extern "C" moe_status moe_layernorm_backward(int64_t S, int64_t H, int32_t dtype, const void* dY,
                                             const void* X, const void* gamma, const float* mean,
                                             const float* rstd, void* dX, float* dgamma,
                                             float* dbeta, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  moe_status st = check_ln(S, H, dtype);
  if (st != MOE_OK) return st;
  if ((dgamma == nullptr) != (dbeta == nullptr)) return MOE_ERR_INVALID_ARGUMENT;
  if (S > 0 && (dY == nullptr || X == nullptr || mean == nullptr || rstd == nullptr ||
                dX == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ffn_shared({dX, dgamma, dbeta, dgamma != nullptr ? workspace : nullptr},
                 {dY, X, gamma, mean, rstd}))
    return MOE_ERR_INVALID_ARGUMENT;
  if (dgamma != nullptr &&
      (workspace == nullptr ||
       workspace_bytes < moe_layernorm_backward_workspace_bytes(S, H, dtype)))
    return MOE_ERR_WORKSPACE_TOO_SMALL;
  const int es = dtype == MOE_F32 ? 4 : 2;
  if (misaligned(X, es) || misaligned(dY, es) || misaligned(dX, es) || misaligned(gamma, es) ||
      misaligned(mean, 4) || misaligned(rstd, 4) || misaligned(dgamma, 4) ||
      misaligned(dbeta, 4) || (dgamma != nullptr && misaligned(workspace, 16)))
    return MOE_ERR_UNSUPPORTED;
  if (S == 0 && dgamma == nullptr) return MOE_OK;
  const LnPlan p = ln_plan(H, es, ffn_aligned16(X) && ffn_aligned16(dY) && ffn_aligned16(dX) &&
                                      ffn_aligned16(gamma));
  const int64_t groups = bwd_groups(S, p);
  float* part = dgamma != nullptr ? (float*)workspace : nullptr;
  if (S > 0) {
    auto go = [&](auto tag) {
      using T = decltype(tag);
      auto call = [&](auto rag) {
        backward_t<T, decltype(rag)::value>(p, S, H, (const T*)dY, (const T*)X, (const T*)gamma,
                                            mean, rstd, (T*)dX, part, groups,
                                            (hipStream_t)stream);
      };
      if (p.rag)
        call(std::true_type{});
      else
        call(std::false_type{});
    };
    if (dtype == MOE_F32)
      go(float{});
    else
      go(bf16_t{});
  }
  if (dgamma != nullptr) {
    const int64_t cols = (2 * H + 63) / 64;
    ln_reduce_kernel<<<(unsigned)(cols < kReduceGroups ? cols : kReduceGroups), 1024, 0,
                       (hipStream_t)stream>>>(S > 0 ? groups : 0, H, part, dgamma, dbeta);
  }
  return enqueued();
}
