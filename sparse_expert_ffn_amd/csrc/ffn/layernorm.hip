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
// A row is shared by TPR threads: a wave where its registers hold the row (no
// barrier then), else a workgroup of 256 or 512. Rows too long for that are read
// again for each sum (they then come from L2). The workgroups walk over the rows,
// a few to a CU, and the next row's loads are out before the sums of the current
// one: what gamma, beta (and their gradients' sums) hold stays in registers.
#include "ffn_common.h"

namespace moe {
namespace {

constexpr int64_t kMaxRow = 1 << 27;
constexpr int kThreads = 256;  // of the kernels that share rows by waves, or re-read them

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xF, 0xF,
                                                         false));
}
// Sum over a wave in every lane, without LDS: exchanges within quads, half rows and
// rows of 16 lanes, then between rows and halves.
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0xB1>(v);   // quad_perm 1 0 3 2
  v = dpp_add<0x4E>(v);   // quad_perm 2 3 0 1
  v = dpp_add<0x141>(v);  // row_half_mirror
  v = dpp_add<0x140>(v);  // row_mirror
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
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
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

// VEC consecutive elements as loaded (one of them, or 16 bytes). Rows are read and
// written once: vectors both with the non-temporal hint (16384 x 7168 bf16, cold
// caches: forward 119 -> 88 us, backward 169 -> 131 us, 5.4 TB/s; the hint on the
// stores alone made them slower). Not single elements, whose accesses share cache
// lines with each other's (4099 x 1001 fp32 backward out of a warm cache: 18 us
// with the hint, 15 us without).
template <typename T, int VEC>
struct Raw {
  T v[VEC];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 1)
      v[0] = p[0];
    else
      *this = __builtin_bit_cast(Raw, *reinterpret_cast<const f32x4_t*>(p));
  }
  __device__ __forceinline__ void load_once(const T* p) {
    if constexpr (VEC == 1)
      v[0] = p[0];
    else
      *this = __builtin_bit_cast(
          Raw, __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p)));
  }
  __device__ __forceinline__ float operator[](int i) const { return to_f32<T>(v[i]); }
};
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
  Raw<T, VEC> t;
#pragma unroll
  for (int i = 0; i < VEC; ++i) t.v[i] = from_f32<T>(f[i]);
  if constexpr (VEC == 1)
    p[0] = t.v[0];
  else
    __builtin_nontemporal_store(__builtin_bit_cast(f32x4_t, t), reinterpret_cast<f32x4_t*>(p));
}

// Column sums: 4 to a store (whole 16-byte vectors wherever rows are).
template <int VEC>
__device__ __forceinline__ void store_sums(float* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1)
    p[0] = f[0];
  else
    store_n(p, f);
}

// This thread's vectors of a row (IT of them, TPR apart).
template <typename T, int VEC, int TPR, int IT, bool ONCE = true>
__device__ __forceinline__ void load_row(const T* row, int64_t H, int t, Raw<T, VEC> (&v)[IT]) {
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (i * TPR + t) * VEC;
    if (c < H) {
      if constexpr (ONCE)
        v[i].load_once(row + c);
      else
        v[i].load(row + c);
    }
  }
}

template <int TPR>
constexpr int group_threads() { return TPR > kThreads ? TPR : kThreads; }

// Rows of at most TPR * VEC * IT elements, held in registers.
template <typename T, int VEC, int TPR, int IT>
__global__ __launch_bounds__(group_threads<TPR>()) void ln_fwd_kernel(
    int64_t S, int64_t H, const T* X, const T* gamma, const T* beta, float eps, T* Y, float* mean,
    float* rstd) {
  constexpr int RPB = group_threads<TPR>() / TPR;
  __shared__ float red[2 * (TPR / 64)];
  int par = 0;
  const int t = threadIdx.x % TPR;
  const int64_t stride = (int64_t)gridDim.x * RPB;
  // the same rows for every thread of a row's TPR: barriers stay uniform
  int64_t s = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  Raw<T, VEC> g[IT], b[IT], next[IT];
  if (gamma) load_row<T, VEC, TPR, IT, false>(gamma, H, t, g);
  if (beta) load_row<T, VEC, TPR, IT, false>(beta, H, t, b);
  if (s < S) load_row<T, VEC, TPR, IT>(X + s * H, H, t, next);
  for (; s < S; s += stride) {
    float v[IT][VEC];
    float sum[1] = {0.f}, sq[1] = {0.f};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const bool in = (i * TPR + t) * VEC < H;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] = in ? next[i][e] : 0.f;
        sum[0] += v[i][e];
      }
    }
    if (s + stride < S) load_row<T, VEC, TPR, IT>(X + (s + stride) * H, H, t, next);
    row_sum<TPR, 1>(sum, red, par);
    const float m = sum[0] / (float)H;
#pragma unroll
    for (int i = 0; i < IT; ++i)
      if ((i * TPR + t) * VEC < H)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          v[i][e] -= m;
          sq[0] += v[i][e] * v[i][e];
        }
    row_sum<TPR, 1>(sq, red, par);
    const float r = 1.0f / sqrtf(sq[0] / (float)H + eps);
    T* y = Y + s * H;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (c < H) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          o[e] = v[i][e] * r * (gamma ? g[i][e] : 1.f) + (beta ? b[i][e] : 0.f);
        store_vec<T, VEC>(y + c, o);
      }
    }
    if (mean != nullptr && t == 0) {
      mean[s] = m;
      rstd[s] = r;
    }
  }
}

// Rows of any length: three passes over the row.
template <typename T, int VEC>
__global__ __launch_bounds__(kThreads) void ln_fwd_long_kernel(int64_t S, int64_t H, const T* X,
                                                               const T* gamma, const T* beta,
                                                               float eps, T* Y, float* mean,
                                                               float* rstd) {
  __shared__ float red[2 * (kThreads / 64)];
  int par = 0;
  for (int64_t s = blockIdx.x; s < S; s += gridDim.x) {
    const T* x = X + s * H;
    float sum[1] = {0.f}, sq[1] = {0.f};
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      Raw<T, VEC> v;
      v.load(x + c);
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum[0] += v[e];
    }
    row_sum<kThreads, 1>(sum, red, par);
    const float m = sum[0] / (float)H;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      Raw<T, VEC> v;
      v.load(x + c);
#pragma unroll
      for (int e = 0; e < VEC; ++e) sq[0] += (v[e] - m) * (v[e] - m);
    }
    row_sum<kThreads, 1>(sq, red, par);
    const float r = 1.0f / sqrtf(sq[0] / (float)H + eps);
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      Raw<T, VEC> v, g, b;
      v.load(x + c);
      if (gamma) g.load(gamma + c);
      if (beta) b.load(beta + c);
      float o[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        o[e] = (v[e] - m) * r * (gamma ? g[e] : 1.f) + (beta ? b[e] : 0.f);
      store_vec<T, VEC>(Y + s * H + c, o);
    }
    if (mean != nullptr && threadIdx.x == 0) {
      mean[s] = m;
      rstd[s] = r;
    }
  }
}

// Backward for rows held in registers. part: [gridDim.x][2][H] (dgamma, dbeta
// of this workgroup's rows), or null.
template <typename T, int VEC, int TPR, int IT>
__global__ __launch_bounds__(group_threads<TPR>()) void ln_bwd_kernel(
    int64_t S, int64_t H, const T* dY, const T* X, const T* gamma, const float* mean,
    const float* rstd, T* dX, float* part) {
  constexpr int RPB = group_threads<TPR>() / TPR;
  __shared__ float red[2 * 2 * (TPR / 64)];
  int par = 0;
  const int t = threadIdx.x % TPR;
  const int sub = threadIdx.x / TPR;
  Raw<T, VEC> g[IT], nx[IT], nd[IT];
  float ag[IT][VEC], ab[IT][VEC];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) ag[i][e] = ab[i][e] = 0.f;
  if (gamma) load_row<T, VEC, TPR, IT, false>(gamma, H, t, g);
  const float inv = 1.0f / (float)H;
  const int64_t stride = (int64_t)gridDim.x * RPB;
  int64_t s = (int64_t)blockIdx.x * RPB + sub;
  float nm = 0.f, nr = 0.f;
  if (s < S) {
    load_row<T, VEC, TPR, IT>(X + s * H, H, t, nx);
    load_row<T, VEC, TPR, IT>(dY + s * H, H, t, nd);
    nm = mean[s];
    nr = rstd[s];
  }
  for (; s < S; s += stride) {
    const float m = nm, r = nr;
    float n[IT][VEC], d[IT][VEC];
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < IT; ++i)
      if ((i * TPR + t) * VEC < H)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          n[i][e] = (nx[i][e] - m) * r;
          d[i][e] = nd[i][e];
          ag[i][e] += d[i][e] * n[i][e];
          ab[i][e] += d[i][e];
          if (gamma) d[i][e] *= g[i][e];
          sums[0] += d[i][e];
          sums[1] += d[i][e] * n[i][e];
        }
    if (s + stride < S) {
      load_row<T, VEC, TPR, IT>(X + (s + stride) * H, H, t, nx);
      load_row<T, VEC, TPR, IT>(dY + (s + stride) * H, H, t, nd);
      nm = mean[s + stride];
      nr = rstd[s + stride];
    }
    row_sum<TPR, 2>(sums, red, par);
    const float c0 = sums[0] * inv, c1 = sums[1] * inv;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * TPR + t) * VEC;
      if (c < H) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[i][e] = r * (d[i][e] - c0 - n[i][e] * c1);
        store_vec<T, VEC>(dX + s * H + c, d[i]);
      }
    }
  }
  if (part == nullptr) return;
  float* pg = part + (int64_t)blockIdx.x * 2 * H;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int64_t c = ((int64_t)i * TPR + t) * VEC;
      if (c < H) {
        store_sums<VEC>(pg + c, ag[i]);
        store_sums<VEC>(pg + H + c, ab[i]);
      }
    }
  } else {
    // the waves' columns added in wave order through LDS
    __shared__ float cols[RPB][2][TPR * VEC];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      if (i) __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        cols[sub][0][t * VEC + e] = ag[i][e];
        cols[sub][1][t * VEC + e] = ab[i][e];
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
template <typename T, int VEC>
__global__ __launch_bounds__(kThreads) void ln_bwd_long_kernel(int64_t S, int64_t H, const T* dY,
                                                               const T* X, const T* gamma,
                                                               const float* mean,
                                                               const float* rstd, T* dX) {
  __shared__ float red[2 * 2 * (kThreads / 64)];
  int par = 0;
  for (int64_t s = blockIdx.x; s < S; s += gridDim.x) {
    const float m = mean[s], r = rstd[s];
    float sums[2] = {0.f, 0.f};
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      Raw<T, VEC> x, d, g;
      x.load(X + s * H + c);
      d.load(dY + s * H + c);
      if (gamma) g.load(gamma + c);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float dg = gamma ? d[e] * g[e] : d[e];
        sums[0] += dg;
        sums[1] += dg * ((x[e] - m) * r);
      }
    }
    row_sum<kThreads, 2>(sums, red, par);
    const float inv = 1.0f / (float)H;
    const float c0 = sums[0] * inv, c1 = sums[1] * inv;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      Raw<T, VEC> x, d, g;
      x.load(X + s * H + c);
      d.load(dY + s * H + c);
      if (gamma) g.load(gamma + c);
      float o[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float dg = gamma ? d[e] * g[e] : d[e];
        o[e] = r * (dg - c0 - (x[e] - m) * r * c1);
      }
      store_vec<T, VEC>(dX + s * H + c, o);
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
// columns per workgroup, each of 16 waves a sixteenth of the partials, 8 loads at
// a time. (4 waves with one load at a time took 60 us for P = 512, H = 2048: one
// memory latency after another.)
__global__ __launch_bounds__(1024) void ln_reduce_kernel(int64_t P, int64_t H, const float* part,
                                                         float* dgamma, float* dbeta) {
  constexpr int W = 16, B = 8;
  __shared__ float red[W][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t j = (int64_t)blockIdx.x * 64 + lane;
  float a = 0.f;
  if (j < 2 * H)
    for (int64_t p = w; p < P; p += W * B) {
      float v[B];
#pragma unroll
      for (int e = 0; e < B; ++e) v[e] = p + e * W < P ? part[(p + e * W) * 2 * H + j] : 0.f;
#pragma unroll
      for (int e = 0; e < B; ++e) a += v[e];
    }
  red[w][lane] = a;
  __syncthreads();
  if (w == 0 && j < 2 * H) {
#pragma unroll
    for (int q = 1; q < W; ++q) a += red[q][lane];
    (j < H ? dgamma[j] : dbeta[j - H]) = a;
  }
}

// Which kernel takes a row: a wave per row up to 1 vector (or 4 elements) per lane,
// a workgroup of 256 or 512 per row up to 4 vectors (16 elements) per thread, else
// the re-reading kernels. (Rows of 4 vectors per lane by waves: 66 us where a
// workgroup per row takes 58, 16384 x 2048 bf16 backward: too few rows in flight
// at 220 registers.)
struct LnPlan {
  bool vec;
  int tpr, it;  // it = 0: long rows
};
LnPlan ln_plan(int64_t H, int es, bool aligned) {
  LnPlan p;
  p.vec = aligned && (H * es) % 16 == 0;
  const int64_t v = p.vec ? 16 / es : 1;
  for (int tpr : {64, 256, 512}) {
    const int64_t it = (H + tpr * v - 1) / (tpr * v);
    if (it > (p.vec ? (tpr == 64 ? 1 : 4) : (tpr == 64 ? 4 : 16))) continue;
    p.tpr = tpr;
    p.it = (int)it;
    if (!p.vec)  // compiled for 1, 2, 4, 8 and 16
      for (p.it = 1; p.it < it; p.it *= 2) {
      }
    return p;
  }
  p.tpr = kThreads;
  p.it = 0;
  return p;
}

// Most workgroups of the backward pass, each with partial sums of its own (1024: dX
// as fast, the sums' way through memory twice as long).
constexpr int64_t kBwdGroups = 512;
constexpr int64_t kRowGroups = 2048;  // of the forward pass: 8 of 256 threads to a CU

int64_t bwd_groups(int64_t S, const LnPlan& p) {
  const int64_t rpb = p.tpr < kThreads ? kThreads / p.tpr : 1;
  const int64_t n = (S + rpb - 1) / rpb;
  return n < kBwdGroups ? n : kBwdGroups;
}

template <typename T, int VEC, typename F>
void dispatch(const LnPlan& p, F f) {
  auto with = [&](auto tpr) {
    auto it = [&](auto n) {
      if (p.tpr == decltype(tpr)::value && p.it == decltype(n)::value) f(tpr, n);
    };
    // what ln_plan can ask for: longer rows begin where the smaller group's end
    constexpr int TPR = decltype(tpr)::value;
    constexpr bool V = VEC > 1;
    if constexpr (V ? TPR <= 256 : TPR == 64) it(std::integral_constant<int, 1>{});
    if constexpr (V ? TPR == 256 : TPR <= 256) it(std::integral_constant<int, 2>{});
    if constexpr (V && TPR >= 256) it(std::integral_constant<int, 3>{});
    if constexpr (V ? TPR >= 256 : TPR <= 256) it(std::integral_constant<int, 4>{});
    if constexpr (!V && TPR == 256) it(std::integral_constant<int, 8>{});
    if constexpr (!V && TPR >= 256) it(std::integral_constant<int, 16>{});
  };
  with(std::integral_constant<int, 64>{});
  with(std::integral_constant<int, 256>{});
  with(std::integral_constant<int, 512>{});
}

// Workgroups over n rows; the kernels walk over further rows.
unsigned row_grid(int64_t n) { return (unsigned)(n < kRowGroups ? n : kRowGroups); }

template <typename T, int VEC>
void forward_t(const LnPlan& p, int64_t S, int64_t H, const T* X, const T* gamma, const T* beta,
               float eps, T* Y, float* mean, float* rstd, hipStream_t st) {
  if (p.it == 0) {
    ln_fwd_long_kernel<T, VEC><<<row_grid(S), kThreads, 0, st>>>(S, H, X, gamma, beta, eps, Y,
                                                                mean, rstd);
    return;
  }
  dispatch<T, VEC>(p, [&](auto tpr, auto it) {
    constexpr int TPR = decltype(tpr)::value, NT = group_threads<TPR>(), RPB = NT / TPR;
    ln_fwd_kernel<T, VEC, TPR, decltype(it)::value>
        <<<row_grid((S + RPB - 1) / RPB), NT, 0, st>>>(S, H, X, gamma, beta, eps, Y, mean, rstd);
  });
}

template <typename T, int VEC>
void backward_t(const LnPlan& p, int64_t S, int64_t H, const T* dY, const T* X, const T* gamma,
                const float* mean, const float* rstd, T* dX, float* part, int64_t groups,
                hipStream_t st) {
  if (p.it == 0) {
    ln_bwd_long_kernel<T, VEC>
        <<<row_grid(S), kThreads, 0, st>>>(S, H, dY, X, gamma, mean, rstd, dX);
    if (part)
      ln_cols_kernel<T><<<dim3((unsigned)((H + kThreads - 1) / kThreads), (unsigned)groups),
                          kThreads, 0, st>>>(S, H, dY, X, mean, rstd, part);
    return;
  }
  dispatch<T, VEC>(p, [&](auto tpr, auto it) {
    constexpr int TPR = decltype(tpr)::value;
    ln_bwd_kernel<T, VEC, TPR, decltype(it)::value>
        <<<(unsigned)groups, group_threads<TPR>(), 0, st>>>(S, H, dY, X, gamma, mean, rstd, dX,
                                                            part);
  });
}

moe_status check_ln(int64_t S, int64_t H, int32_t dtype) {
  if (S < 0 || H < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (dtype == MOE_MXFP8) return MOE_ERR_UNSUPPORTED;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  // the column sums' launch: 32 H threads, below 2^32
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
    constexpr int V = 16 / (int)sizeof(T);
    auto call = [&](auto vec) {
      forward_t<T, decltype(vec)::value>(p, S, H, (const T*)X, (const T*)gamma, (const T*)beta,
                                         eps, (T*)Y, mean, rstd, (hipStream_t)stream);
    };
    if (p.vec)
      call(std::integral_constant<int, V>{});
    else
      call(std::integral_constant<int, 1>{});
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
      constexpr int V = 16 / (int)sizeof(T);
      auto call = [&](auto vec) {
        backward_t<T, decltype(vec)::value>(p, S, H, (const T*)dY, (const T*)X, (const T*)gamma,
                                            mean, rstd, (T*)dX, part, groups,
                                            (hipStream_t)stream);
      };
      if (p.vec)
        call(std::integral_constant<int, V>{});
      else
        call(std::integral_constant<int, 1>{});
    };
    if (dtype == MOE_F32)
      go(float{});
    else
      go(bf16_t{});
  }
  if (dgamma != nullptr)
    ln_reduce_kernel<<<(unsigned)((2 * H + 63) / 64), 1024, 0, (hipStream_t)stream>>>(
        S > 0 ? groups : 0, H, part, dgamma, dbeta);
  return enqueued();
}
