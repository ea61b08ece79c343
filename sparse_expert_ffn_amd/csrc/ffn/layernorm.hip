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
// A row is shared by TPR threads: a wave where its registers hold the row, else
// the workgroup. Rows too long for that are read again for each sum (they
// then come from L2).
#include "ffn_common.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Sum over the TPR threads of a row: a wave's by lane exchange, a workgroup's
// through LDS in wave order. `red` has room for 2 x (waves) x NV floats and is
// used in turn (par), so one barrier per sum is enough.
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float* red, int& par) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int o = 32; o; o >>= 1) v[i] += __shfl_xor(v[i], o);
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

// VEC consecutive elements of p as floats (VEC = 1, or 16 bytes of them).
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = to_f32<T>(p[0]);
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const Vec16<T> t = __builtin_bit_cast(Vec16<T>, w);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = to_f32<T>(t.v[i]);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    p[0] = from_f32<T>(f[0]);
  } else {
    Vec16<T> t;
#pragma unroll
    for (int i = 0; i < VEC; ++i) t.v[i] = from_f32<T>(f[i]);
    *reinterpret_cast<uint4*>(p) = __builtin_bit_cast(uint4, t);
  }
}

// Rows of at most TPR * VEC * IT elements, held in registers.
template <typename T, int VEC, int TPR, int IT>
__global__ __launch_bounds__(kThreads) void ln_fwd_kernel(int64_t S, int64_t H, const T* X,
                                                          const T* gamma, const T* beta,
                                                          float eps, T* Y, float* mean,
                                                          float* rstd) {
  constexpr int RPB = kThreads / TPR;
  __shared__ float red[2 * (TPR / 64)];
  int par = 0;
  const int t = threadIdx.x % TPR;
  // the same rows for every thread of a row's TPR: barriers stay uniform
  for (int64_t s = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; s < S;
       s += (int64_t)gridDim.x * RPB) {
    const T* x = X + s * H;
    float v[IT][VEC];
    float sum[1] = {0.f};
  #pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int64_t c = ((int64_t)i * TPR + t) * VEC;
      if (c < H) {
        load_vec<T, VEC>(x + c, v[i]);
      } else {
  #pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
      }
    }
  #pragma unroll
    for (int i = 0; i < IT; ++i)
  #pragma unroll
      for (int e = 0; e < VEC; ++e) sum[0] += v[i][e];
    row_sum<TPR, 1>(sum, red, par);
    const float m = sum[0] / (float)H;
    float sq[1] = {0.f};
  #pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int64_t c = ((int64_t)i * TPR + t) * VEC;
      if (c < H)
  #pragma unroll
        for (int e = 0; e < VEC; ++e) {
          v[i][e] -= m;
          sq[0] += v[i][e] * v[i][e];
        }
    }
    row_sum<TPR, 1>(sq, red, par);
    const float r = 1.0f / sqrtf(sq[0] / (float)H + eps);
    T* y = Y + s * H;
  #pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int64_t c = ((int64_t)i * TPR + t) * VEC;
      if (c < H) {
        float g[VEC], b[VEC], o[VEC];
        if (gamma) load_vec<T, VEC>(gamma + c, g);
        if (beta) load_vec<T, VEC>(beta + c, b);
  #pragma unroll
        for (int e = 0; e < VEC; ++e)
          o[e] = v[i][e] * r * (gamma ? g[e] : 1.f) + (beta ? b[e] : 0.f);
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
      float v[VEC];
      load_vec<T, VEC>(x + c, v);
  #pragma unroll
      for (int e = 0; e < VEC; ++e) sum[0] += v[e];
    }
    row_sum<kThreads, 1>(sum, red, par);
    const float m = sum[0] / (float)H;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      float v[VEC];
      load_vec<T, VEC>(x + c, v);
  #pragma unroll
      for (int e = 0; e < VEC; ++e) sq[0] += (v[e] - m) * (v[e] - m);
    }
    row_sum<kThreads, 1>(sq, red, par);
    const float r = 1.0f / sqrtf(sq[0] / (float)H + eps);
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      float v[VEC], g[VEC], b[VEC];
      load_vec<T, VEC>(x + c, v);
      if (gamma) load_vec<T, VEC>(gamma + c, g);
      if (beta) load_vec<T, VEC>(beta + c, b);
  #pragma unroll
      for (int e = 0; e < VEC; ++e)
        v[e] = (v[e] - m) * r * (gamma ? g[e] : 1.f) + (beta ? b[e] : 0.f);
      store_vec<T, VEC>(Y + s * H + c, v);
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
__global__ __launch_bounds__(kThreads) void ln_bwd_kernel(int64_t S, int64_t H, const T* dY,
                                                          const T* X, const T* gamma,
                                                          const float* mean, const float* rstd,
                                                          T* dX, float* part) {
  constexpr int RPB = kThreads / TPR;
  __shared__ float red[2 * 2 * (TPR / 64)];
  int par = 0;
  const int t = threadIdx.x % TPR;
  const int sub = threadIdx.x / TPR;
  float g[IT][VEC], ag[IT][VEC], ab[IT][VEC];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int64_t c = ((int64_t)i * TPR + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      g[i][e] = 1.f;
      ag[i][e] = ab[i][e] = 0.f;
    }
    if (gamma && c < H) load_vec<T, VEC>(gamma + c, g[i]);
  }
  const float inv = 1.0f / (float)H;
  for (int64_t s = (int64_t)blockIdx.x * RPB + sub; s < S; s += (int64_t)gridDim.x * RPB) {
    const float m = mean[s], r = rstd[s];
    float n[IT][VEC], d[IT][VEC];
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int64_t c = ((int64_t)i * TPR + t) * VEC;
      if (c < H) {
        load_vec<T, VEC>(X + s * H + c, n[i]);
        load_vec<T, VEC>(dY + s * H + c, d[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int64_t c = ((int64_t)i * TPR + t) * VEC;
      if (c < H)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          n[i][e] = (n[i][e] - m) * r;
          ag[i][e] += d[i][e] * n[i][e];
          ab[i][e] += d[i][e];
          d[i][e] *= g[i][e];
          sums[0] += d[i][e];
          sums[1] += d[i][e] * n[i][e];
        }
    }
    row_sum<TPR, 2>(sums, red, par);
    const float c0 = sums[0] * inv, c1 = sums[1] * inv;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int64_t c = ((int64_t)i * TPR + t) * VEC;
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
      if (c < H)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          pg[c + e] = ag[i][e];
          pg[H + c + e] = ab[i][e];
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
__global__ __launch_bounds__(kThreads) void ln_bwd_long_kernel(int64_t S, int64_t H, const T* dY, const T* X,
                                                               const T* gamma, const float* mean,
                                                               const float* rstd, T* dX) {
  __shared__ float red[2 * 2 * (kThreads / 64)];
  int par = 0;
  for (int64_t s = blockIdx.x; s < S; s += gridDim.x) {
    const float m = mean[s], r = rstd[s];
    float sums[2] = {0.f, 0.f};
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kThreads * VEC) {
      float x[VEC], d[VEC], g[VEC];
      load_vec<T, VEC>(X + s * H + c, x);
      load_vec<T, VEC>(dY + s * H + c, d);
      if (gamma) load_vec<T, VEC>(gamma + c, g);
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
      float x[VEC], d[VEC], g[VEC];
      load_vec<T, VEC>(X + s * H + c, x);
      load_vec<T, VEC>(dY + s * H + c, d);
      if (gamma) load_vec<T, VEC>(gamma + c, g);
  #pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float dg = gamma ? d[e] * g[e] : d[e];
        d[e] = r * (dg - c0 - (x[e] - m) * r * c1);
      }
      store_vec<T, VEC>(dX + s * H + c, d);
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

// dgamma, dbeta: the P partial sums of each of 2 H columns in a fixed order,
// 64 columns per workgroup, each wave a quarter of the partials.
__global__ __launch_bounds__(kThreads) void ln_reduce_kernel(int64_t P, int64_t H,
                                                             const float* part, float* dgamma,
                                                             float* dbeta) {
  __shared__ float red[kThreads / 64][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t j = (int64_t)blockIdx.x * 64 + lane;
  float a = 0.f;
  if (j < 2 * H)
    for (int64_t p = w; p < P; p += kThreads / 64) a += part[p * 2 * H + j];
  red[w][lane] = a;
  __syncthreads();
  if (w == 0 && j < 2 * H) {
#pragma unroll
    for (int q = 1; q < kThreads / 64; ++q) a += red[q][lane];
    (j < H ? dgamma[j] : dbeta[j - H]) = a;
  }
}

// Which kernel takes a row: a wave per row up to 4 vectors (or 8 elements) per
// lane, a workgroup per row up to 8 vectors (16 elements) per thread, else the
// re-reading kernels.
struct LnPlan {
  bool vec;
  int tpr, it;  // it = 0: long rows
};
LnPlan ln_plan(int64_t H, int es, bool aligned) {
  LnPlan p;
  p.vec = aligned && (H * es) % 16 == 0;
  const int64_t v = p.vec ? 16 / es : 1;
  const int wave_it = p.vec ? 4 : 8, wg_it = p.vec ? 8 : 16;
  auto pow2 = [](int64_t n) {
    int r = 1;
    while (r < n) r *= 2;
    return r;
  };
  if (H <= 64 * v * wave_it) {
    p.tpr = 64;
    p.it = pow2((H + 64 * v - 1) / (64 * v));
  } else if (H <= kThreads * v * wg_it) {
    p.tpr = kThreads;
    p.it = pow2((H + kThreads * v - 1) / (kThreads * v));
  } else {
    p.tpr = kThreads;
    p.it = 0;
  }
  return p;
}

constexpr int64_t kBwdGroups = 512;  // most workgroups of the backward pass (partial sums each)

int64_t bwd_groups(int64_t S, const LnPlan& p) {
  const int64_t rpb = kThreads / p.tpr;
  const int64_t n = (S + rpb - 1) / rpb;
  return n < kBwdGroups ? n : kBwdGroups;
}

template <typename T, int VEC, typename F>
bool dispatch(const LnPlan& p, F f) {
#define MOE_LN_CASE(TPR, IT)                                              \
  if (p.tpr == TPR && p.it == IT) {                                       \
    f(std::integral_constant<int, TPR>{}, std::integral_constant<int, IT>{}); \
    return true;                                                          \
  }
  MOE_LN_CASE(64, 1) MOE_LN_CASE(64, 2) MOE_LN_CASE(64, 4)
  if constexpr (VEC == 1) { MOE_LN_CASE(64, 8) }
  MOE_LN_CASE(256, 1) MOE_LN_CASE(256, 2) MOE_LN_CASE(256, 4) MOE_LN_CASE(256, 8)
  if constexpr (VEC == 1) { MOE_LN_CASE(256, 16) }
#undef MOE_LN_CASE
  return false;
}

// Workgroups over n rows (a launch holds fewer than 2^32 threads; the kernels
// walk over further rows).
unsigned row_grid(int64_t n) { return (unsigned)(n < (1 << 20) ? n : (1 << 20)); }

template <typename T, int VEC>
void forward_t(const LnPlan& p, int64_t S, int64_t H, const T* X, const T* gamma, const T* beta,
               float eps, T* Y, float* mean, float* rstd, hipStream_t st) {
  if (p.it == 0) {
    ln_fwd_long_kernel<T, VEC><<<row_grid(S), kThreads, 0, st>>>(S, H, X, gamma, beta, eps, Y,
                                                                mean, rstd);
    return;
  }
  dispatch<T, VEC>(p, [&](auto tpr, auto it) {
    constexpr int RPB = kThreads / decltype(tpr)::value;
    ln_fwd_kernel<T, VEC, decltype(tpr)::value, decltype(it)::value>
        <<<row_grid((S + RPB - 1) / RPB), kThreads, 0, st>>>(S, H, X, gamma, beta, eps, Y,
                                                               mean, rstd);
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
    ln_bwd_kernel<T, VEC, decltype(tpr)::value, decltype(it)::value>
        <<<(unsigned)groups, kThreads, 0, st>>>(S, H, dY, X, gamma, mean, rstd, dX, part);
  });
}

moe_status check_ln(int64_t S, int64_t H, int32_t dtype) {
  if (S < 0 || H < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (dtype == MOE_MXFP8) return MOE_ERR_UNSUPPORTED;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (S >= INT32_MAX || H >= INT32_MAX) return MOE_ERR_UNSUPPORTED;
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
  if (X == nullptr || Y == nullptr || X == Y) return MOE_ERR_INVALID_ARGUMENT;
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
                dX == nullptr || dX == dY || dX == X))
    return MOE_ERR_INVALID_ARGUMENT;
  if (dgamma != nullptr && (workspace == nullptr || dgamma == dbeta))
    return workspace == nullptr ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_ERR_INVALID_ARGUMENT;
  if (dgamma != nullptr &&
      workspace_bytes < moe_layernorm_backward_workspace_bytes(S, H, dtype))
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
    ln_reduce_kernel<<<(unsigned)((2 * H + 63) / 64), kThreads, 0, (hipStream_t)stream>>>(
        S > 0 ? groups : 0, H, part, dgamma, dbeta);
  return enqueued();
}
