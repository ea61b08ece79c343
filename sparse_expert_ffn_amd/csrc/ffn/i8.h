// 8-bit codes with one scale per vector: what the kernels of i8.hip and few.hip share.
//
// A vector x is quantised to q = rint(x / s), ties to even, s = max |x| / 127 rounded to
// fp32. The quotient is decided exactly: from the estimate q0 = rint(x (1 / s)), which
// is off by one at most, the remainder x - q0 s is exact in an fma (both are whole
// multiples of the smaller of their last places, and it is at most about s), and is
// compared with s / 2. So the codes do not depend on how that quotient rounds. They do on the
// scale: max |x| / 127 is the correctly rounded quotient here, and whoever rounds it so gets
// the same codes (max |x| times the rounded 1 / 127 is an ulp off in 3 to 6% of the vectors and
// moves a code now and then).
#pragma once

#include "ffn_common.h"

namespace moe {

constexpr int64_t kI8MaxK = 1 << 17;   // 127^2 K < 2^31: sums of codes' products fit
constexpr int kI8TileN = 16, kI8TileK = 64;

__host__ __device__ inline int64_t i8_tiles_k(int64_t K) { return (K + kI8TileK - 1) / kI8TileK; }
__host__ __device__ inline int64_t i8_tiles_n(int64_t N) { return (N + kI8TileN - 1) / kI8TileN; }
// A packed matrix: its tiles, then a scale for each column of them.
__host__ __device__ inline int64_t i8_code_bytes(int64_t K, int64_t N) {
  return i8_tiles_n(N) * i8_tiles_k(K) * 1024;
}
__host__ __device__ inline int64_t i8_matrix_bytes(int64_t K, int64_t N) {
  return i8_code_bytes(K, N) + i8_tiles_n(N) * kI8TileN * 4;
}

// |x| as bits: their order is that of the magnitudes, infinity and NaN on top, so that a
// maximum of them loses neither.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// A sum of products of codes times both scales. The one nearer to 0 first: the sum is a whole
// number, so nothing between overflows or leaves the normal range that the result does not.
// (A scale of NaN stays.)
__device__ __forceinline__ float scaled(int sum, float a, float b) {
  const bool a_is_more = __builtin_fabsf(a) > __builtin_fabsf(b);
  return (float)sum * (a_is_more ? b : a) * (a_is_more ? a : b);
}

struct Quant {
  float scale;         // the vector's; NaN where a value is not finite (its products are NaN)
  float f, s, inv, half;

  // top: abs_bits of the largest magnitude
  __device__ __forceinline__ explicit Quant(uint32_t top) {
    const float a = __uint_as_float(top);
    const bool finite = top < 0x7F800000u;
    scale = finite ? a / 127.0f : __uint_as_float(0x7FC00000u);
    // tiny vectors: x and s times 2^80, exactly, so that 1 / s is finite
    f = a < 0x1p-60f ? 0x1p80f : 1.0f;
    s = scale * f;
    const bool live = finite && scale > 0.f;
    inv = live ? 1.0f / s : 0.f;
    half = 0.5f * s;
  }
  __device__ __forceinline__ int operator()(float x) const {
    const float t = x * f;
    float q = rintf(t * inv);
    const float r = __builtin_fmaf(-q, s, t);
    if (__builtin_fabsf(r) >= half) {
      const float step = r < 0.f ? -1.f : 1.f;
      if (__builtin_fabsf(r) > half || ((int)q & 1)) q += step;
    }
    q = fminf(fmaxf(q, -127.f), 127.f);
    return inv > 0.f ? (int)q : 0;
  }
  // 16 values in the bytes of 4 dwords. x (1 / s) + 1.5 2^23 has the rounded quotient in its
  // low byte: where no remainder reaches s / 2 that is the code, 4 operations to a value
  // (one by one 14: the rows of 16384 x 7168 in bf16 took 70 us, their bytes take 60).
  __device__ __forceinline__ uint4 pack16(const float (&x)[16]) const {
    uint32_t d[4];
    bool sure = f == 1.0f && inv > 0.f;
    if (sure) {
      constexpr float magic = 12582912.0f;
      float worst = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float v = __builtin_fmaf(x[4 * i + j], inv, magic);
          worst = fmaxf(worst, __builtin_fabsf(__builtin_fmaf(magic - v, s, x[4 * i + j])));
          t[j] = __float_as_uint(v);
        }
        d[i] = __builtin_amdgcn_perm(t[1], t[0], 0x0C0C0400u) |
               __builtin_amdgcn_perm(t[3], t[2], 0x04000C0Cu);
      }
      sure = worst < half;
    }
    if (!sure)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[i] = pack4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    return make_uint4(d[0], d[1], d[2], d[3]);
  }
  // 4 values in the bytes of a dword
  __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) const {
    return ((uint32_t)(*this)(a) & 255u) | (((uint32_t)(*this)(b) & 255u) << 8) |
           (((uint32_t)(*this)(c) & 255u) << 16) | ((uint32_t)(*this)(d) << 24);
  }
};

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t y = (uint32_t)__shfl_xor((int)x, o, 64);
    x = x > y ? x : y;
  }
  return x;
}

// Rows of X [S][K] to codes [S][K] and scales [S] (few rows or many).
hipError_t launch_quantize_rows(const void* X, int64_t S, int64_t K, bool f32, int8_t* codes,
                                float* scales, hipStream_t st);

}  // namespace moe
