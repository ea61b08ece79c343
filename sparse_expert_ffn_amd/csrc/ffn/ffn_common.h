// Definitions shared by the operators declared in include/moe_ffn.h.
#pragma once

#include <initializer_list>

#include "moe_common.h"
#include "moe_ffn.h"

namespace moe {

inline size_t ffn_round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool ffn_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether an output (or workspace) is also an input or another output; absent ones
// (null) are not.
inline bool ffn_shared(std::initializer_list<const void*> outs,
                       std::initializer_list<const void*> ins) {
  for (const void* const* o = outs.begin(); o != outs.end(); ++o) {
    if (*o == nullptr) continue;
    for (const void* q : ins)
      if (*o == q) return true;
    for (const void* const* p = outs.begin(); p != o; ++p)
      if (*o == *p) return true;
  }
  return false;
}

// 4 consecutive floats.
__device__ __forceinline__ f32x4_t load4(const float* p) {
  return *reinterpret_cast<const f32x4_t*>(p);
}

// W consecutive elements as loaded (fp32: 4; bf16: 4 or 8), read as floats.
template <typename T, int W>
struct Pack;
template <int W>
struct Pack<float, W> {
  float f[W];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < W; i += 4)
      *reinterpret_cast<f32x4_t*>(f + i) = *reinterpret_cast<const f32x4_t*>(p + i);
  }
  __device__ __forceinline__ float get(int i) const { return f[i]; }
};
template <int W>
struct Pack<bf16_t, W> {
  uint32_t w[W / 2];
  __device__ __forceinline__ void load(const bf16_t* p) {
    if constexpr (W == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16);
}
// W consecutive elements, each rounded once, in stores of at most 16 bytes.
template <int W>
__device__ __forceinline__ void store_n(float* p, const float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 4)
    *reinterpret_cast<f32x4_t*>(p + i) = f32x4_t{v[i], v[i + 1], v[i + 2], v[i + 3]};
}
template <int W>
__device__ __forceinline__ void store_n(bf16_t* p, const float (&v)[W]) {
  if constexpr (W == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// W sums of 8-bit codes, as they are.
template <int W>
__device__ __forceinline__ void store_n(int* p, const int (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 4)
    *reinterpret_cast<int4*>(p + i) = make_int4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}

}  // namespace moe
