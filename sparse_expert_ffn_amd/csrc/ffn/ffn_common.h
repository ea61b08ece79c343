// Definitions shared by the operators declared in include/moe_ffn.h.
#pragma once

#include "moe_common.h"
#include "moe_ffn.h"

namespace moe {

inline size_t ffn_round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool ffn_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// 16 bytes as T elements.
template <typename T>
struct Vec16 {
  static constexpr int N = 16 / (int)sizeof(T);
  T v[N];
};

// 4 consecutive elements, as one load or store.
__device__ __forceinline__ f32x4_t load4(const float* p) {
  return *reinterpret_cast<const f32x4_t*>(p);
}
__device__ __forceinline__ f32x4_t load4(const bf16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  f32x4_t r;
  r[0] = __uint_as_float(w.x << 16);
  r[1] = __uint_as_float(w.x & 0xFFFF0000u);
  r[2] = __uint_as_float(w.y << 16);
  r[3] = __uint_as_float(w.y & 0xFFFF0000u);
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16);
}
__device__ __forceinline__ void store4(float* p, f32x4_t v) {
  *reinterpret_cast<f32x4_t*>(p) = v;
}
__device__ __forceinline__ void store4(bf16_t* p, f32x4_t v) {
  uint2 w;
  w.x = pack_bf16(v[0], v[1]);
  w.y = pack_bf16(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = w;
}

}  // namespace moe
