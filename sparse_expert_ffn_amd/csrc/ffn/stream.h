// Products of up to 16 rows with a weight that is read once: a wave streams 128 columns from
// memory into registers, where they become MFMA operands, with no LDS on their way. Rows of
// 256 bytes to 16 lanes (with 128 the weights of a layer of 7168 x 2048 came at 3.0 TB/s,
// with two waves side by side at 3.6, so at 4.9).
//   bf16: a lane holds 8 rows of 8 columns; byte permutes give the operands (8 rows of a
//         column) of v_mfma_f32_16x16x32_bf16
//   fp32: 4 rows of 2 x 4 columns, v_mfma_f32_16x16x4_f32 (K in an order that suits)
//   int8: packed in operand order (8 tiles of 16 columns), v_mfma_i32_16x16x64_i8
// One row or sixteen cost the same. Three steps of 8 KB ahead to a wave: with 8 waves to a CU
// 192 KB are under way (two steps or four were no faster).
#pragma once

#include <type_traits>

#include "i8.h"

namespace moe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
using rsrc_t = __amdgpu_buffer_rsrc_t;
constexpr uint32_t kPastEnd = 0x80000000u;  // above every descriptor's range
constexpr int64_t kMaxMatrix = 0x7F000000;
constexpr int kNonTemporal = 2;      // load hint: weights are read once
constexpr int kCols = 128;           // columns of a wave

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
  static constexpr int ES = 2, STEP = 32;  // bytes of a weight, K per step
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

// A wave's columns of a matrix [K][N] from n0 on.
template <int P>
struct Columns {
  rsrc_t r;
  uint32_t off, row, step;
  uint32_t past[P == kF32 ? 2 : 1];  // fp32: two halves of 64 columns, which end at N each

  __device__ __forceinline__ Columns() {}
  __device__ __forceinline__ Columns(const char* matrix, int K, int N, int n0) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    if constexpr (P == kI8) {
      const uint32_t kt = (uint32_t)i8_tiles_k(K);
      r = make_rsrc(matrix, n0 < N ? i8_code_bytes(K, N) : 0);
      off = (uint32_t)((n0 / 16) * kt) * 1024 + lane * 16;
      row = kt * 1024;
      step = 1024;
    } else {
      constexpr int ES = Kind<P>::ES;
      r = make_rsrc(matrix, (int64_t)K * N * ES);
      off = (uint32_t)((P == kBf16 ? 8 : 4) * g * N + n0 + (P == kBf16 ? 8 : 4) * c) * ES;
      if constexpr (P == kBf16) {
        if (n0 + 8 * c >= N) off = kPastEnd;
      } else {
        past[0] = n0 + 4 * c < N ? 0 : kPastEnd;
        past[1] = n0 + 64 + 4 * c < N ? 0 : kPastEnd;
      }
      row = (uint32_t)N * ES;
      step = row * Kind<P>::STEP;
    }
  }
};

template <int P>
struct Step {
  using Acc = typename Kind<P>::Acc;
  uint4 w[8];

  __device__ __forceinline__ void load(const Columns<P>& m, uint32_t o) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t at = o + i * m.row;
      if constexpr (P == kF32) at = (o + (i >> 1) * m.row + (i & 1) * 256) | m.past[i & 1];
      w[i] = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(m.r, at, 0, kNonTemporal));
    }
  }
  // Step s of the columns; from `end` on: zeros.
  __device__ __forceinline__ void load(const Columns<P>& m, int s, int end) {
    load(m, s < end ? m.off + (uint32_t)s * m.step : kPastEnd);
  }
  __device__ __forceinline__ void compute(const uint4& x, Acc (&acc)[8]) const {
    if constexpr (P == kBf16) {
      const bf16x8_t a = __builtin_bit_cast(bf16x8_t, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // column j of the lane's 8: rows 2 i and 2 i + 1 in dword i
        const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
        uint32_t d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          d[i] = __builtin_amdgcn_perm(word(w[2 * i + 1], j / 2), word(w[2 * i], j / 2), sel);
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            a, __builtin_bit_cast(bf16x8_t, make_uint4(d[0], d[1], d[2], d[3])), acc[j], 0, 0, 0);
      }
    } else if constexpr (P == kF32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(word(x, i));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
              a, __uint_as_float(word(w[2 * i + j / 4], j % 4)), acc[j], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, x),
                                                       __builtin_bit_cast(i32x4_t, w[j]), acc[j],
                                                       0, 0, 0);
    }
  }
};

// 16 rows of the other operand, 64 bytes of each per step (lane l: row l % 16, bytes 16 (l
// / 16) .. + 15); rows that are not there and what lies behind a row's end read as zeros.
struct Rows {
  rsrc_t r;
  uint32_t off;    // of this lane's row
  uint32_t bytes;  // of a row
  // step s; from `end` on: zeros
  __device__ __forceinline__ uint4 load(int s, int end) const {
    const uint32_t at = (uint32_t)s * 64 + ((threadIdx.x & 63) >> 4) * 16;
    return load16(r, s < end && at < bytes ? off + at : kPastEnd);
  }
};

// This lane's sums into LDS as rows of the wave's columns: rows 4 (l / 16) .. + 3 below n.
template <int P>
__device__ __forceinline__ void put_sums(const typename Kind<P>::Acc (&acc)[8],
                                         typename Kind<P>::Val* to, int n) {
  using Acc = typename Kind<P>::Acc;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
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

// This wave's share of K's steps below `end`: every SHARES-th from `first` on.
template <int P, int SHARES>
struct Stream {
  static constexpr int DEPTH = 3;
  Step<P> st[DEPTH];
  uint4 x[DEPTH];

  // the first loads of weights, which may go out before the rows are known
  __device__ __forceinline__ void start(const Columns<P>& m, int first, int end) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) st[d].load(m, first + d * SHARES, end);
  }
  __device__ __forceinline__ void run(const Columns<P>& m, const Rows& a, int first, int end,
                                      typename Kind<P>::Acc (&acc)[8]) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) x[d] = a.load(first + d * SHARES, end);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = typename Kind<P>::Acc{};
    for (int s = first; s < end;) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d, s += SHARES) {
        st[d].compute(x[d], acc);
        st[d].load(m, s + DEPTH * SHARES, end);
        x[d] = a.load(s + DEPTH * SHARES, end);
        __builtin_amdgcn_sched_barrier(0);  // the loads go out here, not behind the next step
      }
    }
  }
};

}  // namespace moe
