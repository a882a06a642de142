// Building blocks of the kernels that take whole rows: sums and maxima over a wave, and loads
// and stores of VEC consecutive elements of a row as fp32.
#pragma once

#include "moe_device.h"

namespace moe {

// Work items of a dispatch of whole rows, at most.  A dimension holds fewer than 2^32 of them, and a
// launch of more runs what is left modulo 2^32, without an error; launchers take their rows in slices.
constexpr int64_t MAX_ITEMS = (int64_t)1 << 31;

// Lane exchanges on the VALU: quad_perm and the row mirrors inside each row of 16 lanes, then the
// two row swaps.  Every step combines a lane with one partner that does the same with it, so for a
// commutative operation all 64 lanes end with the same bits.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
enum : int { DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_HALF_MIRROR = 0x141, DPP_MIRROR = 0x140 };

template <class F>
__device__ __forceinline__ float wave_reduce(float v, F f) {
  v = f(v, dpp_f32<DPP_XOR1>(v));
  v = f(v, dpp_f32<DPP_XOR2>(v));
  v = f(v, dpp_f32<DPP_HALF_MIRROR>(v));
  v = f(v, dpp_f32<DPP_MIRROR>(v));
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(h[0]), __uint_as_float(h[1]));
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_reduce(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
// maximum of bit patterns of magnitudes (NaN above infinity)
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) { return cross_row_max_u32(row16_max_u32(v)); }

// ------------------------------------------------------------------ VEC elements of a row
//
// load_row, store_row: VEC 8 in 16-byte accesses (addresses 16-byte aligned), VEC 1 single elements.

typedef float v4f_ __attribute__((ext_vector_type(4)));
typedef uint32_t v4u_ __attribute__((ext_vector_type(4)));

template <int VEC>
__device__ __forceinline__ void load_row(const uint16_t* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const v4u_ q = *reinterpret_cast<const v4u_*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(q[j] << 16);
      v[2 * j + 1] = __uint_as_float(q[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = __uint_as_float((uint32_t)p[j] << 16);
  }
}
template <int VEC>
__device__ __forceinline__ void load_row(const float* p, float (&v)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
      const v4f_ q = reinterpret_cast<const v4f_*>(p)[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = q[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = p[j];
  }
}
// fp32 -> bf16, rounded to nearest (off by at most 2^-8 of the value)
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const v2bf r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}
template <int VEC>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    v4u_ q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<v4u_*>(p) = q;
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) p[j] = __builtin_bit_cast(uint16_t, (__bf16)v[j]);
  }
}
template <int VEC>
__device__ __forceinline__ void store_row(float* p, const float (&v)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) reinterpret_cast<v4f_*>(p)[j] = v4f_{v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) p[j] = v[j];
  }
}

// load_any, store_any: the same at any address of global memory, which needs no alignment beyond an
// element's: the hardware takes the wide accesses apart where they cross lines.
typedef float v4f_any_ __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t v4u_any_ __attribute__((ext_vector_type(4), aligned(2)));

template <int VEC>
__device__ __forceinline__ void load_any(const uint16_t* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const v4u_any_ q = *reinterpret_cast<const v4u_any_*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(q[j] << 16);
      v[2 * j + 1] = __uint_as_float(q[j] & 0xFFFF0000u);
    }
  } else {
    load_row<VEC>(p, v);
  }
}
template <int VEC>
__device__ __forceinline__ void load_any(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const v4f_any_ q = reinterpret_cast<const v4f_any_*>(p)[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = q[i];
    }
  } else {
    load_row<VEC>(p, v);
  }
}
template <int VEC>
__device__ __forceinline__ void store_any(uint16_t* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    v4u_any_ q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<v4u_any_*>(p) = q;
  } else {
    store_row<VEC>(p, v);
  }
}
template <int VEC>
__device__ __forceinline__ void store_any(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      reinterpret_cast<v4f_any_*>(p)[j] = v4f_any_{v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
  } else {
    store_row<VEC>(p, v);
  }
}

// The same elements as they are in memory, to be unpacked later: what is asked for ahead.
template <int VEC, class T>
struct RawRow {
  static constexpr int N = VEC == 8 ? 2 * (int)sizeof(T) : VEC;  // registers
  uint32_t w[N];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 8) {
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        const v4u_any_ q = reinterpret_cast<const v4u_any_*>(p)[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * k + j] = q[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) w[j] = sizeof(T) == 4 ? __float_as_uint((float)p[j]) : (uint32_t)p[j] << 16;
    }
  }
  __device__ __forceinline__ void values(float (&v)[VEC]) const {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if constexpr (VEC == 8 && sizeof(T) == 2) v[j] = __uint_as_float(j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
      else v[j] = __uint_as_float(w[j]);
    }
  }
};

// ------------------------------------------------------------------ int8 codes of a row
//
// Symmetric, one fp32 scale per row: scale = amax / 127, code = v * (127 / amax) rounded to
// nearest (ties to even), so |code| <= 127.  A row whose largest magnitude is below 2^-100 (where
// 127 / amax could overflow) has scale 0 and codes 0; a row holding Inf or NaN has scale NaN and
// codes 0.
struct RowScaleI8 {
  float scale, mul;
  __device__ __forceinline__ explicit RowScaleI8(uint32_t amax_bits) {
    const float amax = __uint_as_float(amax_bits);
    const bool bad = amax_bits >= 0x7F800000u, tiny = amax < 0x1p-100f;
    scale = bad ? __uint_as_float(0x7FC00000u) : tiny ? 0.0f : amax / 127.0f;
    mul = bad || tiny ? 0.0f : 127.0f / amax;
  }
  // a masked multiply keeps the codes of a bad row at 0 (0 * Inf would be NaN)
  __device__ __forceinline__ uint32_t code(float v) const {
    return mul == 0.0f ? 0u : (uint32_t)(uint8_t)(int8_t)(int)__builtin_rintf(__builtin_amdgcn_fmed3f(v * mul, -127.0f, 127.0f));
  }
};

}  // namespace moe
