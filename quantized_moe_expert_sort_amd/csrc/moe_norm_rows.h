// What the kernels of the norms share (moe_norm.hip, moe_layer_norm.hip): rows of W waves with up to 8
// elements a lane and chunk, sums over them, loads and stores of rows of any width and address, MX
// codes, and the sum of the workgroups' partial sums.
#pragma once

#include <type_traits>

#include "moe_kernels.h"
#include "moe_rows.h"

namespace moe {

namespace {

constexpr int MAX_W = 16;                     // waves of a row, at most

// Element `i` of a row whose address is wave-uniform: one 32-bit offset per lane serves every row
// (64-bit addresses per lane and row took more registers than the data).
template <class T>
__device__ __forceinline__ T* el(T* row, int i) {
  typedef std::conditional_t<std::is_const_v<T>, const char, char> byte;
  return reinterpret_cast<T*>(reinterpret_cast<byte*>(row) + (uint32_t)(i * (int)sizeof(T)));
}

// This wave's LDS accesses are done; meet the other waves.  Only LDS is exchanged here, and
// __syncthreads would also wait for the rows' stores.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Sums over a row of W waves of NV values, the waves from `first` on; buf is this reduction's own
// NV * MAX_W floats.
template <int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float* buf, int W, int first = 0) {
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = wave_sum(v[k]);
  if (W == 1) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) buf[k * MAX_W + wave] = v[k];
  }
  lds_barrier();
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float s = (lane & 15) < W ? buf[k * MAX_W + first + (lane & 15)] : 0.0f;
    s += dpp_f32<DPP_XOR1>(s);
    s += dpp_f32<DPP_XOR2>(s);
    s += dpp_f32<DPP_HALF_MIRROR>(s);
    s += dpp_f32<DPP_MIRROR>(s);
    v[k] = s;
  }
}
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v, float* buf, int W) {
  v = wave_max_u32(v);
  if (W == 1) return v;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane == 0) buf[wave] = __uint_as_float(v);
  lds_barrier();
  return row16_max_u32((lane & 15) < W ? __float_as_uint(buf[lane & 15]) : 0u);
}

// 1 / sqrt(v): the hardware's estimate (1 ulp) and one Newton step.  An error here moves a whole row,
// and with it every code of the row that is near a border.
__device__ __forceinline__ float rsqrt_f(float v) {
  const float r = __builtin_amdgcn_rsqf(v);
  const float e = __builtin_fmaf(-v * r, r, 1.0f);
  return r > 0.0f && r < INFINITY ? __builtin_fmaf(0.5f * r, e, r) : r;
}
// VEC elements of a row of D from column `col`, at any address (global memory needs no alignment).
// Where D is no multiple of 8 (SHORT) one lane's last piece is short: it reads the VEC elements that end with
// the row and moves its own down, zeros behind them (own_part, only in the wave that holds that
// piece).  Lanes past the row read the same ones, for others to replace.
// Kernels of their own for SHORT rows: with the branch on it the backward pass of whole pieces took 54 us
// instead of 51.5; single elements instead of the moved piece took 2.4 times as long at 8192 x 3585.
template <int VEC, class T>
__device__ __forceinline__ void load_at(const T* row, int col, int D, float (&v)[VEC]) {
  load_any<VEC>(el(row, min(col, D - VEC)), v);
}
// Whether this wave holds the short piece, of lane `tr` of W waves a row; the same in all its lanes.
template <int VEC, int CH>
__device__ __forceinline__ bool holds_short(int W, int tr, int D) {
  bool mine = false;
#pragma unroll
  for (int c = 0; c < CH; ++c) mine |= c * W * 64 + tr == D / 8;
  return __ballot(mine) != 0;
}
template <int VEC>
__device__ __forceinline__ void own_part(int col, int D, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const bool last = col == (D & ~7);
    const int shift = -D & 7;
#pragma unroll
    for (int b = 4; b > 0; b >>= 1)
      if (shift & b) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = !last ? v[j] : j + b < 8 ? v[(j + b) & 7] : 0.0f;
      }
  }
}
template <int VEC, class T>
__device__ __forceinline__ void load_own(const T* row, int col, int D, bool split, float (&v)[VEC]) {
  load_at<VEC>(row, col, D, v);
  if (split) own_part<VEC>(col, D, v);
}
// Stores the elements before D (col < D).
template <int VEC, class T>
__device__ __forceinline__ void store_own(T* row, int col, int D, bool split, const float (&v)[VEC]) {
  if (!split || col + VEC <= D) {
    store_any<VEC>(el(row, col), v);
  } else {
#pragma unroll
    for (int j = 0; j < VEC - 1; ++j) {
      const float one[1] = {v[j]};
      if (col + j < D) store_row<1>(el(row, col + j), one);
    }
  }
}

// Codes of VEC = 8 consecutive elements; four adjacent lanes hold a block of 32 (inactive lanes
// of the last wave hold zeros, and D % 32 == 0, so no block is split between the two kinds).
__device__ __forceinline__ void store_mx(const float (&v)[8], void* codes, void* scales, int q_dt, int64_t at, bool active) {
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, DPP_XOR1, 0xF, 0xF, false));
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, DPP_XOR2, 0xF, 0xF, false));
  if (!active) return;
  const bool bad = amax >= 0x7F800000u;
  uint8_t* const q = static_cast<uint8_t*>(codes);
  int sexp;
  if (q_dt == MOE_DT_FP8_E4M3) {
    sexp = block_sexp_any(bad ? 0u : amax, Fp8Fmt::EMAX);
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = bad ? 0u : encode_pair_fp8_hw(v[2 * j], v[2 * j + 1], sexp);
    *reinterpret_cast<uint2*>(q + at) = uint2{c[0] | (c[1] << 16), c[2] | (c[3] << 16)};
  } else {
    sexp = block_sexp_any(bad ? 0u : amax, Fp4Fmt::EMAX);
    const float scale = e8m0_scale_float(sexp);
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) word |= encode_pair_fp4_hw(v[2 * j], v[2 * j + 1], scale) << (8 * j);
    *reinterpret_cast<uint32_t*>(q + at / 2) = bad ? 0u : word;
  }
  if ((at & 31) == 0) static_cast<uint8_t*>(scales)[at / 32] = (uint8_t)(bad ? 255u : (uint32_t)(sexp + 127));
}

// out_k[col] = sum over the partial rows, for the sums that are asked for (blockIdx.y = k).
// 64 columns x 16 row classes per workgroup; every class adds its rows in order, then the
// classes are added in order; with `add` to what out_k holds.  (16 columns x 16 classes took 12 us for
// 512 x 3 x 3584.)
__global__ __launch_bounds__(1024) void norm_sum_parts_kernel(const float* __restrict__ part, int nparts, int kinds, int D,
                                                              bool add, float* out_0, float* out_1, float* out_2) {
  float* const out = blockIdx.y == 0 ? out_0 : blockIdx.y == 1 ? out_1 : out_2;
  if (!out) return;
  __shared__ float lds[16][64];
  const int cl = threadIdx.x & 63, rc = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + cl;
  const float* const src = part + (int64_t)blockIdx.y * D + min(col, D - 1);
  float s = 0.0f;
#pragma unroll 8
  for (int p = rc; p < nparts; p += 16) s += src[(int64_t)p * kinds * D];
  lds[rc][cl] = s;
  __syncthreads();
  if (rc == 0 && col < D) {
    for (int i = 1; i < 16; ++i) s += lds[i][cl];
    out[col] = add ? out[col] + s : s;
  }
}

// 8 elements per lane and access in one or two chunks, as 16 waves hold them; one element in rows
// of fewer than 8.
struct Shape { int vec, ch, W, threads, R; };
Shape norm_shape(int D) {
  Shape s;
  s.vec = D < 8 ? 1 : 8;
  s.ch = D <= MAX_W * 512 ? 1 : 2;
  const int per_wave = 64 * s.vec * s.ch;
  s.W = (D + per_wave - 1) / per_wave;
  s.R = s.W == 1 ? 4 : 1;
  s.threads = 64 * s.W * s.R;
  return s;
}

template <class T>
T* bytes(T* p, int64_t off) { return p ? (T*)((const uint8_t*)p + off) : p; }

}  // namespace

}  // namespace moe
