// Norms after and before a block, with the block's gate, the residual sum and the coding of the
// normed rows, and their backward pass.
//
// Row t of the forward pass (sums in fp32, rms(v) = sqrt(mean(v^2) + eps)):
//   z = y / rms(y) * w_post;   h = x + scale * g * z;   n = h / rms(h) * w_pre;   q = codes of n
// and of the backward pass (hh = h / rms(h), yh = y / rms(y)):
//   e = dh + (w_pre dn - hh mean(w_pre dn hh)) / rms(h);   dx = e
//   dz = scale g e;   dg = scale z e;   dy = (w_post dz - yh mean(w_post dz yh)) / rms(y)
//   dw_pre = sum_t dn hh;   dw_post = sum_t dz yh
//
// Both are bound by the bytes of their rows: a row is read once, kept in registers through its
// two or three dependent sums, and written once.  W waves take a row together, 8 elements a lane
// and chunk.  The backward pass computes h again from x and y (the same bytes as reading h, and h
// in bf16 would carry its rounding into the gradients); its sums over rows are kept in registers
// over the rows a workgroup takes, written as partial sums and added in a fixed order by a second
// launch, so that the gradients do not depend on timing.
//
// Measured on MI355X (medians of traced launches; a 2 GiB copy runs at 4.9 TB/s): forward 8192 x 3584 bf16,
// gate per token, 57 us with fp8 codes (265 MB, 54 us at the copy's rate), 48 with fp4 and 50 with int8 codes;
// 4096 x 3584 with an fp32 stream 38 us (176 MB), one row 3.2 us; backward 4096 x 3584, fp32 stream, gate per
// channel 50 us and 4.7 for the partial sums (264 MB).  Widths that 8 does not divide: 8192 x 3585 with a
// sigmoid gate per element 72 us (54 at 3584), its backward pass 134 (110); 4096 x 8191 backward 157.
// Rows of more than 8192 elements fill a lane's 128 registers in the backward pass (17 to 21 spilled with a
// gate per channel or element, 28 where 8 does not divide the width): 1000 x 12000 bf16 65 us with a sigmoid
// gate per channel, 78 per element, 49 without a gate.
#include "moe_kernels.h"
#include "moe_rows.h"

#include <type_traits>

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
// sigmoid with the rounding of the exponent's product and of the reciprocal taken back (2 ulp); 0 or 1
// where the exponent leaves the range (infinities too), NaN of NaN
__device__ __forceinline__ float sigmoid_f(float x) {
  constexpr float L2E = 1.4426950408889634f, L2E_LOW = 1.92596299e-8f;
  const float p = -L2E * x;
  const float t = p > 126.0f ? 126.0f : p;                    // a comparison: fminf would lose NaN
  const float low = __builtin_fmaf(-L2E, x, -t) - L2E_LOW * x;
  const float e = __builtin_amdgcn_exp2f(t);
  const float d = 1.0f + (t < 126.0f && t > -126.0f ? __builtin_fmaf(e, low * 0.6931472f, e) : e);
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r);
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

// The sigmoid and its slope.  With p = sigmoid(-|x|) <= 1/2 the slope is p (1 - p) on both sides; from s
// alone, s (1 - s) loses its digits where s is next to 1 (4e-5 of the slope at x = 8) and is 0 from 17 on.
__device__ __forceinline__ float sigmoid_slope(float x, float& slope) {
  const float p = sigmoid_f(-__builtin_fabsf(x));
  slope = __builtin_fmaf(-p, p, p);
  return x > 0.0f ? 1.0f - p : p;
}
// Both in one register: p with the sign of -x, and from it the slope and, with one = 1, the sigmoid.
__device__ __forceinline__ float signed_sigmoid(float x) {
  return __builtin_copysignf(sigmoid_f(-__builtin_fabsf(x)), -x);
}
__device__ __forceinline__ float signed_slope(float c) {
  const float p = __builtin_fabsf(c);
  return __builtin_fmaf(-p, p, p);
}
__device__ __forceinline__ float signed_value(float c, float one) { return c + (__float_as_int(c) < 0 ? one : 0.0f); }

// The gate of this lane's VEC elements after its activation (GATE: what it is shared by), from what
// was loaded for them.  row_gate: the row's gate with MOE_GATE_TOKEN.
template <int GATE, int VEC>
__device__ __forceinline__ void gate_values(const NormArgs& a, float row_gate, float (&g)[VEC]) {
  g[0] = GATE == MOE_GATE_NONE ? 1.0f : GATE == MOE_GATE_TOKEN ? row_gate : g[0];
  constexpr int n = GATE == MOE_GATE_CHANNEL || GATE == MOE_GATE_ELEMENT ? VEC : 1;   // distinct values
  if (GATE != MOE_GATE_NONE && a.gate_act == MOE_GATE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < n; ++j) g[j] = sigmoid_f(g[j]);
  }
#pragma unroll
  for (int j = n; j < VEC; ++j) g[j] = g[0];
}
template <int GATE, int VEC>
__device__ __forceinline__ void load_gate(const NormArgs& a, int64_t base, int col, float row_gate, bool split, float (&g)[VEC]) {
  if constexpr (GATE == MOE_GATE_CHANNEL) load_own<VEC>(static_cast<const float*>(a.gate), col, a.D, split, g);
  if constexpr (GATE == MOE_GATE_ELEMENT) load_own<VEC>(static_cast<const uint16_t*>(a.gate) + base, col, a.D, split, g);
  gate_values<GATE, VEC>(a, row_gate, g);
}

// Codes of VEC = 8 consecutive elements; four adjacent lanes hold a block of 32 (inactive lanes
// of the last wave hold zeros, and D % 32 == 0, so no block is split between the two kinds).
__device__ __forceinline__ void store_mx(const float (&v)[8], const NormArgs& a, int64_t at, bool active) {
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, DPP_XOR1, 0xF, 0xF, false));
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, DPP_XOR2, 0xF, 0xF, false));
  if (!active) return;
  const bool bad = amax >= 0x7F800000u;
  uint8_t* const q = static_cast<uint8_t*>(a.q);
  int sexp;
  if (a.q_dt == MOE_DT_FP8_E4M3) {
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
  if ((at & 31) == 0) static_cast<uint8_t*>(a.q_scale)[at / 32] = (uint8_t)(bad ? 255u : (uint32_t)(sexp + 127));
}

// One row per W waves; R = blockDim.x / (64 W) rows per workgroup (R > 1 only with W == 1, so no
// barrier is ever reached by part of a workgroup).
template <int VEC, int CH, int GATE, bool SHORT, class XT>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a, int W) {
  __shared__ float red[3][MAX_W];
  const int tr = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int sub = W == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 6) + sub : blockIdx.x;
  if (row >= a.T) return;
  const int64_t base = row * a.D;
  const XT* const x = static_cast<const XT*>(a.x);
  const float inv_d = 1.0f / (float)a.D;
  const bool split = SHORT && holds_short<VEC, CH>(W, tr, a.D);
  // Lanes past the row read its last elements again and hold zeros: loads without branches, all of
  // them in flight together.
  float h[CH][VEC], y[CH][VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c) load_at<VEC>(x + base, (c * W * 64 + tr) * VEC, a.D, h[c]);
  if (a.y) {
#pragma unroll
    for (int c = 0; c < CH; ++c) load_at<VEC>(a.y + base, (c * W * 64 + tr) * VEC, a.D, y[c]);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * W * 64 + tr) * VEC;
    if (split) {
      own_part<VEC>(col, a.D, h[c]);
      if (a.y) own_part<VEC>(col, a.D, y[c]);
    }
    if (col >= a.D) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[c][j] = y[c][j] = 0.0f;
    }
  }
  if (a.y) {
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[0] += y[c][j] * y[c][j];
    float ry = 1.0f;
    if (a.w_post) {
      row_sums<1>(s, red[0], W);
      ry = rsqrt_f(s[0] * inv_d + a.eps);
      if (a.rstd_y && tr == 0) a.rstd_y[row] = ry;
    }
    const float row_gate = GATE == MOE_GATE_TOKEN ? static_cast<const float*>(a.gate)[row] : 1.0f;
    const float k = a.scale * ry;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * W * 64 + tr) * VEC;
      if (col < a.D) {
        float g[VEC], w[VEC];
        load_gate<GATE, VEC>(a, base, col, row_gate, split, g);
        if (a.w_post) {
          load_own<VEC>(a.w_post, col, a.D, split, w);
#pragma unroll
          for (int j = 0; j < VEC; ++j) y[c][j] *= w[j];
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[c][j] += k * g[j] * y[c][j];
        if (a.h) store_own<VEC>(static_cast<XT*>(a.h) + base, col, a.D, split, h[c]);
      }
    }
  } else if (a.h) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * W * 64 + tr) * VEC;
      if (col < a.D) store_own<VEC>(static_cast<XT*>(a.h) + base, col, a.D, split, h[c]);
    }
  }
  if (!a.w_pre) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += h[c][j] * h[c][j];
  row_sums<1>(s, red[1], W);
  const float rh = rsqrt_f(s[0] * inv_d + a.eps);
  if (a.rstd_h && tr == 0) a.rstd_h[row] = rh;
  uint32_t amax = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * W * 64 + tr) * VEC;
    const bool active = col < a.D;
    if (active) {
      float w[VEC];
      load_own<VEC>(a.w_pre, col, a.D, split, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[c][j] = h[c][j] * rh * w[j];
      if (a.n) store_own<VEC>(a.n + base, col, a.D, split, h[c]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[c][j] = 0.0f;
    }
    if constexpr (VEC == 8) {
      if (a.q && a.q_dt != MOE_DT_I8) store_mx(h[c], a, base + col, active);
      if (a.q && a.q_dt == MOE_DT_I8) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) amax = max(amax, __float_as_uint(h[c][j]) & 0x7FFFFFFFu);
      }
    }
  }
  if constexpr (VEC == 8) {
    if (a.q && a.q_dt == MOE_DT_I8) {
      const RowScaleI8 rs(row_max_u32(amax, red[2], W));
      if (tr == 0) static_cast<float*>(a.q_scale)[row] = rs.scale;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (c * W * 64 + tr) * VEC;
        if (col < a.D) {
          uint32_t q[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < VEC; ++j) q[j / 4] |= rs.code(h[c][j]) << (8 * (j % 4));
          *reinterpret_cast<uint2*>(el(static_cast<uint8_t*>(a.q) + base, col)) = uint2{q[0], q[1]};
        }
      }
    }
  }
}

// R rows at a time per workgroup, from blockIdx.x * R on, then every gridDim.x * R rows; all waves
// make the same number of turns, so every barrier is reached by all of them.  Each workgroup
// writes one partial row of the three sums over rows: [dw_pre | dw_post | dgate (per channel)].
template <int VEC, int CH, int GATE, bool SHORT, class XT>
__global__ __launch_bounds__(1024) void norm_backward_kernel(const NormBackwardArgs b, int W, int R) {
  __shared__ float red[2][2][2 * MAX_W];
  const NormArgs& a = b.f;
  const int sub = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) / W), first = sub * W;
  const int tr = (int)threadIdx.x - first * 64;
  const float inv_d = 1.0f / (float)a.D;
  const XT* const x = static_cast<const XT*>(a.x);
  const bool has_y = a.y != nullptr, post = a.w_post != nullptr, has_dn = b.dn != nullptr, has_dh = b.dh != nullptr;
  const bool sigmoid = a.gate_act == MOE_GATE_SIGMOID;
  constexpr bool fixed_gate = GATE == MOE_GATE_CHANNEL || GATE == MOE_GATE_NONE;
  // A sigmoid per element: gate and slope in two registers, or both in one where registers are short
  // (bf16 4096 x 3584 50 us, 54 in one; 1000 x 12000 in one 74 us with its partial sums, 83 in two)
  constexpr bool KEEP_SLOPE = GATE == MOE_GATE_ELEMENT && CH * VEC <= 8;
  constexpr bool IN_ONE = GATE == MOE_GATE_ELEMENT && !KEEP_SLOPE;
  const float one = sigmoid ? 1.0f : 0.0f;
  const bool split = SHORT && holds_short<VEC, CH>(W, tr, a.D);
  // acc_post: sum of dz yh, or with a gate per channel of scale e yh, which gives both dw_post (times
  // g) and the gate's gradient (times w_post and the activation's slope) after the last row
  float acc_pre[CH][VEC], acc_post[CH][VEC], g[CH][VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc_pre[c][j] = acc_post[c][j] = 0.0f;
    if constexpr (fixed_gate) load_gate<GATE, VEC>(a, 0, (c * W * 64 + tr) * VEC, 1.0f, split, g[c]);
  }
  // The norms' weights stay on chip: a row would wait for them once per use (three times 0.7 us).  Up
  // to 8 elements per lane in registers, else in LDS (one workgroup of 16 waves per CU as it is).
  constexpr bool IN_LDS = CH * VEC > 8;
  __shared__ float lds_w[IN_LDS ? 2 * MOE_NORM_MAX_DIM : 1];
  float w_post[IN_LDS ? 1 : CH][VEC], w_pre[IN_LDS ? 1 : CH][VEC];
  if constexpr (IN_LDS) {
    for (int i = threadIdx.x; i < ((a.D + 7) & ~7); i += blockDim.x) {   // zeros past a row's end
      lds_w[i] = i >= a.D ? 0.0f : post ? a.w_post[i] : 1.0f;
      lds_w[MOE_NORM_MAX_DIM + i] = i < a.D && has_dn ? a.w_pre[i] : 0.0f;
    }
    lds_barrier();
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * W * 64 + tr) * VEC;
      if (post) load_own<VEC>(a.w_post, col, a.D, split, w_post[c]);
      if (has_dn) load_own<VEC>(a.w_pre, col, a.D, split, w_pre[c]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        w_post[c][j] = post ? w_post[c][j] : 1.0f;
        w_pre[c][j] = has_dn ? w_pre[c][j] : 0.0f;
      }
    }
  }
  // weights of the lane's elements of chunk c (columns from `col`)
  const auto weights = [&](const float (&reg)[IN_LDS ? 1 : CH][VEC], int c, int col, int which, float (&w)[VEC]) {
    if constexpr (IN_LDS) {
      load_row<VEC>(lds_w + which * MOE_NORM_MAX_DIM + min(col, (a.D - 1) & ~(VEC - 1)), w);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) w[j] = reg[c][j];
    }
  };
  const auto gate_at = [&](int c, int j) { return IN_ONE ? signed_value(g[c][j], one) : g[c][j]; };
  int parity = 0;
  for (int64_t top = (int64_t)blockIdx.x * R; top < a.T; top += (int64_t)gridDim.x * R, parity ^= 1) {
    const bool live = top + sub < a.T;                        // else a turn without a row: zeros, no stores
    const int64_t row = live ? top + sub : a.T - 1;
    const int64_t base = row * a.D;
    // opaque, so that the compiler keeps one 32-bit offset instead of a 64-bit address per array and chunk
    int lane_at = tr * VEC;
    asm volatile("" : "+v"(lane_at));
    const float ry = post ? a.rstd_y[row] : 1.0f;
    const float rh = has_dn ? a.rstd_h[row] : 0.0f;
    const float row_gate = GATE == MOE_GATE_TOKEN ? static_cast<const float*>(a.gate)[row] : 1.0f;
    float h[CH][VEC], y[CH][VEC], u[CH][VEC], e[CH][VEC], slope[KEEP_SLOPE ? CH : 1][VEC];
    // as in the forward pass: loads without branches on the lane, all in flight together; lanes past
    // the row hold zeros in h, y, u and e
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = c * W * 64 * VEC + lane_at;
      load_at<VEC>(x + base, col, a.D, h[c]);
      if (has_y) load_at<VEC>(a.y + base, col, a.D, y[c]);
      if (has_dn) load_at<VEC>(b.dn + base, col, a.D, u[c]);
      if (has_dh) load_at<VEC>(static_cast<const XT*>(b.dh) + base, col, a.D, e[c]);
      if constexpr (GATE == MOE_GATE_ELEMENT) load_at<VEC>(static_cast<const uint16_t*>(a.gate) + base, col, a.D, g[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = c * W * 64 * VEC + lane_at;
      const bool out = col >= a.D || !live;
      if (split) {
        own_part<VEC>(col, a.D, h[c]);
        if (has_y) own_part<VEC>(col, a.D, y[c]);
        if (has_dn) own_part<VEC>(col, a.D, u[c]);
        if (has_dh) own_part<VEC>(col, a.D, e[c]);
        if constexpr (GATE == MOE_GATE_ELEMENT) own_part<VEC>(col, a.D, g[c]);
      }
      if constexpr (GATE == MOE_GATE_TOKEN) gate_values<GATE, VEC>(a, row_gate, g[c]);
      if constexpr (GATE == MOE_GATE_ELEMENT) {
        if (sigmoid) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            if constexpr (KEEP_SLOPE) g[c][j] = sigmoid_slope(g[c][j], slope[c][j]);
            else g[c][j] = signed_sigmoid(g[c][j]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        h[c][j] = out ? 0.0f : h[c][j];
        y[c][j] = out || !has_y ? 0.0f : y[c][j] * ry;        // yh (y itself without w_post)
        u[c][j] = out || !has_dn ? 0.0f : u[c][j];
        e[c][j] = out || !has_dh ? 0.0f : e[c][j];
      }
    }
    float s1[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = c * W * 64 * VEC + lane_at;
      if (has_y) {
        float w[VEC];
        weights(w_post, c, at, 0, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[c][j] += a.scale * gate_at(c, j) * (y[c][j] * w[j]);
      }
      if (has_dn) {
        float v[VEC];
        weights(w_pre, c, at, 1, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          h[c][j] *= rh;                                      // hh
          acc_pre[c][j] += u[c][j] * h[c][j];
          u[c][j] *= v[j];
          s1[0] += u[c][j] * h[c][j];
        }
      }
    }
    if (has_dn) {
      row_sums<1>(s1, red[parity][0], W, first);
      const float m = s1[0] * inv_d;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) e[c][j] += rh * (u[c][j] - h[c][j] * m);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = c * W * 64 * VEC + lane_at;
      if (live && col < a.D) store_own<VEC>(static_cast<XT*>(b.dx) + base, col, a.D, split, e[c]);
    }
    if (!has_y) continue;
    float s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = c * W * 64 * VEC + lane_at;
      float w[VEC], dg[VEC];
      weights(w_post, c, col, 0, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float se = a.scale * e[c][j];
        const float dz = se * gate_at(c, j);
        u[c][j] = dz * w[j];
        acc_post[c][j] += (GATE == MOE_GATE_CHANNEL ? se : dz) * y[c][j];
        s2[0] += u[c][j] * y[c][j];
        if constexpr (GATE == MOE_GATE_TOKEN || GATE == MOE_GATE_ELEMENT) {
          dg[j] = se * (y[c][j] * w[j]);
          if constexpr (GATE == MOE_GATE_TOKEN) s2[1] += dg[j];
          else if (sigmoid) dg[j] *= KEEP_SLOPE ? slope[c][j] : signed_slope(g[c][j]);
        }
      }
      if constexpr (GATE == MOE_GATE_ELEMENT)
        if (live && col < a.D) store_own<VEC>(static_cast<uint16_t*>(b.dgate) + base, col, a.D, split, dg);
    }
    if constexpr (GATE == MOE_GATE_TOKEN) {
      row_sums<2>(s2, red[parity][1], W, first);
      if (sigmoid) {
        float k;
        sigmoid_slope(row_gate, k);
        s2[1] *= k;
      }
      if (live && tr == 0) static_cast<float*>(b.dgate)[row] = s2[1];
    } else if (post) {
      row_sums<1>(reinterpret_cast<float(&)[1]>(s2), red[parity][1], W, first);
    }
    const float m = post ? s2[0] * inv_d : 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = c * W * 64 * VEC + lane_at;
      if (live && col < a.D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[c][j] = ry * (u[c][j] - y[c][j] * m);
        store_own<VEC>(b.dy + base, col, a.D, split, u[c]);
      }
    }
  }
  // the rows' sums of the workgroup, added in order into the first row's waves (R > 1: rows of up to
  // 16 / R waves, so the others' sums of one kind fit SPREAD floats)
  constexpr int SPREAD = CH * VEC > 8 ? 1 : 64 * MAX_W * CH * VEC;
  __shared__ float spread[SPREAD];
  float* const part = b.part + (int64_t)blockIdx.x * 3 * a.D;
  const auto finish = [&](float (&acc)[CH][VEC], float* out) {
    const int width = W * 64 * CH * VEC;
    if constexpr (SPREAD > 1) {
      if (R > 1) {
        lds_barrier();                                        // the previous kind has been read
        if (sub > 0) {
#pragma unroll
          for (int c = 0; c < CH; ++c) store_row<VEC>(spread + (sub - 1) * width + (c * W * 64 + tr) * VEC, acc[c]);
        }
        lds_barrier();
        if (sub == 0) {
          for (int r = 0; r + 1 < R; ++r)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              float v[VEC];
              load_row<VEC>(spread + r * width + (c * W * 64 + tr) * VEC, v);
#pragma unroll
              for (int j = 0; j < VEC; ++j) acc[c][j] += v[j];
            }
        }
      }
    }
    if (sub == 0) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (c * W * 64 + tr) * VEC;
        if (col < a.D) store_own<VEC>(out, col, a.D, split, acc[c]);
      }
    }
  };
  if (b.dw_pre) finish(acc_pre, part);
  if constexpr (GATE == MOE_GATE_CHANNEL) {
    float dg[CH][VEC];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * W * 64 + tr) * VEC;
      float w[VEC];
      weights(w_post, c, col, 0, w);
      if (sigmoid) {
        float raw[VEC];
        load_own<VEC>(static_cast<const float*>(a.gate), col, a.D, split, raw);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float k;
          sigmoid_slope(raw[j], k);
          w[j] *= k;
        }
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        dg[c][j] = acc_post[c][j] * w[j];
        acc_post[c][j] *= g[c][j];
      }
    }
    finish(dg, part + 2 * (int64_t)a.D);
  }
  if (b.dw_post) finish(acc_post, part + a.D);
}

// out_k[col] = sum over the partial rows, for the sums that are asked for (blockIdx.y = k).
// 64 columns x 16 row classes per workgroup; every class adds its rows in order, then the
// classes are added in order; with `add` to what out_k holds.  (16 columns x 16 classes took 12 us for
// 512 x 3 x 3584.)
__global__ __launch_bounds__(1024) void norm_sum_parts_kernel(const float* __restrict__ part, int nparts, int D, bool add,
                                                              float* dw_pre, float* dw_post, float* dgate) {
  float* const out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
  if (!out) return;
  __shared__ float lds[16][64];
  const int cl = threadIdx.x & 63, rc = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + cl;
  const float* const src = part + (int64_t)blockIdx.y * D + min(col, D - 1);
  float s = 0.0f;
#pragma unroll 8
  for (int p = rc; p < nparts; p += 16) s += src[(int64_t)p * 3 * D];
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

// f(VEC, CH, GATE, SHORT as integral constants, a value of the residual stream's type)
template <int V>
using Const = std::integral_constant<int, V>;
template <int VEC, int CH, class F>
void norm_typed(const NormArgs& a, const F& f) {
  const auto of_short = [&](auto is_short, auto xt) {
    switch (a.gate_kind) {
      case MOE_GATE_CHANNEL: f(Const<VEC>(), Const<CH>(), Const<MOE_GATE_CHANNEL>(), is_short, xt); break;
      case MOE_GATE_TOKEN: f(Const<VEC>(), Const<CH>(), Const<MOE_GATE_TOKEN>(), is_short, xt); break;
      case MOE_GATE_ELEMENT: f(Const<VEC>(), Const<CH>(), Const<MOE_GATE_ELEMENT>(), is_short, xt); break;
      default: f(Const<VEC>(), Const<CH>(), Const<MOE_GATE_NONE>(), is_short, xt); break;
    }
  };
  const auto typed = [&](auto xt) {
    if constexpr (VEC > 1) {
      if (a.D % VEC) return of_short(std::true_type(), xt);
    }
    of_short(std::false_type(), xt);
  };
  if (a.x_dt == MOE_DT_F32) typed(float());
  else typed(uint16_t());
}
template <class F>
void norm_dispatch(const NormArgs& a, const Shape& sh, const F& f) {
  if (sh.vec == 1) norm_typed<1, 1>(a, f);
  else if (sh.ch == 1) norm_typed<8, 1>(a, f);
  else norm_typed<8, 2>(a, f);
}

template <class T>
T* bytes(T* p, int64_t off) { return p ? (T*)((const uint8_t*)p + off) : p; }

// The forward call's rows t .. t + n - 1.
NormArgs rows_from(const NormArgs& a, int64_t t, int64_t n) {
  const int64_t at = t * a.D;
  NormArgs r = a;
  r.T = (int)n;
  r.x = bytes(a.x, at * (a.x_dt == MOE_DT_F32 ? 4 : 2));
  r.h = bytes(a.h, at * (a.x_dt == MOE_DT_F32 ? 4 : 2));
  r.y = bytes(a.y, at * 2);
  r.n = bytes(a.n, at * 2);
  r.gate = bytes(a.gate, a.gate_kind == MOE_GATE_TOKEN ? t * 4 : a.gate_kind == MOE_GATE_ELEMENT ? at * 2 : 0);
  r.q = bytes(a.q, a.q_dt == MOE_DT_FP4_E2M1 ? at / 2 : at);
  r.q_scale = bytes(a.q_scale, a.q_dt == MOE_DT_I8 ? t * 4 : at / 32);
  r.rstd_y = bytes(a.rstd_y, t * 4);
  r.rstd_h = bytes(a.rstd_h, t * 4);
  return r;
}
// The backward call's.
NormBackwardArgs rows_from(const NormBackwardArgs& b, int64_t t, int64_t n) {
  const NormArgs& a = b.f;
  const int64_t at = t * a.D, wide = at * (a.x_dt == MOE_DT_F32 ? 4 : 2);
  NormBackwardArgs r = b;
  r.f = rows_from(a, t, n);
  r.dh = bytes(b.dh, wide);
  r.dn = bytes(b.dn, at * 2);
  r.dx = bytes(b.dx, wide);
  r.dy = bytes(b.dy, at * 2);
  r.dgate = bytes(b.dgate, a.gate_kind == MOE_GATE_TOKEN ? t * 4 : a.gate_kind == MOE_GATE_ELEMENT ? at * 2 : 0);
  return r;
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
  const Shape sh = norm_shape(a.D);
  const int64_t slice = MAX_ITEMS / (64 * sh.W);
  for (int64_t t = 0; t < a.T; t += slice) {
    const NormArgs part = rows_from(a, t, a.T - t < slice ? a.T - t : slice);
    const unsigned grid = (unsigned)((part.T + sh.R - 1) / sh.R);
    norm_dispatch(a, sh, [&](auto vec, auto ch, auto gate, auto is_short, auto xt) {
      norm_kernel<vec(), ch(), gate(), is_short(), decltype(xt)><<<grid, sh.threads, 0, s>>>(part, sh.W);
    });
  }
  return hipGetLastError();
}

hipError_t launch_block_norm_backward(const NormBackwardArgs& b, hipStream_t s) {
  const NormArgs& a = b.f;
  const Shape sh = norm_shape(a.D);
  // Beyond a row per workgroup, as many rows at a time as 16 waves take: fewer partial sums than
  // with more workgroups of fewer waves (4096 x 3584: 54 us, 60 with 512 workgroups; 9000 x 130: 14, 17)
  const int64_t want = ((int64_t)a.T + MOE_NORM_PARTS - 1) / MOE_NORM_PARTS;
  const int fit = sh.ch * sh.vec > 8 ? 1 : MAX_W / sh.W, R = want < fit ? (int)want : fit;
  float* const dgate = a.gate_kind == MOE_GATE_CHANNEL ? static_cast<float*>(b.dgate) : nullptr;
  // A register adds up TURNS rows at most, then the sums go to the results: the rounding of a sum over
  // rows hardly grows with their number (200000 x 3584 bf16 1.65 ms, 1.69 with 64, 1.63 in one piece).
  constexpr int TURNS = 128;
  const int64_t slice = (int64_t)TURNS * MOE_NORM_PARTS * (R > 0 ? R : 1);
  int64_t t = 0;
  do {                                                        // no rows: the sums are zero
    const NormBackwardArgs part = rows_from(b, t, a.T - t < slice ? a.T - t : slice);
    const int64_t groups = R > 0 ? ((int64_t)part.f.T + R - 1) / R : 0;
    const unsigned grid = (unsigned)(groups < MOE_NORM_PARTS ? groups : MOE_NORM_PARTS);
    if (grid > 0) {
      norm_dispatch(a, sh, [&](auto vec, auto ch, auto gate, auto is_short, auto xt) {
        norm_backward_kernel<vec(), ch(), gate(), is_short(), decltype(xt)><<<grid, 64 * sh.W * R, 0, s>>>(part, sh.W, R);
      });
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (b.dw_pre || b.dw_post || dgate)
      norm_sum_parts_kernel<<<dim3((unsigned)((a.D + 63) / 64), 3), 1024, 0, s>>>(b.part, (int)grid, a.D, t > 0, b.dw_pre,
                                                                                 b.dw_post, dgate);
    t += slice;
  } while (t < a.T);
  return hipGetLastError();
}

}  // namespace moe
