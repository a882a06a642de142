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
#include "moe_kernels.h"
#include "moe_rows.h"

namespace moe {

namespace {

constexpr int MAX_W = 16;                     // waves of a row, at most

// Sums over a row of W waves of NV values; buf is this reduction's own NV * MAX_W floats.
template <int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float* buf, int W) {
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = wave_sum(v[k]);
  if (W == 1) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) buf[k * MAX_W + wave] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float s = (lane & 15) < W ? buf[k * MAX_W + (lane & 15)] : 0.0f;
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
  __syncthreads();
  return row16_max_u32((lane & 15) < W ? __float_as_uint(buf[lane & 15]) : 0u);
}

__device__ __forceinline__ float gate_value(float g, int act) {
  return act == MOE_GATE_SIGMOID ? fast_sigmoid(g) : g;
}

// The gate of this lane's VEC elements (columns from `col`), before its activation; ones without one.
template <int VEC>
__device__ __forceinline__ void load_gate(const NormArgs& a, int64_t at, int col, float token_gate, float (&g)[VEC]) {
  if (a.gate_kind == MOE_GATE_CHANNEL) {
    load_row<VEC>(static_cast<const float*>(a.gate) + col, g);
  } else if (a.gate_kind == MOE_GATE_ELEMENT) {
    load_row<VEC>(static_cast<const uint16_t*>(a.gate) + at, g);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) g[j] = token_gate;          // MOE_GATE_TOKEN, or 1
  }
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
template <int VEC, int CH, class XT>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a, int W) {
  __shared__ float red[3][MAX_W];
  const int tr = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6) : blockIdx.x;
  if (row >= a.T) return;
  const int64_t base = row * a.D;
  const XT* const x = static_cast<const XT*>(a.x);
  const float inv_d = 1.0f / (float)a.D;
  float h[CH][VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * W * 64 + tr) * VEC;
    if (col < a.D) {
      load_row<VEC>(x + base + col, h[c]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[c][j] = 0.0f;
    }
  }
  if (a.y) {
    float y[CH][VEC];
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * W * 64 + tr) * VEC;
      if (col < a.D) {
        load_row<VEC>(a.y + base + col, y[c]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[0] += y[c][j] * y[c][j];
      }
    }
    float ry = 1.0f;
    if (a.w_post) {
      row_sums<1>(s, red[0], W);
      ry = __builtin_amdgcn_rsqf(s[0] * inv_d + a.eps);
      if (a.rstd && tr == 0) a.rstd[row] = ry;
    }
    const float token_gate = a.gate_kind == MOE_GATE_TOKEN ? static_cast<const float*>(a.gate)[row] : 1.0f;
    const float k = a.scale * ry;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * W * 64 + tr) * VEC;
      if (col < a.D) {
        float g[VEC], w[VEC];
        load_gate<VEC>(a, base + col, col, token_gate, g);
        if (a.w_post) load_row<VEC>(a.w_post + col, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          h[c][j] += k * gate_value(g[j], a.gate_act) * (a.w_post ? y[c][j] * w[j] : y[c][j]);
        if (a.h) store_row<VEC>(static_cast<XT*>(a.h) + base + col, h[c]);
      }
    }
  } else if (a.h) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * W * 64 + tr) * VEC;
      if (col < a.D) store_row<VEC>(static_cast<XT*>(a.h) + base + col, h[c]);
    }
  }
  if (!a.w_pre) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += h[c][j] * h[c][j];
  row_sums<1>(s, red[1], W);
  const float rh = __builtin_amdgcn_rsqf(s[0] * inv_d + a.eps);
  if (a.rstd && tr == 0) a.rstd[a.T + row] = rh;
  uint32_t amax = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * W * 64 + tr) * VEC;
    const bool active = col < a.D;
    if (active) {
      float w[VEC];
      load_row<VEC>(a.w_pre + col, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[c][j] = h[c][j] * rh * w[j];
      if (a.n) store_row<VEC>(a.n + base + col, h[c]);
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
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.q) + base + col) = uint2{q[0], q[1]};
        }
      }
    }
  }
}

// Rows blockIdx.x * R + sub, then every gridDim.x * R rows.  Each (workgroup, sub) writes one
// partial row of the three sums over rows: [dw_pre | dw_post | dgate (per channel)].
template <int VEC, int CH, class XT>
__global__ __launch_bounds__(1024) void norm_backward_kernel(const NormBackwardArgs b, int W) {
  __shared__ float red[2][2][2 * MAX_W];
  const NormArgs& a = b.f;
  const int R = W == 1 ? blockDim.x >> 6 : 1, sub = W == 1 ? threadIdx.x >> 6 : 0;
  const int tr = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const float inv_d = 1.0f / (float)a.D;
  const XT* const x = static_cast<const XT*>(a.x);
  const bool token = a.gate_kind == MOE_GATE_TOKEN, element = a.gate_kind == MOE_GATE_ELEMENT;
  float acc_pre[CH][VEC], acc_post[CH][VEC], acc_gate[CH][VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc_pre[c][j] = acc_post[c][j] = acc_gate[c][j] = 0.0f;
  int parity = 0;
  for (int64_t row = (int64_t)blockIdx.x * R + sub; row < a.T; row += (int64_t)gridDim.x * R, parity ^= 1) {
    const int64_t base = row * a.D;
    const float ry = a.w_post ? a.rstd[row] : 1.0f;
    const float token_gate = token ? static_cast<const float*>(a.gate)[row] : 1.0f;
    float h[CH][VEC], y[CH][VEC], g[CH][VEC], u[CH][VEC], e[CH][VEC];
    float s1[1] = {0.0f};
    const float rh = a.w_pre ? a.rstd[a.T + row] : 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * W * 64 + tr) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[c][j] = y[c][j] = g[c][j] = u[c][j] = e[c][j] = 0.0f;
      if (col < a.D) {
        load_row<VEC>(x + base + col, h[c]);
        if (a.y) {
          load_row<VEC>(a.y + base + col, y[c]);
          load_gate<VEC>(a, base + col, col, token_gate, g[c]);
        }
        if (b.dn) load_row<VEC>(b.dn + base + col, u[c]);
        if (b.dh) load_row<VEC>(static_cast<const XT*>(b.dh) + base + col, e[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * W * 64 + tr) * VEC;
      if (col < a.D) {
        float w[VEC], v[VEC];
        if (a.y) {
          if (a.w_post) load_row<VEC>(a.w_post + col, w);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            y[c][j] *= ry;                                    // yh (y itself without w_post)
            h[c][j] += a.scale * gate_value(g[c][j], a.gate_act) * (a.w_post ? y[c][j] * w[j] : y[c][j]);
          }
        }
        if (b.dn) {
          load_row<VEC>(a.w_pre + col, v);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            h[c][j] *= rh;                                    // hh
            acc_pre[c][j] += u[c][j] * h[c][j];
            u[c][j] *= v[j];
            s1[0] += u[c][j] * h[c][j];
          }
        }
      }
    }
    if (b.dn) {
      row_sums<1>(s1, red[parity][0], W);
      const float m = s1[0] * inv_d;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) e[c][j] += rh * (u[c][j] - h[c][j] * m);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * W * 64 + tr) * VEC;
      if (col < a.D) store_row<VEC>(static_cast<XT*>(b.dx) + base + col, e[c]);
    }
    if (a.y) {
      float s2[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (c * W * 64 + tr) * VEC;
        if (col < a.D) {
          float w[VEC], dg[VEC];
          if (a.w_post) load_row<VEC>(a.w_post + col, w);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float gv = gate_value(g[c][j], a.gate_act);
            const float se = a.scale * e[c][j];
            const float z = a.w_post ? y[c][j] * w[j] : y[c][j];
            dg[j] = se * z * (a.gate_act == MOE_GATE_SIGMOID ? gv * (1.0f - gv) : 1.0f);
            const float dz = se * gv;
            u[c][j] = a.w_post ? dz * w[j] : dz;
            acc_post[c][j] += dz * y[c][j];
            acc_gate[c][j] += dg[j];
            s2[0] += u[c][j] * y[c][j];
            s2[1] += dg[j];
          }
          if (element) store_row<VEC>(static_cast<uint16_t*>(b.dgate) + base + col, dg);
        }
      }
      if (a.w_post || token) row_sums<2>(s2, red[parity][1], W);
      if (token && tr == 0) static_cast<float*>(b.dgate)[row] = s2[1];
      const float m = a.w_post ? s2[0] * inv_d : 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (c * W * 64 + tr) * VEC;
        if (col < a.D) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) u[c][j] = ry * (u[c][j] - y[c][j] * m);
          store_row<VEC>(b.dy + base + col, u[c]);
        }
      }
    }
  }
  float* const part = b.part + ((int64_t)blockIdx.x * R + sub) * 3 * a.D;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * W * 64 + tr) * VEC;
    if (col < a.D) {
      if (b.dw_pre) store_row<VEC>(part + col, acc_pre[c]);
      if (b.dw_post) store_row<VEC>(part + a.D + col, acc_post[c]);
      if (a.gate_kind == MOE_GATE_CHANNEL) store_row<VEC>(part + 2 * (int64_t)a.D + col, acc_gate[c]);
    }
  }
}

// out_k[col] = sum over the partial rows, for the sums that are asked for (blockIdx.y = k).
// 16 columns x 16 row classes per workgroup; every class adds its rows in order, then the
// classes are added in order.
__global__ __launch_bounds__(256) void norm_sum_parts_kernel(const float* __restrict__ part, int nparts, int D,
                                                             float* dw_pre, float* dw_post, float* dgate) {
  float* const out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
  if (!out) return;
  __shared__ float lds[16][17];
  const int cl = threadIdx.x & 15, rc = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + cl;
  float s = 0.0f;
  if (col < D)
    for (int p = rc; p < nparts; p += 16) s += part[((int64_t)p * 3 + blockIdx.y) * D + col];
  lds[rc][cl] = s;
  __syncthreads();
  if (rc == 0 && col < D) {
    for (int i = 1; i < 16; ++i) s += lds[i][cl];
    out[col] = s;
  }
}

// Whether every row of every given tensor can be read 16 bytes at a time.
bool aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((uintptr_t)p & 15) return false;
  return true;
}

struct Shape { int vec, ch, W, threads, R; };
// 8 elements per lane where rows and pointers allow it (else one), in as few chunks as 16 waves hold.
Shape norm_shape(int D, bool wide) {
  Shape s;
  s.vec = wide ? 8 : 1;
  const int per_wave = 64 * s.vec;
  s.ch = wide ? (D > MAX_W * per_wave ? 2 : 1) : (D > 4 * MAX_W * per_wave ? 16 : 4);
  s.W = (D + per_wave * s.ch - 1) / (per_wave * s.ch);
  s.R = s.W == 1 ? 4 : 1;
  s.threads = 64 * s.W * s.R;
  return s;
}

template <class XT>
void norm_forward(const NormArgs& a, const Shape& sh, hipStream_t s) {
  const unsigned grid = (unsigned)((a.T + sh.R - 1) / sh.R);
  if (sh.vec == 8 && sh.ch == 1) norm_kernel<8, 1, XT><<<grid, sh.threads, 0, s>>>(a, sh.W);
  else if (sh.vec == 8) norm_kernel<8, 2, XT><<<grid, sh.threads, 0, s>>>(a, sh.W);
  else if (sh.ch == 4) norm_kernel<1, 4, XT><<<grid, sh.threads, 0, s>>>(a, sh.W);
  else norm_kernel<1, 16, XT><<<grid, sh.threads, 0, s>>>(a, sh.W);
}

template <class XT>
void norm_backward(const NormBackwardArgs& b, const Shape& sh, unsigned grid, hipStream_t s) {
  if (sh.vec == 8 && sh.ch == 1) norm_backward_kernel<8, 1, XT><<<grid, sh.threads, 0, s>>>(b, sh.W);
  else if (sh.vec == 8) norm_backward_kernel<8, 2, XT><<<grid, sh.threads, 0, s>>>(b, sh.W);
  else if (sh.ch == 4) norm_backward_kernel<1, 4, XT><<<grid, sh.threads, 0, s>>>(b, sh.W);
  else norm_backward_kernel<1, 16, XT><<<grid, sh.threads, 0, s>>>(b, sh.W);
}

const void* wide_gate(const NormArgs& a) { return a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate; }

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
  const bool wide = a.D % 8 == 0 && aligned16({a.x, a.y, a.w_post, wide_gate(a), a.w_pre, a.h, a.n, a.q});
  const Shape sh = norm_shape(a.D, wide);
  if (a.x_dt == MOE_DT_F32) norm_forward<float>(a, sh, s);
  else norm_forward<uint16_t>(a, sh, s);
  return hipGetLastError();
}

hipError_t launch_block_norm_backward(const NormBackwardArgs& b, hipStream_t s) {
  const NormArgs& a = b.f;
  const bool wide = a.D % 8 == 0 && aligned16({a.x, a.y, a.w_post, wide_gate(a), a.w_pre, b.dh, b.dn, b.dx, b.dy,
                                               a.gate_kind == MOE_GATE_ELEMENT ? b.dgate : nullptr, b.part});
  const Shape sh = norm_shape(a.D, wide);
  const int groups = (a.T + sh.R - 1) / sh.R, most = MOE_NORM_PARTS / sh.R;
  const unsigned grid = (unsigned)(groups < most ? groups : most);
  if (grid > 0) {                                             // no rows: the sums below are zero
    if (a.x_dt == MOE_DT_F32) norm_backward<float>(b, sh, grid, s);
    else norm_backward<uint16_t>(b, sh, grid, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  float* const dgate = a.gate_kind == MOE_GATE_CHANNEL ? static_cast<float*>(b.dgate) : nullptr;
  if (!b.dw_pre && !b.dw_post && !dgate) return hipSuccess;
  norm_sum_parts_kernel<<<dim3((unsigned)((a.D + 15) / 16), 3), 256, 0, s>>>(b.part, (int)grid * sh.R, a.D, b.dw_pre,
                                                                            b.dw_post, dgate);
  return hipGetLastError();
}

}  // namespace moe
