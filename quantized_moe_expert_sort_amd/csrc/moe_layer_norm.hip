// Layer norm with the residual sum before it and the coding of its result, and its backward pass.
//
// Row t (sums in fp32, D columns):
//   h = x + y;  m = mean(h);  r = 1 / sqrt(mean((h - m)^2) + eps);  z = (h - m) r;  n = z w + b;
//   q = codes of n
// and backward (u = w dn):
//   dx = dh + r (u - mean(u) - z mean(u z));  dy = dx;  dw = sum_t dn z;  db = sum_t dn
//
// The variance is taken from the deviations from the mean, in a second sum over the registers: as
// mean(h^2) - m^2 it would lose its digits where the mean is large beside it.  Bound by the bytes of the rows, like the
// norms of moe_norm.hip, and laid out like them: a row is read once, held in registers through its
// sums, written once; the backward pass computes h again from x and y, and writes its sums over rows
// as partial sums, which a second launch adds in a fixed order.
//
// Measured on MI355X (medians of traced launches; a 2 GiB copy runs at 4.9 TB/s): forward 8192 x 3584 bf16 with y
// 41 us (235 MB, 48 us at the copy's rate: a part stays in the last-level cache), 4096 x 3584 with an fp32 stream
// 36 us (176 MB, 4.9 TB/s), one row 2.7 us; with codes instead of n 8192 x 3584 bf16 fp8 43 us (206 MB, 4.8 TB/s),
// fp4 41, int8 45 (one reduction more, of the row's largest value), 4096 x 3584 fp32 fp8 32 us (162 MB, 5.0 TB/s);
// backward 4096 x 3584 fp32 46 us (x, y, dn, dh, dx and dy: 264 MB, 5.7 TB/s, above the copy's rate with the
// last-level cache's part) and 4.7 for the partial sums; 1000 x 12000 bf16 47 to 49 us (144 MB, 3.0 TB/s: one workgroup
// of 12 waves a CU, whose loads, sums and stores follow one another, in 128 registers with 3 to 14 more in
// scratch); 777 x 1790 bf16 5.1, 7.7 and 4.
#include "moe_norm_rows.h"

namespace moe {

namespace {

// One row per W waves; R = blockDim.x / (64 W) rows per workgroup (R > 1 only with W == 1, so no
// barrier is ever reached by part of a workgroup).
template <int VEC, int CH, bool SHORT, class XT>
__global__ __launch_bounds__(1024) void layer_norm_kernel(const LayerNormArgs a, int W) {
  __shared__ float red[3][2 * MAX_W];
  const int tr = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int sub = W == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 6) + sub : blockIdx.x;
  if (row >= a.T) return;
  const int64_t base = row * a.D;
  const float inv_d = 1.0f / (float)a.D;
  const bool split = SHORT && holds_short<VEC, CH>(W, tr, a.D);
  // Lanes past the row read its last elements again and hold zeros: loads without branches, all of
  // them in flight together.
  float h[CH][VEC], y[CH][VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c) load_at<VEC>(static_cast<const XT*>(a.x) + base, (c * W * 64 + tr) * VEC, a.D, h[c]);
  if (a.y) {
#pragma unroll
    for (int c = 0; c < CH; ++c) load_at<VEC>(a.y + base, (c * W * 64 + tr) * VEC, a.D, y[c]);
  }
  float s[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * W * 64 + tr) * VEC;
    if (a.y) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[c][j] += y[c][j];
    }
    if (split) own_part<VEC>(col, a.D, h[c]);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      h[c][j] = col < a.D ? h[c][j] : 0.0f;
      s[0] += h[c][j];
    }
    if (a.h && col < a.D) store_own<VEC>(static_cast<XT*>(a.h) + base, col, a.D, split, h[c]);
  }
  if (!a.n && !a.q && !a.mean) return;
  row_sums<1>(s, red[0], W);
  const float m = s[0] * inv_d;
  // The deviations' own mean takes back the rounding of m, which a mean of 1e4 deviations would show
  // (2e-3 of a deviation).
  float d[2] = {0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * W * 64 + tr) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      h[c][j] = (SHORT ? col + j : col) < a.D ? h[c][j] - m : 0.0f;
      d[0] += h[c][j];
      d[1] += h[c][j] * h[c][j];
    }
  }
  row_sums<2>(d, red[1], W);
  const float m2 = d[0] * inv_d;
  const float r = rsqrt_f(__builtin_fmaxf(__builtin_fmaf(-m2, m2, d[1] * inv_d), d[1] * 0.0f) + a.eps);
  if (a.mean && tr == 0) {
    a.mean[row] = m + m2;
    a.rstd[row] = r;
  }
  if (!a.n && !a.q) return;
  uint32_t amax = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * W * 64 + tr) * VEC;
    const bool active = col < a.D;
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[c][j] = (h[c][j] - m2) * r;
    if (active) {
      float v[VEC];
      if (a.w) {
        load_own<VEC>(a.w, col, a.D, split, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[c][j] *= v[j];
      }
      if (a.b) {
        load_own<VEC>(a.b, col, a.D, split, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[c][j] += v[j];
      }
      if (a.n) store_own<VEC>(a.n + base, col, a.D, split, h[c]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[c][j] = 0.0f;           // not the NaN of a row that holds one
    }
    if constexpr (VEC == 8) {
      if (a.q && a.q_dt != MOE_DT_I8) store_mx(h[c], a.q, a.q_scale, a.q_dt, base + col, active);
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
// writes one partial row of the two sums over rows: [dw | db].
template <int VEC, int CH, bool SHORT, class XT>
__global__ __launch_bounds__(1024) void layer_norm_backward_kernel(const LayerNormBackwardArgs b, int W, int R) {
  __shared__ float red[2][2 * MAX_W];
  const LayerNormArgs& a = b.f;
  const int sub = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) / W), first = sub * W;
  const int tr = (int)threadIdx.x - first * 64;
  const float inv_d = 1.0f / (float)a.D;
  const bool has_y = a.y != nullptr, has_dh = b.dh != nullptr;
  const bool split = SHORT && holds_short<VEC, CH>(W, tr, a.D);
  // The weights stay on chip: up to 8 elements per lane in registers, else in LDS (one workgroup per CU as it is).
  constexpr bool IN_LDS = CH * VEC > 8;
  __shared__ float lds_w[IN_LDS ? MOE_NORM_MAX_DIM : 1];
  float acc_w[CH][VEC], acc_b[CH][VEC], w[IN_LDS ? 1 : CH][VEC];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc_w[c][j] = acc_b[c][j] = 0.0f;
  if constexpr (IN_LDS) {
    for (int i = threadIdx.x; i < ((a.D + 7) & ~7); i += blockDim.x) lds_w[i] = i >= a.D ? 0.0f : a.w ? a.w[i] : 1.0f;
    lds_barrier();
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (a.w) load_own<VEC>(a.w, (c * W * 64 + tr) * VEC, a.D, split, w[c]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) w[c][j] = a.w ? w[c][j] : 1.0f;
    }
  }
  // The next row is asked for as soon as this one is unpacked, where the registers hold both (4096 x 3584 fp32
  // 50.3 -> 46.7 us); not in wide rows, which spill without it, nor in fp32 rows with a short piece, which would.
  constexpr bool AHEAD = CH == 1 && !(SHORT && sizeof(XT) == 4);
  RawRow<VEC, XT> xr[CH], er[CH];
  RawRow<VEC, uint16_t> yr[CH], ur[CH];
  float m_next = 0.0f, r_next = 0.0f;
  // opaque, so that the compiler keeps one 32-bit offset instead of a 64-bit address per array and chunk
  int lane_at = tr * VEC;
  asm volatile("" : "+v"(lane_at));
  const auto ask = [&](int64_t row) {
    const int64_t base = row * a.D;
    m_next = a.mean[row];
    r_next = a.rstd[row];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = min(c * W * 64 * VEC + lane_at, a.D - VEC);
      xr[c].load(el(static_cast<const XT*>(a.x) + base, at));
      if (has_y) yr[c].load(el(a.y + base, at));
      ur[c].load(el(b.dn + base, at));
      if (has_dh) er[c].load(el(static_cast<const XT*>(b.dh) + base, at));
    }
  };
  int parity = 0;
  const int64_t step = (int64_t)gridDim.x * R;
  if (AHEAD) ask(min((int64_t)blockIdx.x * R + sub, (int64_t)a.T - 1));
  for (int64_t top = (int64_t)blockIdx.x * R; top < a.T; top += step, parity ^= 1) {
    const bool live = top + sub < a.T;                        // else a turn without a row: zeros, no stores
    const int64_t base = (live ? top + sub : a.T - 1) * a.D;
    if constexpr (!AHEAD) {
      asm volatile("" : "+v"(lane_at));
      m_next = a.mean[live ? top + sub : a.T - 1];
      r_next = a.rstd[live ? top + sub : a.T - 1];
    }
    const float m = m_next, r = r_next;
    float z[CH][VEC], y[CH][VEC], u[CH][VEC], e[CH][VEC];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (!AHEAD) {
        const int col = c * W * 64 * VEC + lane_at;
        load_at<VEC>(static_cast<const XT*>(a.x) + base, col, a.D, z[c]);
        if (has_y) load_at<VEC>(a.y + base, col, a.D, y[c]);
        load_at<VEC>(b.dn + base, col, a.D, u[c]);
        if (has_dh) load_at<VEC>(static_cast<const XT*>(b.dh) + base, col, a.D, e[c]);
        continue;
      }
      xr[c].values(z[c]);
      if (has_y) yr[c].values(y[c]);
      ur[c].values(u[c]);
      if (has_dh) er[c].values(e[c]);
    }
    if (AHEAD && top + step < a.T) ask(min(top + step + sub, (int64_t)a.T - 1));
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = c * W * 64 * VEC + lane_at;
      const bool out = col >= a.D || !live;
      if (has_y) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[c][j] += y[c][j];
      }
      if (split) {
        own_part<VEC>(col, a.D, z[c]);
        own_part<VEC>(col, a.D, u[c]);
        if (has_dh) own_part<VEC>(col, a.D, e[c]);
      }
      float wc[VEC];
      if constexpr (IN_LDS) {
        load_row<VEC>(lds_w + min(col, (a.D - 1) & ~(VEC - 1)), wc);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) wc[j] = w[c][j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        z[c][j] = out ? 0.0f : (z[c][j] - m) * r;             // past a short piece's end u is zero
        u[c][j] = out ? 0.0f : u[c][j];
        e[c][j] = out || !has_dh ? 0.0f : e[c][j];
        acc_w[c][j] += u[c][j] * z[c][j];
        acc_b[c][j] += u[c][j];
        u[c][j] *= wc[j];
        s[0] += u[c][j];
        s[1] += u[c][j] * z[c][j];
      }
    }
    row_sums<2>(s, red[parity], W, first);
    const float mu = s[0] * inv_d, mz = s[1] * inv_d;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = c * W * 64 * VEC + lane_at;
      if (live && col < a.D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) e[c][j] += r * (u[c][j] - mu - z[c][j] * mz);
        store_own<VEC>(static_cast<XT*>(b.dx) + base, col, a.D, split, e[c]);
        if (b.dy) store_own<VEC>(b.dy + base, col, a.D, split, e[c]);
      }
    }
  }
  // the rows' sums of the workgroup, added in order into the first row's waves (R > 1: rows of up to
  // 16 / R waves, so the others' sums of one kind fit SPREAD floats)
  constexpr int SPREAD = CH * VEC > 8 ? 1 : 64 * MAX_W * CH * VEC;
  __shared__ float spread[SPREAD];
  float* const part = b.part + (int64_t)blockIdx.x * 2 * a.D;
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
          for (int k = 0; k + 1 < R; ++k)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              float v[VEC];
              load_row<VEC>(spread + k * width + (c * W * 64 + tr) * VEC, v);
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
  if (b.dw) finish(acc_w, part);
  if (b.db) finish(acc_b, part + a.D);
}

// f(VEC, CH, SHORT as integral constants, a value of the residual stream's type)
template <int V>
using Const = std::integral_constant<int, V>;
template <class F>
void layer_norm_dispatch(const LayerNormArgs& a, const Shape& sh, const F& f) {
  const auto typed = [&](auto vec, auto ch, auto is_short) {
    if (a.x_dt == MOE_DT_F32) f(vec, ch, is_short, float());
    else f(vec, ch, is_short, uint16_t());
  };
  const auto sized = [&](auto ch) {
    if (a.D % 8) typed(Const<8>(), ch, std::true_type());
    else typed(Const<8>(), ch, std::false_type());
  };
  if (sh.vec == 1) typed(Const<1>(), Const<1>(), std::false_type());
  else if (sh.ch == 1) sized(Const<1>());
  else sized(Const<2>());
}

// The call's rows t .. t + n - 1.
LayerNormArgs rows_from(const LayerNormArgs& a, int64_t t, int64_t n) {
  const int64_t at = t * a.D, wide = at * (a.x_dt == MOE_DT_F32 ? 4 : 2);
  LayerNormArgs r = a;
  r.T = (int)n;
  r.x = bytes(a.x, wide);
  r.h = bytes(a.h, wide);
  r.y = bytes(a.y, at * 2);
  r.n = bytes(a.n, at * 2);
  r.q = bytes(a.q, a.q_dt == MOE_DT_FP4_E2M1 ? at / 2 : at);
  r.q_scale = bytes(a.q_scale, a.q_dt == MOE_DT_I8 ? t * 4 : at / 32);
  r.mean = bytes(a.mean, t * 4);
  r.rstd = bytes(a.rstd, t * 4);
  return r;
}
LayerNormBackwardArgs rows_from(const LayerNormBackwardArgs& b, int64_t t, int64_t n) {
  const int64_t at = t * b.f.D, wide = at * (b.f.x_dt == MOE_DT_F32 ? 4 : 2);
  LayerNormBackwardArgs r = b;
  r.f = rows_from(b.f, t, n);
  r.dh = bytes(b.dh, wide);
  r.dn = bytes(b.dn, at * 2);
  r.dx = bytes(b.dx, wide);
  r.dy = bytes(b.dy, at * 2);
  return r;
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s) {
  const Shape sh = norm_shape(a.D);
  const int64_t slice = MAX_ITEMS / (64 * sh.W);
  for (int64_t t = 0; t < a.T; t += slice) {
    const LayerNormArgs part = rows_from(a, t, a.T - t < slice ? a.T - t : slice);
    const unsigned grid = (unsigned)(((int64_t)part.T + sh.R - 1) / sh.R);
    layer_norm_dispatch(a, sh, [&](auto vec, auto ch, auto is_short, auto xt) {
      layer_norm_kernel<vec(), ch(), is_short(), decltype(xt)><<<grid, sh.threads, 0, s>>>(part, sh.W);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_layer_norm_backward(const LayerNormBackwardArgs& b, hipStream_t s) {
  const LayerNormArgs& a = b.f;
  const Shape sh = norm_shape(a.D);
  const int64_t want = ((int64_t)a.T + MOE_NORM_PARTS - 1) / MOE_NORM_PARTS;
  const int fit = sh.ch * sh.vec > 8 ? 1 : MAX_W / sh.W, R = want < fit ? (int)want : fit;
  // as in moe_norm.hip: a register adds up TURNS rows at most, then the sums go to the results
  constexpr int TURNS = 128;
  const int64_t slice = (int64_t)TURNS * MOE_NORM_PARTS * (R > 0 ? R : 1);
  int64_t t = 0;
  do {                                                        // no rows: the sums are zero
    const LayerNormBackwardArgs part = rows_from(b, t, a.T - t < slice ? a.T - t : slice);
    const int64_t groups = R > 0 ? ((int64_t)part.f.T + R - 1) / R : 0;
    const unsigned grid = (unsigned)(groups < MOE_NORM_PARTS ? groups : MOE_NORM_PARTS);
    if (grid > 0) {
      layer_norm_dispatch(a, sh, [&](auto vec, auto ch, auto is_short, auto xt) {
        layer_norm_backward_kernel<vec(), ch(), is_short(), decltype(xt)><<<grid, 64 * sh.W * R, 0, s>>>(part, sh.W, R);
      });
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (b.dw || b.db)
      norm_sum_parts_kernel<<<dim3((unsigned)((a.D + 63) / 64), 2), 1024, 0, s>>>(b.part, (int)grid, 2, a.D, t > 0, b.dw, b.db,
                                                                                 nullptr);
    t += slice;
  } while (t < a.T);
  return hipGetLastError();
}

}  // namespace moe
