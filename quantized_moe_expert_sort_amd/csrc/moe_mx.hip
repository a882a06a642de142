// Microscaled coding of matrices (fp8 e4m3 or fp4 e2m1 elements, one e8m0 scale per 32) along their
// rows, along their columns (the codes of the transpose), or both from one read, and the layout of
// MXFP4 weights for the products of moe_mx_gemm.hip.
//
// Block of 32 values: s = floor(log2 max|v|) - emax, element = v / 2^s rounded to the element grid and
// saturated, as in moe_device.h.  Rounded to nearest, ties to even; or with noise n in 0 .. 255 per
// element to one of the two neighbours on the grid: in units of the element's last place,
// floor(|v| / 2^s + (2 n + 1) / 512), so that over uniform n the mean is the value (to 1/512 of a place).
//
// Rows of codes are filled up with zeros to a multiple of 128 (one K step of the product), so that
// matrices of any size can be multiplied.  Packed weights are blocks (f, s) of 16 rows x 128 columns:
// 1 KB of codes, byte 16 (16 g + r) + b = row 16 f + r, columns 128 s + 32 g + 2 b and + 1; and 64 bytes of
// scales, byte 4 r + g; s fastest; rows past the matrix are zero.
//
// Measured on MI355X (medians of traced launches; a 2 GiB copy runs at 4.9 TB/s): along the rows 8192 x 3584 bf16
// to fp4 16 us (4.7 TB/s), one row 2.2; both ways 4096 x 3584 bf16 to fp4 15.4 us (45 MB: 2.9 TB/s; the passes of a
// workgroup, load, barrier, codes, overlap only with other workgroups'), 3584 x 3584 fp32 to fp4 18 us (65 MB,
// 3.6 TB/s; 144 registers, three workgroups on a CU), 777 x 1790 fp32 8.6 us (one workgroup's latency); with noise
// 4096 x 3584 bf16 21 to 24 us (60 MB, 2.5 to 2.8 TB/s), fp32 28 us (89 MB, 3.2 TB/s; 216 registers, two workgroups).
#include "moe_kernels.h"
#include "moe_products.h"
#include "moe_rows.h"

#include <type_traits>

namespace moe {

namespace {

// Where the codes of rows [rows, cols] go; kp: cols rounded up to 128.
struct Codes {
  uint8_t* q;
  uint8_t* scale;
  int dt, packed;
  int rows, kp;            // rows that are written: with packed a multiple of 16
};

// Address of the codes of columns col .. of a row (col a multiple of 8), and of a block's scale.
__device__ __forceinline__ uint8_t* code_at(const Codes& o, int row, int col) {
  if (!o.packed) return o.q + (o.dt == MOE_DT_FP8_E4M3 ? (int64_t)row * o.kp + col : ((int64_t)row * o.kp + col) / 2);
  return o.q + ((int64_t)(row >> 4) * (o.kp >> 7) + (col >> 7)) * 1024 + (((col >> 5) & 3) * 16 + (row & 15)) * 16 + ((col & 31) >> 1);
}
__device__ __forceinline__ uint8_t* scale_at(const Codes& o, int row, int col) {
  if (!o.packed) return o.scale + (int64_t)row * (o.kp >> 5) + (col >> 5);
  return o.scale + ((int64_t)(row >> 4) * (o.kp >> 7) + (col >> 7)) * 64 + (row & 15) * 4 + ((col >> 5) & 3);
}

struct Block {             // what the elements of a block share
  int sexp;
  bool bad;                // Inf or NaN: scale 255, codes 0
  float inv;               // 2^-sexp
  __device__ __forceinline__ Block(uint32_t amax, int dt) {
    bad = amax >= 0x7F800000u;
    sexp = block_sexp_any(bad ? 0u : amax, dt == MOE_DT_FP8_E4M3 ? Fp8Fmt::EMAX : Fp4Fmt::EMAX);
    inv = e8m0_scale_float(-sexp);
  }
  __device__ __forceinline__ uint8_t byte() const { return (uint8_t)(bad ? 255 : sexp + 127); }
};

// v / 2^sexp moved to the neighbour on the element grid that byte `k` of `noise` chooses.  Exact but for the sum
// with the noise, whose 2^-9 steps fp32 holds beside numbers up to 16.
__device__ __forceinline__ float stochastic(float v, uint32_t noise, int k, const Block& b, int dt) {
  const bool f8 = dt == MOE_DT_FP8_E4M3;
  const uint32_t mant = f8 ? 3u << 23 : 1u << 23;
  const float a = __builtin_fminf(__builtin_fabsf(v) * b.inv, f8 ? 448.0f : 6.0f);
  const uint32_t e = max(__float_as_uint(a) & 0x7F800000u, f8 ? 121u << 23 : 127u << 23);   // a's binade, at least the lowest
  const float up = __builtin_fmaf((float)((noise >> (8 * k)) & 255u), 1.0f / 256.0f, 1.0f / 512.0f);
  const float t = __builtin_floorf(__builtin_fmaf(a, __uint_as_float((254u << 23) + mant - e), up));
  return __builtin_copysignf(t * __uint_as_float(e - mant), v);
}

// Codes of eight values in units of 2^sexp: four bytes (fp4) or eight.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], const Block& b, int sexp, int dt) {
  uint2 w = {0, 0};
  if (b.bad) return w;
  const float unit = e8m0_scale_float(sexp);
  if (dt == MOE_DT_FP8_E4M3) {
    w.x = encode_pair_fp8_hw(v[0], v[1], sexp) | (encode_pair_fp8_hw(v[2], v[3], sexp) << 16);
    w.y = encode_pair_fp8_hw(v[4], v[5], sexp) | (encode_pair_fp8_hw(v[6], v[7], sexp) << 16);
  } else {
    w.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w.x, v[0], v[1], unit, 0);   // into one byte each
    w.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w.x, v[2], v[3], unit, 1);
    w.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w.x, v[4], v[5], unit, 2);
    w.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w.x, v[6], v[7], unit, 3);
  }
  return w;
}

typedef uint32_t v2u_any __attribute__((ext_vector_type(2), aligned(1)));

// Eight elements of row `row` from column col (a multiple of 8), zeros outside the matrix; their noise.
template <bool NOISE, class XT>
__device__ __forceinline__ void load8(const XT* x, const uint8_t* noise, int rows, int cols, int row, int col, float (&v)[8],
                                      uint32_t (&nz)[2]) {
  nz[0] = nz[1] = 0;
  if (row < rows && col + 8 <= cols) {
    const int64_t at = (int64_t)row * cols + col;
    load_any<8>(x + at, v);
    if constexpr (NOISE) {
      const v2u_any n = *reinterpret_cast<const v2u_any*>(noise + at);
      nz[0] = n[0];
      nz[1] = n[1];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
      if (row < rows && col + j < cols) {
        const int64_t at = (int64_t)row * cols + col + j;
        float one[1];
        load_row<1>(x + at, one);
        v[j] = one[0];
        if constexpr (NOISE) nz[j / 4] |= (uint32_t)noise[at] << (8 * (j % 4));
      }
    }
  }
}

// Codes of eight columns of a row; the block's other columns are in the three adjacent lanes.
template <bool NOISE>
__device__ __forceinline__ void store8(const Codes& o, int row, int col, const float (&v)[8], const uint32_t (&nz)[2]) {
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, DPP_XOR1, 0xF, 0xF, false));
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, DPP_XOR2, 0xF, 0xF, false));
  if (row >= o.rows || col >= o.kp) return;
  const Block b(amax, o.dt);
  uint2 w;
  if constexpr (NOISE) {
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = stochastic(v[j], nz[j / 4], j % 4, b, o.dt);
    w = encode8(s, b, 0, o.dt);
  } else {
    w = encode8(v, b, b.sexp, o.dt);
  }
  uint8_t* const q = code_at(o, row, col);
  if (o.dt == MOE_DT_FP8_E4M3) *reinterpret_cast<uint2*>(q) = w;
  else *reinterpret_cast<uint32_t*>(q) = w.x;
  if ((col & 31) == 0) *scale_at(o, row, col) = b.byte();
}

// Along the rows only: a thread takes eight columns.
template <bool NOISE, class XT>
__global__ __launch_bounds__(256) void quant_rows_kernel(const XT* __restrict__ x, const uint8_t* __restrict__ noise, int rows,
                                                         int cols, int row0, const Codes o) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x, per_row = (uint32_t)o.kp / 8;
  const int row = row0 + (int)(id / per_row), col = (int)(id % per_row) * 8;
  float v[8];
  uint32_t nz[2];
  load8<NOISE>(x, noise, rows, cols, row, col, v, nz);
  store8<NOISE>(o, row, col, v, nz);
}

// Tiles of 128 rows x 64 columns through LDS: the codes of the rows (where asked for) from the registers they
// were loaded into, those of the columns from LDS.
//   fp32: a thread takes the 32 rows of one block of one column; column c of row r stands at c ^ (16 (r / 32)),
//     so that the four blocks' lanes read distinct banks.
//   bf16: as it came, two columns to a dword, which leaves room for eight workgroups on a CU (4096 x 3584 to
//     fp4 both ways 15.4 us, with noise 24.5; with fp32 copies, four on a CU, 18.9 and 29.4).  A thread takes 16 rows
//     of two columns and shares their maxima with its neighbour; the dword's place is turned by the 16-row
//     group, rows from 64 on change places in pairs.
constexpr int TR = 128, TC = 64, PASS = TR / 32, TILE_P = TC + 4;

// Codes of 8 n consecutive columns of a row of codes that starts at `col`, and with `lead` their block's scale.
template <int N, bool NOISE>
__device__ __forceinline__ void store_column(const Codes& o, int row, int col, const float (&v)[8 * N], const Block& b, bool lead) {
  if (row >= o.rows || col >= o.kp) return;
  uint2 w[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float e[8] = {v[8 * k], v[8 * k + 1], v[8 * k + 2], v[8 * k + 3], v[8 * k + 4], v[8 * k + 5], v[8 * k + 6], v[8 * k + 7]};
    w[k] = encode8(e, b, NOISE ? 0 : b.sexp, o.dt);
  }
  uint8_t* const q = code_at(o, row, col);
  if (o.dt == MOE_DT_FP8_E4M3) {
#pragma unroll
    for (int k = 0; k < N; k += 2) reinterpret_cast<uint4*>(q)[k / 2] = uint4{w[k].x, w[k].y, w[k + 1].x, w[k + 1].y};
  } else if constexpr (N == 4) {
    *reinterpret_cast<uint4*>(q) = uint4{w[0].x, w[1].x, w[2].x, w[3].x};
  } else {
    *reinterpret_cast<uint2*>(q) = uint2{w[0].x, w[1].x};
  }
  if (lead) *scale_at(o, row, col) = b.byte();
}

template <bool NOISE, class XT>
__global__ __launch_bounds__(256) void quant_tiles_kernel(const XT* __restrict__ x, const uint8_t* __restrict__ noise, int rows,
                                                          int cols, int tile0, int tiles_c, const Codes o, const Codes ot) {
  constexpr bool PAIRS = sizeof(XT) == 2;
  __shared__ __attribute__((aligned(16))) float tile[PAIRS ? TR * TC / 2 : TR * TILE_P];
  __shared__ uint32_t ntile[NOISE ? TR * (TC / 4 + 1) : 1];
  // neighbouring tiles of a row on one XCD: they share lines of the codes and scales
  const int id = tile0 + run_of_xcd(blockIdx.x, gridDim.x);
  const int r0 = id / tiles_c * TR, c0 = id % tiles_c * TC;
  const int lr = threadIdx.x >> 3, lc = (threadIdx.x & 7) * 8;
  float in[PASS][8];
  uint32_t nz[PASS][2];
  if (r0 + TR <= rows && c0 + TC <= cols) {                   // without tests per lane, all loads are in flight together
#pragma unroll
    for (int p = 0; p < PASS; ++p) {
      const int64_t at = (int64_t)(r0 + p * 32 + lr) * cols + c0 + lc;
      load_any<8>(x + at, in[p]);
      if constexpr (NOISE) {
        const v2u_any n = *reinterpret_cast<const v2u_any*>(noise + at);
        nz[p][0] = n[0];
        nz[p][1] = n[1];
      }
    }
  } else {
#pragma unroll
    for (int p = 0; p < PASS; ++p) load8<NOISE>(x, noise, rows, cols, r0 + p * 32 + lr, c0 + lc, in[p], nz[p]);
  }
#pragma unroll
  for (int p = 0; p < PASS; ++p) {
    const int r = p * 32 + lr;
    if constexpr (PAIRS) {                                    // the values are bf16: their upper halves
      v4u_ w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __builtin_amdgcn_perm(__float_as_uint(in[p][2 * j + 1]), __float_as_uint(in[p][2 * j]), 0x07060302u);
      *reinterpret_cast<v4u_*>(tile + (r ^ (r >> 6)) * (TC / 2) + ((lc / 2) ^ (8 * ((r >> 4) & 3)))) = w;
    } else {
      store_row<8>(tile + r * TILE_P + (lc ^ (16 * p)), in[p]);
    }
    if constexpr (NOISE) {
      ntile[r * (TC / 4 + 1) + lc / 4] = nz[p][0];
      ntile[r * (TC / 4 + 1) + lc / 4 + 1] = nz[p][1];
    }
  }
  __syncthreads();
  if (o.q) {
#pragma unroll
    for (int p = 0; p < PASS; ++p) store8<NOISE>(o, r0 + p * 32 + lr, c0 + lc, in[p], nz[p]);
  }
  if constexpr (PAIRS) {
    const int k = threadIdx.x & 7, c2 = threadIdx.x >> 3;     // 16-row group, pair of columns
    float v[2][16];
    uint32_t amax[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t w = __float_as_uint(tile[((16 * k + i) ^ (k >> 2)) * (TC / 2) + (c2 ^ (8 * (k & 3)))]);
      v[0][i] = __uint_as_float(w << 16);
      v[1][i] = __uint_as_float(w & 0xFFFF0000u);
#pragma unroll
      for (int c = 0; c < 2; ++c) amax[c] = max(amax[c], __float_as_uint(v[c][i]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const Block b(max(amax[c], (uint32_t)__builtin_amdgcn_mov_dpp((int)amax[c], DPP_XOR1, 0xF, 0xF, false)), ot.dt);
      if constexpr (NOISE) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          v[c][i] = stochastic(v[c][i], ntile[(16 * k + i) * (TC / 4 + 1) + c2 / 2] >> (16 * (c2 & 1)), c, b, ot.dt);
      }
      store_column<2, NOISE>(ot, c0 + 2 * c2 + c, r0 + 16 * k, v[c], b, (k & 1) == 0);
    }
  } else {
    const int c = threadIdx.x >> 2, g = threadIdx.x & 3;     // a column, 32 of its rows
    float v[32];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      v[i] = tile[(32 * g + i) * TILE_P + (c ^ (16 * g))];
      amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    const Block b(amax, ot.dt);
    if constexpr (NOISE) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        v[i] = stochastic(v[i], ntile[(32 * g + i) * (TC / 4 + 1) + c / 4] >> (8 * (c & 3)), 0, b, ot.dt);
    }
    store_column<4, NOISE>(ot, c0 + c, r0 + 32 * g, v, b, true);
  }
}

// Row-major codes [N, K / 2] and scales [N, K / 32], K a multiple of 32, to the packed layout: a thread
// moves one block's 16 bytes and its scale.
__global__ __launch_bounds__(256) void pack_mx_kernel(const uint8_t* __restrict__ w, const uint8_t* __restrict__ ws, int N, int K,
                                                      int64_t pieces, const Codes o) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= pieces) return;
  const int l = (int)(id & 63), steps = o.kp >> 7;
  const int64_t blk = id >> 6;
  const int row = (int)(blk / steps) * 16 + (l & 15), col = (int)(blk % steps) * 128 + (l >> 4) * 32;
  uint4 v = {0, 0, 0, 0};
  uint8_t s = 0;
  if (row < N && col < K) {
    v = *reinterpret_cast<const uint4*>(w + ((int64_t)row * K + col) / 2);
    s = ws[(int64_t)row * (K / 32) + col / 32];
  }
  *reinterpret_cast<uint4*>(code_at(o, row, col)) = v;
  *scale_at(o, row, col) = s;
}

Codes codes_of(void* q, uint8_t* scale, int dt, int packed, int64_t rows, int64_t cols) {
  return Codes{(uint8_t*)q, scale, dt, packed, (int)(packed ? (rows + 15) / 16 * 16 : rows), (int)moe_mx_padded_k(cols)};
}

template <bool NOISE, class XT>
hipError_t quant(const QuantMxArgs& a, hipStream_t s) {
  const XT* const x = static_cast<const XT*>(a.x);
  const Codes o = codes_of(a.q, a.q_scale, a.q_dt, a.q_packed, a.rows, a.cols);
  if (!a.t) {
    const int64_t per_row = o.kp / 8, slice = MAX_ITEMS / per_row;   // rows of one dispatch
    for (int64_t r = 0; r < o.rows; r += slice) {
      const int64_t n = (o.rows - r < slice ? o.rows - r : slice) * per_row;
      quant_rows_kernel<NOISE><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(x, a.noise, a.rows, a.cols, (int)r, o);
    }
    return hipGetLastError();
  }
  const Codes ot = codes_of(a.t, a.t_scale, a.t_dt, a.t_packed, a.cols, a.rows);
  // tiles over everything that is written: the rows' codes and the transpose's, with what fills them up
  const int64_t rows = o.q && o.rows > ot.kp ? o.rows : ot.kp, cols = o.q && o.kp > ot.rows ? o.kp : ot.rows;
  const int64_t tiles_c = (cols + TC - 1) / TC, tiles = tiles_c * ((rows + TR - 1) / TR), slice = MAX_ITEMS / 256;
  for (int64_t t = 0; t < tiles; t += slice)
    quant_tiles_kernel<NOISE><<<(unsigned)(tiles - t < slice ? tiles - t : slice), 256, 0, s>>>(x, a.noise, a.rows, a.cols, (int)t,
                                                                                             (int)tiles_c, o, ot);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_mx(const QuantMxArgs& a, hipStream_t s) {
  if (a.x_dt == MOE_DT_F32) return a.noise ? quant<true, float>(a, s) : quant<false, float>(a, s);
  return a.noise ? quant<true, uint16_t>(a, s) : quant<false, uint16_t>(a, s);
}

hipError_t launch_pack_mx(const uint8_t* w, const uint8_t* ws, int N, int K, uint8_t* out, uint8_t* out_scale, hipStream_t s) {
  const Codes o = codes_of(out, out_scale, MOE_DT_FP4_E2M1, 1, N, K);
  const int64_t pieces = (int64_t)o.rows * (o.kp / 32);
  pack_mx_kernel<<<(unsigned)((pieces + 255) / 256), 256, 0, s>>>(w, ws, N, K, pieces, o);
  return hipGetLastError();
}

}  // namespace moe
