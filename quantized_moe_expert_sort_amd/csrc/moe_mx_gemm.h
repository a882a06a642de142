// Product of tokens in fp4 or fp8 with one e8m0 scale per 32 and packed MXFP4 weights:
//
//   r[t, c] = sum_k a[t, k] 2^(sa[t, k/32]) w[c, k] 2^(sw[c, k/32])   (+ add[t, c]);
//   with an activation, w holds the gate rows and then the up rows: out[t, i] = act(g) u (+ add).
//
// The block-scaled matrix instruction (16 x 16, 128 deep) takes both scales, so the codes go in
// without any other arithmetic; the sums are fp32.  The weights are its row operand and the tokens its
// column operand: a lane ends with four consecutive channels of one token.  K is a multiple of 128 (what
// codes a matrix fills rows up with zeros), so no step has a tail.
#pragma once

#include "moe_kernels.h"
#include "moe_operands.h"
#include "moe_rows.h"
#include "moe_products.h"

#include <type_traits>

#pragma clang diagnostic ignored "-Winline-asm"   // m0 is written by the load-to-LDS copies

namespace moe {

namespace {

template <int V>
using Const = std::integral_constant<int, V>;

struct Gemm : ActArgs {
  const uint8_t* a;        // [T, K] codes, row-major
  const uint8_t* as;       // [T, K / 32]
  const uint8_t* w;        // packed: 1 KB blocks of 16 rows x 128 columns
  const uint8_t* ws;       // packed: 64 bytes per block
  const void* add;         // [T, No] of the output's type, or null
  void* out;               // [T, No] bf16 or fp32
  int T, N, K, No;         // No = N, or N / 2 with an activation
  int f32;                 // the output's type
};

// What a lane holds of 16 weight rows (w: its 32 columns) and of 16 tokens for one 128-deep product.
//   DT_FP4, DT_FP8: codes and scales go into the block-scaled instruction.  Products of fp4 values keep all
//     their bits.  Of fp8 tokens it adds eight products at a time (columns 8 i .. 8 i + 7) in fixed point and
//     drops what lies 2^14 below the largest of the eight: 4.6e-6 of a result (2-norm, normal data), far
//     below a bf16 result's rounding.
//   FP8_WIDE, for fp32 results of fp8 tokens: codes and scales are widened to bf16, which holds them exactly,
//     and go through the bf16 instruction at half the rate.
constexpr int FP8_WIDE = 16;
template <int ADT>
struct Operand {
  static constexpr int STEP = ADT == DT_FP4 ? 64 : 128;       // bytes of a row's 128 columns
  struct W { uint4 q; uint32_t s; };
  struct A { v8i q; uint32_t s; };
  // 16-byte pieces of a token's step that lane group g reads
  static __device__ __forceinline__ int lo(int g) { return g; }
  static __device__ __forceinline__ int hi(int g) { return 4 + g; }
  // the scale bytes are the low ones
  static __device__ __forceinline__ W weights(const uint4& q, uint32_t s) { return W{q, s}; }
  static __device__ __forceinline__ A tokens(const uint4& x, const uint4& y, uint32_t s) {
    if constexpr (ADT == DT_FP4) return A{fp4_operand_lo(x), s};
    else return A{v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w}, s};
  }
  static __device__ __forceinline__ v4f mma(const W& w, const A& a, const v4f& c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand_lo(w.q), a.q, c, MFMA_FMT_FP4,
                                                           ADT == DT_FP4 ? MFMA_FMT_FP4 : MFMA_FMT_FP8, 0, w.s, 0, a.s);
  }
};
template <>
struct Operand<FP8_WIDE> {
  static constexpr int STEP = 128;
  struct W { v8bf b[4]; };
  struct A { v8bf b[4]; };
  // columns 32 g .. 32 g + 31, as the weights'
  static __device__ __forceinline__ int lo(int g) { return 2 * g; }
  static __device__ __forceinline__ int hi(int g) { return 2 * g + 1; }
  static __device__ __forceinline__ float scale(uint32_t s) {
    s &= 0xFFu;
    return s == 255u ? __uint_as_float(0x7FC00000u) : e8m0_to_float(s);
  }
  static __device__ __forceinline__ W weights(const uint4& q, uint32_t s) {
    const float k = scale(s);
    return W{{fp4x8_to_bf16(q.x, k), fp4x8_to_bf16(q.y, k), fp4x8_to_bf16(q.z, k), fp4x8_to_bf16(q.w, k)}};
  }
  static __device__ __forceinline__ v8bf eight(uint32_t lo, uint32_t hi, float k) {
    const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, k, false), p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, k, true);
    const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, k, false), p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, k, true);
    return v8bf{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
  }
  static __device__ __forceinline__ A tokens(const uint4& x, const uint4& y, uint32_t s) {
    const float k = scale(s);
    return A{{eight(x.x, x.y, k), eight(x.z, x.w, k), eight(y.x, y.y, k), eight(y.z, y.w, k)}};
  }
  static __device__ __forceinline__ v4f mma(const W& w, const A& a, v4f c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = mfma_bf16(w.b[j], a.b[j], c);
    return c;
  }
};

// Whether results are fp32: decided by the tokens' type but for fp4's.
template <int ADT>
__device__ __forceinline__ bool wide_out(const Gemm& p) { return ADT == DT_FP4 ? p.f32 != 0 : ADT == FP8_WIDE; }

// VEC outputs, channels c .. of token t.
template <int ADT, int VEC>
__device__ __forceinline__ void store_out(const Gemm& p, int64_t t, int c, float (&v)[VEC]) {
  const int64_t at = t * p.No + c;
  if (p.add) {
    float o[VEC];
    if (wide_out<ADT>(p)) load_any<VEC>(static_cast<const float*>(p.add) + at, o);
    else load_any<VEC>(static_cast<const uint16_t*>(p.add) + at, o);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] += o[i];
  }
  if (wide_out<ADT>(p)) store_any<VEC>(static_cast<float*>(p.out) + at, v);
  else store_any<VEC>(static_cast<uint16_t*>(p.out) + at, v);
}
template <int ADT>
__device__ __forceinline__ void store_one(const Gemm& p, int64_t t, int c, float v) {
  float one[1] = {v};
  store_out<ADT>(p, t, c, one);
}

// ---------------------------------------------------------------- a tile's outputs
//
// acc[n][m] of a wave: FN 16-row groups of weights (with an activation the gate rows' and then the up rows'),
// FM of tokens.  The tile starts at token t0, channel c0; this wave's
// tokens start tw0 in it and its channels are the wn-th share.
template <int ADT, bool ACT, int FM, int FN>
__device__ __forceinline__ void tile_out(const Gemm& p, const v4f (&acc)[FN][FM], int t0, int tw0, int c0, int wn) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  // register i of lane 16 g + r is channel 4 g + i of a 16-channel group, token r.  The odd 16-lane rows of
  // one group and the even ones of the next change places: a lane then holds eight consecutive channels (of
  // the first group for g = 0, 2), which go out together at any address.
  constexpr int FO = ACT ? FN / 2 : FN;                       // 16-channel groups of outputs
#pragma unroll
  for (int n = 0; n < FO; n += 2) {
    const int c = c0 + wn * (FO * 16) + (n + (g & 1)) * 16 + (g >> 1) * 8;
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const int64_t t = t0 + tw0 + m * 16 + r;
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = acc[n][m][i], y = acc[n + 1][m][i];
        if constexpr (ACT) {
          x = activate(p, x, acc[n + FO][m][i]);
          y = activate(p, y, acc[n + 1 + FO][m][i]);
        }
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
        v[i] = __uint_as_float(s[0]);
        v[4 + i] = __uint_as_float(s[1]);
      }
      if (t < p.T && c + 8 <= p.No) {
        store_out<ADT>(p, t, c, v);
      } else if (t < p.T) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < p.No) store_one<ADT>(p, t, c + i, v[i]);
      }
    }
  }
}

// ---------------------------------------------------------------- few tokens: weights streamed
//
// A workgroup takes one 16-channel block (with an activation the gate block and the up block of
// the same outputs) and 16 tokens; its waves split K and add their sums through LDS.  The weights
// are read once, from whole lines, straight into the operand registers, STREAM_U blocks (and as many of
// the gate) in flight per wave before the first product.  Bound by the latency of these loads and of the
// launch: as many waves as there are K steps, up to 16 (1 x 7168 with SiLU, fp8, us at K 512, 1536, 3584, 7168:
// 2.9 4.2 5.8 8.5; up to 8 waves 2.9 4.4 6.7 9.3; waves of four steps, up to 8 of them, 3.0 5.6 6.7 9.2).

constexpr int STREAM_U = 4;                   // K steps a wave loads together
constexpr int STREAM_WAVES = 16;              // waves of a workgroup, at most

template <int ADT, bool ACT>
__global__ __launch_bounds__(STREAM_WAVES * 64) void gemm_mx_stream_kernel(const Gemm p) {
  using O = Operand<ADT>;
  constexpr int NB = ACT ? 2 : 1, STEP = O::STEP;
  __shared__ v4f sums[STREAM_WAVES][NB][64];
  // the wave's number in a scalar register: an MFMA under a lane mask would run with the mask ignored
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int steps = p.K / 128;
  const uint8_t* wp[NB];
  const uint8_t* wsp[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t blk = ((int64_t)blockIdx.x + (b ? p.No / 16 : 0)) * steps;
    wp[b] = p.w + blk * 1024 + lane * 16;
    wsp[b] = p.ws + blk * 64 + 4 * r + g;
  }
  const int64_t tok = min(r, p.T - 1);
  const uint8_t* const ap = p.a + tok * ((int64_t)steps * STEP);
  const uint8_t* const asp = p.as + tok * ((int64_t)steps * 4) + g;
  v4f acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int per = (steps + waves - 1) / waves;
  const int s1 = min((wave + 1) * per, steps);
  // steps s0 .. s0 + STREAM_U - 1, or (not whole) as many of them as this wave has left
  const auto trip = [&](const int s0, auto whole) {
    uint4 wv[STREAM_U][NB];
    uint4 al[STREAM_U], ah[STREAM_U];
    uint32_t sw[STREAM_U][NB], sa[STREAM_U];
#pragma unroll
    for (int j = 0; j < STREAM_U; ++j) {
      const int64_t s = s0 + j;
      if (!decltype(whole)::value && s >= s1) break;
#pragma unroll
      for (int b = 0; b < NB; ++b) wv[j][b] = ldw16(wp[b] + s * 1024);
#pragma unroll
      for (int b = 0; b < NB; ++b) sw[j][b] = wsp[b][s * 64];
      al[j] = *reinterpret_cast<const uint4*>(ap + s * STEP + 16 * O::lo(g));
      if constexpr (STEP == 128) ah[j] = *reinterpret_cast<const uint4*>(ap + s * STEP + 16 * O::hi(g));
      sa[j] = asp[s * 4];
    }
#pragma unroll
    for (int j = 0; j < STREAM_U; ++j) {
      if (!decltype(whole)::value && s0 + j >= s1) break;
      const typename O::A a = O::tokens(al[j], ah[j], sa[j]);
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[b] = O::mma(O::weights(wv[j][b], sw[j][b]), a, acc[b]);
    }
  };
  int s0 = wave * per;
  for (; s0 + STREAM_U <= s1; s0 += STREAM_U) trip(s0, std::true_type());
  if (s0 < s1) trip(s0, std::false_type());
#pragma unroll
  for (int b = 0; b < NB; ++b) sums[wave][b][lane] = acc[b];
  __syncthreads();
  if (wave != 0 || r >= p.T) return;
#pragma unroll
  for (int b = 0; b < NB; ++b)
    for (int w = 1; w < waves; ++w) acc[b] += sums[w][b][lane];
#pragma unroll
  for (int i = 0; i < 4; ++i) {                               // channels 4 g .. 4 g + 3 of token r
    const int c = blockIdx.x * 16 + 4 * g + i;
    if (c < p.No) {
      float v = acc[0][i];
      if constexpr (ACT) v = activate(p, v, acc[1][i]);
      store_one<ADT>(p, r, c, v);
    }
  }
}

// ---------------------------------------------------------------- more tokens: LDS tiles
//
// Tiles of BM tokens x BN weight rows, K in steps of 128 bytes of a token's row (SUB = 2 of 128 columns
// for fp4, 1 for fp8) through S LDS buffers filled by the load-to-LDS copies (S - 1 steps in flight).
// GM x GN waves, each BM / GM tokens x BN / GN weight rows; with KG > 1 that many groups of waves share out
// K and add their sums through LDS.
//
// A copy instruction takes 8 token rows x 128 bytes (whole lines), its 16-byte pieces placed at
// p ^ ((row / 2) % 8) so that the 16 lanes that read one piece of 16 rows hit distinct banks, or one 1 KB
// weight block, which stays in lane order.  The scales come along, a dword (one row's 128 columns) per
// lane and copy.
//
// Measured (a row of launches, cold operands): 8192^3 fp4 309 to 315 us (3.5 PF/s; the instruction alone, on
// registers, 8.3), matrix cores 43% busy at 2.1 GHz, fp8 420 (2.6 PF/s of 4.7), 61%; 8192 x 7168 x 3584 fp4 141, fp8
// 196.  What is left, at 8192^3 fp4: without the copies 247 us, without the outputs 285, without both 230, without
// the products 274; without the scales' copies, whose rows are 8 bytes to a line, 298.  No faster: operands read a unit
// ahead (324 us, 244 registers), four waves of 128 x 128 (324), a higher priority of the products, copies later
// in the step (320); two fours of waves that take turns at reading and multiplying (fp8 443 us); weights straight
// from the L2 into registers (553 us: their latency shows); a third buffer for fp8 (warm operands: 8192^3 405 us where
// two take 400, 8192 x 7168 x 3584 170 and 167).

template <int BM, int BN, int GM, int GN, int S, int KG, int ADT, bool ACT>
struct Tile {
  static constexpr int WAVES = GM * GN, THREADS = WAVES * KG * 64, SUB = ADT == DT_FP4 ? 2 : 1;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 64 * SUB, S_BYTES = ((BM + BN) * SUB + 63) / 64 * 256;
  static constexpr int BUF = A_BYTES + B_BYTES + S_BYTES, LDS = KG * S * BUF;
};

template <int BM, int BN, int GM, int GN, int S, int KG, int ADT, bool ACT>
__device__ __forceinline__ void tile_body(const Gemm& p, int tm, int tn, uint8_t* lds_all) {
  using T = Tile<BM, BN, GM, GN, S, KG, ADT, ACT>;
  constexpr int WAVES = T::WAVES, BUF = T::BUF, SUB = T::SUB, A_BYTES = T::A_BYTES;
  using O = Operand<ADT>;
  constexpr int S_AT = A_BYTES + T::B_BYTES;                  // the scales' place in a buffer
  constexpr int WM = BM / GM, WN = BN / GN;                   // one wave's tokens and weight rows
  constexpr int FM = WM / 16, FN = WN / 16;                   // its 16-row operands
  constexpr int QA = BM / 8 / WAVES, QB = BN / 16 * SUB / WAVES;   // copy instructions of a wave and step
  constexpr int NSC = T::S_BYTES / 256, QS = (NSC + WAVES - 1) / WAVES;   // copies of scales: of a step, of a wave
  constexpr int Q = QA + QB + QS;
  static_assert(QA * 8 * WAVES == BM && QB * WAVES == BN / 16 * SUB && (S - 2) * Q < 63 && S >= 2 && S <= 4,
                "whole copies");
  static_assert(FN % 2 == 0 && (!ACT || FN % 4 == 0), "operands in pairs");
  static_assert(KG == 1 || (KG - 1) * WAVES * FN * FM * 1024 <= T::LDS, "the groups' sums fit");
  const int s128 = p.K / 128, all = (s128 + SUB - 1) / SUB, most = (all + KG - 1) / KG;
  const int lane = threadIdx.x & 63, wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KG == 1 ? 0 : wave_all / WAVES, wave = KG == 1 ? wave_all : wave_all % WAVES;
  const int first = kg * most, steps = max(min(most, all - first), 0);   // this group's steps
  uint8_t* const lds = lds_all + kg * (S * BUF);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int wm = wave % GM, wn = wave / GM;
  const int t0 = tm * BM;
  const int c0 = ACT ? tn * (BN / 2) : tn * BN;               // first output channel

  // 16-row group of the weights that is group rg of the tile: with an activation each wave's gate rows,
  // then its up rows
  const auto group_of = [&](int rg) {
    if constexpr (ACT) {
      const int w = rg / FN, i = rg % FN, half = FN / 2;
      const int gf = min(c0 / 16 + w * half + i % half, p.No / 16 - 1);
      return i < half ? gf : p.No / 16 + gf;
    } else {
      return min(c0 / 16 + rg, (p.N + 15) / 16 - 1);
    }
  };
  // per-lane source offsets of this wave's copies
  const int64_t a_pitch = (int64_t)s128 * O::STEP;
  const uint8_t* const a_base = p.a + (int64_t)t0 * a_pitch;
  uint32_t a_off[QA], b_off[QB];
  int a_piece[QA];
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int row = (wave + WAVES * q) * 8 + (lane >> 3);
    a_piece[q] = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
    a_off[q] = (uint32_t)min(row, p.T - 1 - t0) * (uint32_t)a_pitch + a_piece[q];
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) {
    const int blk = wave + WAVES * q;
    b_off[q] = (uint32_t)group_of(blk / SUB) * (uint32_t)s128 * 1024u + (blk % SUB) * 1024 + lane * 16;
  }
  const uint8_t* s_at[QS];
  int s_inc[QS], s_half[QS];                                  // bytes per step; of the second half of a step
#pragma unroll
  for (int q = 0; q < QS; ++q) {
    const int e = min((min(wave + WAVES * q, NSC - 1)) * 64 + lane, (BM + BN) * SUB - 1);
    const int sub = e / (BM + BN), j = e % (BM + BN);
    const bool tok = j < BM;
    s_half[q] = sub * (tok ? 4 : 64);
    s_inc[q] = SUB * (tok ? 4 : 64);
    s_at[q] = tok ? p.as + (int64_t)(t0 + min(j, p.T - 1 - t0)) * (s128 * 4)
                  : p.ws + ((int64_t)group_of((j - BM) / 16) * s128) * 64 + ((j - BM) & 15) * 4;
  }
  int fill = 0;                                               // the buffer that the next step's copies fill
  const auto fetch = [&](int st) {
    const uint32_t buf = lds0 + fill * BUF;
    fill = fill + 1 == S ? 0 : fill + 1;
    st += first;
    const bool half = SUB == 2 && st * SUB + 1 == s128;       // the last step may have one half: it is read twice
    const uint8_t* ab = a_base + (int64_t)st * 128;
    const uint8_t* bb = p.w + (int64_t)st * (SUB * 1024);
#pragma unroll
    for (int q = 0; q < QA; ++q) copy16(ab, a_off[q] - (half && a_piece[q] >= 64 ? 64u : 0u), buf + (wave + WAVES * q) * 1024);
#pragma unroll
    for (int q = 0; q < QB; ++q) {
      const int blk = wave + WAVES * q;
      copy16(bb, b_off[q] - (half ? (blk % SUB) * 1024u : 0u), buf + A_BYTES + blk * 1024);
    }
#pragma unroll
    for (int q = 0; q < QS; ++q)
      copy4(s_at[q] + (int64_t)st * s_inc[q] + (half ? 0 : s_half[q]), buf + S_AT + min(wave + WAVES * q, NSC - 1) * 256);
  };

  v4f acc[FN][FM];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[n][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // 16-row operands of sub-step ss: lane 16 g + r holds 32 columns of row r
  const int r = lane & 15, g = lane >> 4;
  const int swz = (r >> 1) & 7;                               // a wave's rows start at a multiple of 16
  const uint8_t* const fa = lds + (wm * WM + r) * 128;
  const uint8_t* const fb = lds + A_BYTES + wn * FN * (SUB * 1024) + lane * 16;
  const uint8_t* const fs = lds + S_AT + r * 4;
  const auto work = [&](int buf, int halves) {
#pragma unroll
    for (int ss = 0; ss < SUB; ++ss) {
      if (ss >= halves) break;
      typename O::W w[FN];
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const uint4 q = *reinterpret_cast<const uint4*>(fb + buf * BUF + n * (SUB * 1024) + ss * 1024);
        w[n] = O::weights(q, *reinterpret_cast<const uint32_t*>(fs + buf * BUF + (ss * (BM + BN) + BM + wn * WN + n * 16) * 4) >> (8 * g));
      }
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const uint8_t* const row = fa + buf * BUF + m * 2048;
        const uint32_t sa = *reinterpret_cast<const uint32_t*>(fs + buf * BUF + (ss * (BM + BN) + wm * WM + m * 16) * 4) >> (8 * g);
        const uint4 x = *reinterpret_cast<const uint4*>(row + (((ss * 4 + O::lo(g)) ^ swz) * 16));
        uint4 y;
        if constexpr (O::STEP == 128) y = *reinterpret_cast<const uint4*>(row + ((O::hi(g) ^ swz) * 16));
        const typename O::A a = O::tokens(x, y, sa);
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[n][m] = O::mma(w[n], a, acc[n][m]);
      }
    }
  };
  // All but the newest `later` steps' copies of this wave have landed and its LDS reads are done;
  // then meet the other waves.
  const auto meet = [&](int later) {
    if (later >= S - 2) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * Q) : "memory");
    else if (S > 3 && later == 1) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(Q) : "memory");
    else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };

#pragma unroll
  for (int i = 0; i < S - 1; ++i)
    if (i < steps) fetch(i);
  int buf = 0;
  for (int st = 0; st < most; ++st) {                         // as many steps, so barriers, for every group
    meet(min(steps - 1 - st, S - 2));
    // the buffer of step st - 1 is free: every wave has passed the barrier after reading it
    if (st + S - 1 < steps) fetch(st + S - 1);
    if (KG == 1 || st < steps) work(buf, min(SUB, s128 - (first + st) * SUB));
    buf = buf + 1 == S ? 0 : buf + 1;
  }
  if constexpr (KG > 1) {                                     // the groups' sums, added by the first group
    v4f* const part = reinterpret_cast<v4f*>(lds_all);
    constexpr int V = FN * FM;
    __syncthreads();                                          // every operand read is done
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) part[(((kg - 1) * WAVES + wave) * V + i) * 64 + lane] = acc[i / FM][i % FM];
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int k = 0; k < KG - 1; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i / FM][i % FM] += part[((k * WAVES + wave) * V + i) * 64 + lane];
  }

  tile_out<ADT, ACT, FM, FN>(p, acc, t0, wm * WM, c0, wn);
}

template <int BM, int BN, int GM, int GN, int S, int KG, int ADT, bool ACT>
__global__ __launch_bounds__(GM * GN * KG * 64) void gemm_mx_tile_kernel(const Gemm p, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tile<BM, BN, GM, GN, S, KG, ADT, ACT>::LDS];
  int tm, tn;
  tile_of(run_of_xcd(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
  tile_body<BM, BN, GM, GN, S, KG, ADT, ACT>(p, tm, tn, lds);
}

// 256 x 256 tiles; those past the first `full` are taken in two halves of 128 tokens each, so that
// a last round that would leave half of the CUs idle takes half as long.
template <int ADT, bool ACT>
__global__ __launch_bounds__(512) void gemm_mx_big_kernel(const Gemm p, int tiles_m, int tiles_n, int full) {
  constexpr int WHOLE = Tile<256, 256, 2, 4, 2, 1, ADT, ACT>::LDS, HALF = Tile<128, 256, 2, 4, 3, 1, ADT, ACT>::LDS;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[WHOLE > HALF ? WHOLE : HALF];
  int tm, tn;
  if ((int)blockIdx.x < full) {
    tile_of(run_of_xcd(blockIdx.x, full), tiles_m, tiles_n, tm, tn);
    tile_body<256, 256, 2, 4, 2, 1, ADT, ACT>(p, tm, tn, lds);
  } else {
    const int h = run_of_xcd(blockIdx.x - full, gridDim.x - full);
    tile_of(full + (h >> 1), tiles_m, tiles_n, tm, tn);
    tm = 2 * tm + (h & 1);
    if (tm * 128 < p.T) tile_body<128, 256, 2, 4, 3, 1, ADT, ACT>(p, tm, tn, lds);
  }
}

template <bool ACT>
int64_t tiles(const Gemm& p, int bm, int bn) {
  const int cols = ACT ? bn / 2 : bn;
  return (int64_t)((p.T + bm - 1) / bm) * ((p.No + cols - 1) / cols);
}

template <int BM, int BN, int GM, int GN, int S, int KG, int ADT, bool ACT>
void tile(const Gemm& p, hipStream_t s) {
  const int tm = (p.T + BM - 1) / BM;
  const int64_t n = tiles<ACT>(p, BM, BN);
  gemm_mx_tile_kernel<BM, BN, GM, GN, S, KG, ADT, ACT>
      <<<(unsigned)n, Tile<BM, BN, GM, GN, S, KG, ADT, ACT>::THREADS, 0, s>>>(p, tm, (int)(n / tm));
}

// The smallest tiles that one round of CUS workgroups holds (they take K in more groups), then the largest of
// which there is more than a round.  Measured, us in a graph of 40 calls with cold operands, chosen ones in
// brackets, in the order 32 x 64 in four groups, 64 x 64 in two, 64 x 64, 128 x 128, 256 x 256 (with halves):
//   fp4, K 512:  64 x 7168 [3.4] 3.4 3.6 4.3 5.7   256 x 3584 5.4 [3.6] 3.6 4.8 6.6   256 x 7168 9.6 5.9 [4.4] 5.0 6.8
//       384 x 7168 14.3 8.6 6.3 [5.3] 7.1   1024 x 7168 31.9 18.9 12.1 10.1 [8.9]
//   fp4, K 1536:  64 x 7168 [4.2] 4.5 5.4 7.4 10.0   256 x 3584 7.3 [4.7] 5.6 7.9 11.0   256 x 7168 13.6 8.4 [7.2] 8.5 11.8
//       384 x 7168 19.3 12.0 11.1 [8.9] 12.0   1024 x 7168 43.0 25.4 20.7 16.4 [14.1]
//   fp4, K 3584:  64 x 7168 [6.1] 7.0 9.3 13.1 19.6   256 x 3584 10.5 [7.3] 9.8 14.8 21.0   256 x 7168 19.1 13.0 [12.0] 14.9 21.5
//       384 x 7168 27.5 18.3 19.3 [15.2] 21.8   1024 x 7168 61.9 39.6 36.4 29.4 [24.6]
//   fp4, K 7168:  64 x 7168 [9.0] 11.0 16.0 23.1 35.3   256 x 3584 15.9 [11.6] 16.8 24.9 37.4   256 x 7168 29.5 20.8 [20.0] 25.7 37.6
//       384 x 7168 42.8 29.9 33.0 [25.7] 38.1   1024 x 7168 98.4 66.1 65.6 51.4 [42.1]
//   fp8, K 3584:  64 x 7168 [6.5] 8.4 10.1 16.3 24.6   256 x 3584 11.4 [9.0] 10.7 17.5 25.9   256 x 7168 20.9 13.6 [13.6] 17.8 26.3
//       384 x 7168 30.1 19.5 20.0 [18.1] 26.6   1024 x 7168 68.7 40.2 39.1 35.3 [30.6]
// The rule counts workgroups only, and small batches of very wide weights lie outside the table: past 16384 rows
// 3 to 64 tokens go to 128 x 128 tiles and past 32768 to 256 x 256, which they hardly fill.  As chosen, K 3584, 16 tokens, rows
// 16384, 16400, 28672, 32768, 32784, 65536: fp4 8.0 13.3 14.4 15.1 27.3 41, fp8 7.9 16.9 17.6 18.5 39.3 52.  Against them
// only calls of 8192 rows each were measured: 32768 rows 23 (fp4) and 24 (fp8), 65536 rows 56 and 59.
template <int ADT, bool ACT>
void run_tiles(const Gemm& p, hipStream_t s) {
  constexpr int CUS = 256;
  if (tiles<ACT>(p, 32, 64) <= CUS) {
    tile<32, 64, 1, ACT ? 1 : 2, 3, 4, ADT, ACT>(p, s);       // with ACT a wave holds gate and up operands
  } else if (tiles<ACT>(p, 64, 64) <= CUS) {
    tile<64, 64, 2, ACT ? 1 : 2, 3, 2, ADT, ACT>(p, s);
  } else if (2 * tiles<ACT>(p, 128, 128) <= CUS) {
    tile<64, 64, 2, ACT ? 1 : 2, 4, 1, ADT, ACT>(p, s);
  } else if (tiles<ACT>(p, 128, 128) <= CUS) {
    tile<128, 128, 4, 2, 4, 1, ADT, ACT>(p, s);
  } else {
    const int64_t n = tiles<ACT>(p, 256, 256);
    const int tm = (p.T + 255) / 256, rest = (int)(n % CUS), full = (int)(2 * rest <= CUS ? n - rest : n);
    gemm_mx_big_kernel<ADT, ACT><<<(unsigned)(full + 2 * (n - full)), 512, 0, s>>>(p, tm, (int)(n / tm), full);
  }
}

// Streamed weights up to 16 tokens, where there is at most a workgroup of 16 channels per CU or at most two
// tokens: every workgroup reads all the tokens, which beyond costs more than the tiles.  Measured, us, streamed
// and 32 x 64 tiles, fp8: 1 x 7168 at K 512, 3584, 7168: 2.5 5.6 8.7 and 3.0 6.0 8.9; 8 x 7168 2.6 6.8 11.0 and 3.1 6.0
// 8.9; 16 x 7168 2.9 8.3 14.5 and 3.1 6.0 9.0; 1 x 3584 2.3 4.3 6.0 and 3.0 5.7 8.7; 16 x 3584 2.6 5.5 9.0 and 3.0 5.9 9.0;
// 16 x 1000 2.6 5.2 8.6 and 3.1 5.6 8.8; with SiLU 16 x 7168 3.0 6.6 11.2 and 4.0 8.0 12.3.
template <int ADT, bool ACT>
void run(const Gemm& p, hipStream_t s) {
  const int groups = (p.No + 15) / 16;
  if (p.T <= 16 && (p.T <= 2 || groups <= 256)) {
    const int waves = p.K / 128;                              // a step each, or an equal share
    gemm_mx_stream_kernel<ADT, ACT><<<(unsigned)groups, (waves < STREAM_WAVES ? waves : STREAM_WAVES) * 64, 0, s>>>(p);
  } else {
    run_tiles<ADT, ACT>(p, s);
  }
}
template <int ADT>
hipError_t run(const GemmMxArgs& a, hipStream_t s) {
  Gemm p;
  p.a = a.a;
  p.as = a.as;
  p.w = a.w;
  p.ws = a.ws;
  p.add = a.add;
  p.out = a.out;
  p.T = a.T;
  p.N = a.N;
  p.K = a.K;
  p.f32 = a.out_dt == MOE_DT_F32;
  p.No = a.act >= 0 ? a.N / 2 : a.N;
  p.set(a.act, a.beta, a.linear_beta);
  if (a.act >= 0) run<ADT, true>(p, s);
  else run<ADT, false>(p, s);
  return hipGetLastError();
}

}  // namespace

}  // namespace moe
