// Matrix product in 8-bit integers with a scale per token and per channel, the coding of its
// activations, and the one-time layout of its weights.
//
//   out[t, c] = sa[t] sw[c] sum_k a[t, k] w[c, k]   (+ add[t, c]);
//   with an activation, w holds the gate rows and then the up rows: out[t, i] = act(g) u (+ add).
//
// The sums are exact in int32 (K < 2^17 keeps 128 * 128 * K below 2^31).  Both kernels feed the
// matrix cores with the weights as the row operand and the tokens as the column operand, so a
// lane ends with consecutive channels of one token: what a row-major output stores together.  A
// lane of an i8 MFMA holds 16 consecutive bytes of one row; weights and tokens are read with the
// same (row, byte) map, so the product does not depend on how the instruction numbers them.
//
// Weights are packed once into 1 KB blocks (f, s): rows 16 f .. 16 f + 15, bytes 64 s .. 64 s + 63,
// byte 16 (16 g + r) + b of a block = row 16 f + r, byte 64 s + 16 g + b; rows past N and bytes past
// K are zero (K is padded to 128), so the kernels need no tail for either: what they read of a
// token's row past K is multiplied by zero.
#include "moe_kernels.h"
#include "moe_operands.h"
#include "moe_products.h"
#include "moe_rows.h"

#include <type_traits>

#pragma clang diagnostic ignored "-Winline-asm"   // m0 is written by the load-to-LDS copies

namespace moe {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------- coding of rows

// One row per workgroup of up to 16 waves; 8 elements per lane and step, rows of up to 8 * 1024
// * 2 elements stay in registers between the maximum and the codes, longer ones are read again.
// Bound by the bytes: 8192 x 3584 in 19.6 us, 4.5 TB/s.
__global__ __launch_bounds__(1024) void quant_i8_kernel(const uint16_t* __restrict__ x, int cols,
                                                        uint8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t red[16];
  const int64_t base = (int64_t)blockIdx.x * cols;
  const int step = blockDim.x * 8;
  float v[2][8];
  uint32_t amax = 0;
  for (int c = 0, col = threadIdx.x * 8; col < cols; ++c, col += step) {
    float f[8];
    load_row<8>(x + base + col, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(f[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (c == 0) v[0][j] = f[j];
      if (c == 1) v[1][j] = f[j];
    }
  }
  amax = wave_max_u32(amax);
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  if (waves > 1) {
    if (lane == 0) red[threadIdx.x >> 6] = amax;
    __syncthreads();
    amax = row16_max_u32((lane & 15) < waves ? red[lane & 15] : 0u);
  }
  const RowScaleI8 rs(amax);
  if (threadIdx.x == 0) scale[blockIdx.x] = rs.scale;
  for (int c = 0, col = threadIdx.x * 8; col < cols; ++c, col += step) {
    float f[8];
    if (c < 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = c == 0 ? v[0][j] : v[1][j];
    } else {
      load_row<8>(x + base + col, f);
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j / 4] |= rs.code(f[j]) << (8 * (j % 4));
    *reinterpret_cast<uint2*>(q + base + col) = uint2{w[0], w[1]};
  }
}

// ---------------------------------------------------------------- weight layout

// thread = one 16-byte piece of the packed weights
__global__ __launch_bounds__(256) void pack_i8_kernel(const uint8_t* __restrict__ w, int N, int K, int blocks_k,
                                                      int64_t pieces, uint8_t* __restrict__ out) {
  const int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (o >= pieces) return;
  const int64_t blk = o >> 6;
  const int l = (int)(o & 63);
  const int64_t row = blk / blocks_k * 16 + (l & 15);
  const int k = (int)(blk % blocks_k) * 64 + (l >> 4) * 16;
  uint4 v = {0, 0, 0, 0};
  if (row < N && k < K) v = *reinterpret_cast<const uint4*>(w + row * K + k);   // K % 16 == 0
  *reinterpret_cast<uint4*>(out + o * 16) = v;
}

// ---------------------------------------------------------------- epilogue

struct Gemm : ActArgs {
  const uint8_t* a;        // [T, K]
  const float* sa;         // [T]
  const uint8_t* w;        // packed
  const float* sw;         // [N]
  const uint16_t* add;     // [T, No] or null
  uint16_t* out;           // [T, No]
  int T, N, K, No;         // No = N, or N / 2 with an activation
};

// One output, channel c of token t.
__device__ __forceinline__ void store_one(const Gemm& p, int64_t t, int c, float v) {
  if (p.add) v += __uint_as_float((uint32_t)p.add[t * p.No + c] << 16);
  p.out[t * p.No + c] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// ---------------------------------------------------------------- few tokens: weights streamed
//
// A workgroup takes one 16-channel block (with an activation the gate block and the up block of
// the same outputs) and 16 tokens; its waves split K and add their sums through LDS.  The weights
// are read once, from packed blocks of whole lines, straight into the operand registers, up to
// eight blocks (and as many of the gate) in flight per wave before the first MFMA; what is left of a
// wave's share after whole trips of eight is asked for as it is.  Bound by the weights' bytes: 7168 x K at
// 1 token, cold, us at K 512, 1024, 2048, 3584, 4096, 5120, 7168, 8192: 3.8, 4.3, 5.1, 7.0, 7.5, 9.1, 11.5, 12.9;
// six in flight 3.2, 4.2, 5.2, 7.2, 7.9, 8.4, 11.5, 12.2; the last trip filled up with repeated blocks 3.7, 4.3, 5.5,
// 7.2, 7.8, 10.9, 12.6, 13.0, and with seven in flight 3.8, 4.4, 5.5, 7.1, 9.2, 10.7, 11.8, 14.4.

constexpr int STREAM_U = 8;                   // K blocks a wave loads together
constexpr int STREAM_WAVES = 8;               // waves of a workgroup, at most

template <bool ACT>
__global__ __launch_bounds__(STREAM_WAVES * 64) void gemm_i8_stream_kernel(const Gemm p, int blocks_k) {
  constexpr int NB = ACT ? 2 : 1;
  __shared__ v4i sums[STREAM_WAVES][NB][64];
  // the wave's number in a scalar register: what it decides are branches, and an MFMA under a lane mask
  // would run with the mask ignored
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const uint8_t* wp[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
    wp[b] = p.w + ((int64_t)blockIdx.x + (b ? p.No / 16 : 0)) * blocks_k * 1024 + lane * 16;
  const uint8_t* const ap = p.a + (int64_t)min(r, p.T - 1) * p.K;
  v4i acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = v4i{0, 0, 0, 0};
  const int steps = (p.K + 63) / 64;                          // the padding past them is not read
  const int per = (steps + waves - 1) / waves;
  const int s1 = min((wave + 1) * per, steps);
  // blocks s0 .. s0 + STREAM_U - 1, or (not whole) as many of them as this wave has left
  const auto trip = [&](const int s0, auto whole) {
    uint4 wv[STREAM_U][NB], av[STREAM_U];
#pragma unroll
    for (int j = 0; j < STREAM_U; ++j) {
      const int s = s0 + j;
      if (!decltype(whole)::value && s >= s1) break;
#pragma unroll
      for (int b = 0; b < NB; ++b) wv[j][b] = ldw16(wp[b] + (int64_t)s * 1024);
      av[j] = *reinterpret_cast<const uint4*>(ap + min(s * 64 + g * 16, p.K - 16));   // past K the weights are zero
    }
#pragma unroll
    for (int j = 0; j < STREAM_U; ++j) {
      if (!decltype(whole)::value && s0 + j >= s1) break;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, wv[j][b]), __builtin_bit_cast(v4i, av[j]),
                                                       acc[b], 0, 0, 0);
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
  const float sa = p.sa[r];
#pragma unroll
  for (int i = 0; i < 4; ++i) {                               // channels 4 g .. 4 g + 3 of token r
    const int c = blockIdx.x * 16 + 4 * g + i;
    if (c < p.No) {
      float v = (float)acc[0][i] * (sa * p.sw[c]);
      if constexpr (ACT) v = activate(p, v, (float)acc[1][i] * (sa * p.sw[p.No + c]));
      store_one(p, r, c, v);
    }
  }
}

// ---------------------------------------------------------------- more tokens: LDS tiles
//
// Tiles of BM tokens x BN weight rows, K in steps of 128 bytes through S LDS buffers filled by the
// load-to-LDS copies (S - 1 steps in flight).  GM x GN waves, each BM/GM tokens x BN/GN weight rows
// with 32x32x32 MFMAs; with KG > 1 that many groups of waves share out K and add their sums through
// LDS.  The operands of the next quarter step are read while the matrix cores work on the present
// one, also across the barrier between two steps.
//
// A copy instruction takes 8 token rows x 128 bytes (whole lines: 16 rows x 64 bytes ran at half
// the rate), its 16-byte pieces placed at p ^ ((row / 2) % 8) so that the 16 lanes that read one
// piece of 16 rows hit distinct banks, or one 1 KB weight block, which stays in lane order.  LDS
// bank conflicts: none counted.
//
// Measured (cold weights and tokens, K 3584): one round of tiles on 256 CUs takes 8.1 us at 32 x 64
// (KG 4), 10.2 at 64 x 64 (KG 2), 11.6 at 64 x 64, 18 at 128 x 128, 28 at 128 x 256 and 48 at
// 256 x 256: the smaller the tile, the more it is bound by the copies, which run at 45 to 50 bytes
// a nanosecond and CU (140 from a warm L2).  At 8192^3 the 256 x 256 tiles take 489 us in the first launch
// of a row (2250 TOP/s; a library product 2029) and 523 in the sixth: the clock falls from 1.8 to 1.54 GHz
// and the share of the time that the matrix cores are busy rises from 56 to 63%.  8192 x 7168 x 3584 with
// SiTUv2: 225 us, 1.9 GHz, 45%.  Without the copies the loop runs 1.5 times as fast, without the MFMAs 1.2 times.

template <int BM, int BN, int GM, int GN, int S, int KG, bool ACT>
struct Tile {
  static constexpr int WAVES = GM * GN, THREADS = WAVES * KG * 64;
  static constexpr int BUF = (BM + BN) * 128, LDS = KG * S * BUF;
};

template <int BM, int BN, int GM, int GN, int S, int KG, bool ACT>
__device__ __forceinline__ void tile_body(const Gemm& p, int blocks_k, int tm, int tn, uint8_t* lds_all) {
  using T = Tile<BM, BN, GM, GN, S, KG, ACT>;
  constexpr int WAVES = T::WAVES, BUF = T::BUF;
  constexpr int WM = BM / GM, WN = BN / GN;                   // one wave's tokens and weight rows
  constexpr int FM = WM / 32, FN = WN / 32;                   // its 32-row operands
  constexpr int A_BYTES = BM * 128;
  constexpr int QA = BM / 8 / WAVES, QB = BN / 8 / WAVES;     // copy instructions of a wave and step
  constexpr int Q = QA + QB;
  static_assert(!ACT || FN % 2 == 0, "gate and up operands in pairs");
  static_assert(QA * 8 * WAVES == BM && QB * 8 * WAVES == BN && (S - 2) * Q < 63 && S >= 2 && S <= 4, "whole copies");
  static_assert(KG == 1 || (KG - 1) * WAVES * FN * FM * 4096 <= T::LDS, "the groups' sums fit");
  const int all = blocks_k / 2, most = (all + KG - 1) / KG;   // every step starts inside K
  const int lane = threadIdx.x & 63, wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KG == 1 ? 0 : wave_all / WAVES, wave = KG == 1 ? wave_all : wave_all % WAVES;
  const int first = kg * most, steps = max(min(most, all - first), 0);   // this group's steps
  uint8_t* const lds = lds_all + kg * (S * BUF);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int wm = wave % GM, wn = wave / GM;
  const int t0 = tm * BM;
  const int c0 = ACT ? tn * (BN / 2) : tn * BN;               // first output channel

  // per-lane source offsets of this wave's copies
  const uint8_t* const a_base = p.a + (int64_t)t0 * p.K;
  uint32_t a_off[QA], b_off[QB];
  int a_piece[QA];
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int row = (wave + WAVES * q) * 8 + (lane >> 3);
    a_piece[q] = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
    a_off[q] = (uint32_t)min(row, p.T - 1 - t0) * (uint32_t)p.K + a_piece[q];
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) {
    const int blk = wave + WAVES * q, rg = blk >> 1;          // 16-row group of the tile, half step
    int f;
    if (ACT) {                                                // each wave's rows: its gate rows, then the up rows
      const int w = rg / (WN / 16), i = rg % (WN / 16), half = WN / 32;
      const int gf = min(c0 / 16 + w * half + i % half, p.No / 16 - 1);
      f = i < half ? gf : p.No / 16 + gf;
    } else {
      f = min(c0 / 16 + rg, (p.N + 15) / 16 - 1);
    }
    b_off[q] = (uint32_t)f * (uint32_t)blocks_k * 1024u + (blk & 1) * 1024 + lane * 16;
  }
  int fill = 0;                                               // the buffer that the next step's copies fill
  const auto fetch = [&](int st) {
    const uint32_t buf = lds0 + fill * BUF;
    fill = fill + 1 == S ? 0 : fill + 1;
    st += first;
    const int left = p.K - st * 128;                          // bytes of a row from this step on, >= 16
    const uint8_t* ab = a_base + st * 128;
    const uint8_t* bb = p.w + (int64_t)st * 2048;
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      uint32_t off = a_off[q];
      if (left < 128) off -= max(a_piece[q] + 16 - left, 0);  // past K the weights are zero: any bytes of the row
      copy16(ab, off, buf + (wave + WAVES * q) * 1024);
    }
#pragma unroll
    for (int q = 0; q < QB; ++q) copy16(bb, b_off[q], buf + A_BYTES + (wave + WAVES * q) * 1024);
  };

  v16i acc[FN][FM];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[n][m][i] = 0;

  // 32-row operands, quarter step ss: lane l holds bytes 32 ss + 16 (l / 32) .. + 15 of row l % 32
  const int l32 = lane & 31, hl = lane >> 5;
  const uint8_t* const fa = lds + (wm * WM + l32) * 128;
  const int a_swz = (l32 >> 1) & 7;                           // a wave's rows start at a multiple of 32
  const uint8_t* const fb = lds + A_BYTES + wn * (WN / 16) * 2048 + (l32 >> 4) * 2048 + (hl * 16 + (lane & 15)) * 16;
  v4i av[2][FM], bv[2][FN];
  const auto read = [&](int set, int buf, int ss) {
#pragma unroll
    for (int n = 0; n < FN; ++n)
      bv[set][n] = *reinterpret_cast<const v4i*>(fb + buf * BUF + (ss >> 1) * 1024 + (ss & 1) * 512 + n * 4096);
#pragma unroll
    for (int m = 0; m < FM; ++m)
      av[set][m] = *reinterpret_cast<const v4i*>(fa + buf * BUF + (((2 * ss + hl) ^ a_swz) * 16) + m * 4096);
  };
  const auto mul = [&](int set) {
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int m = 0; m < FM; ++m)
        acc[n][m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bv[set][n], av[set][m], acc[n][m], 0, 0, 0);
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
  meet(min(steps - 1, S - 2));
  int buf = 0;
  if (KG == 1 || steps > 0) read(0, 0, 0);
  for (int st = 0; st < most; ++st) {                         // as many steps, so barriers, for every group
    // the buffer of step st - 1 is free: every wave has passed the barrier after reading it
    if (st + S - 1 < steps) fetch(st + S - 1);
    const bool work = KG == 1 || st < steps;
    if (work) {
#pragma unroll
      for (int ss = 0; ss < 3; ++ss) {
        read((ss + 1) & 1, buf, ss + 1);
        mul(ss & 1);
      }
    }
    buf = buf + 1 == S ? 0 : buf + 1;
    if (st + 1 < most) {
      meet(min(steps - 2 - st, S - 2));
      if (KG == 1 || st + 1 < steps) read(0, buf, 0);
    }
    if (work) mul(1);
  }
  if constexpr (KG > 1) {                                     // the groups' sums, added by the first group
    v4i* const part = reinterpret_cast<v4i*>(lds_all);
    constexpr int V = FN * FM * 4;
    __syncthreads();                                          // every operand read is done
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const v16i& x = acc[i / 4 / FM][i / 4 % FM];
        part[(((kg - 1) * WAVES + wave) * V + i) * 64 + lane] = v4i{x[i % 4 * 4], x[i % 4 * 4 + 1], x[i % 4 * 4 + 2], x[i % 4 * 4 + 3]};
      }
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int k = 0; k < KG - 1; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const v4i y = part[((k * WAVES + wave) * V + i) * 64 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i / 4 / FM][i / 4 % FM][i % 4 * 4 + j] += y[j];
      }
  }

  // epilogue: register i of lane l is weight row 8 (i / 4) + 4 (l / 32) + i % 4, token l % 32
  // Eight channels go out together wherever a row starts (the loads and stores of global memory need
  // no alignment): 7508 x 866 x 320 with add 14.3 us, 38 with an element at a time; 2000 x 4099 x 512
  // 25 and 41.  Rows in multiples of 16 bytes take as long as with aligned accesses.
  constexpr int FO = ACT ? FN / 2 : FN;                       // 32-channel groups of outputs
#pragma unroll
  for (int n = 0; n < FO; ++n) {
    const int cw = c0 + wn * (FO * 32) + n * 32;              // first channel of the group
    float sw[16], sw_up[ACT ? 16 : 1];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int c = min(cw + 8 * (i / 4) + 4 * hl + i % 4, p.No - 1);
      sw[i] = p.sw[c];
      if constexpr (ACT) sw_up[i] = p.sw[p.No + c];
    }
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const int64_t t = t0 + wm * WM + m * 32 + (lane & 31);
      const float sa = t < p.T ? p.sa[t] : 0.0f;
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i] = (float)acc[n][m][i] * (sa * sw[i]);
        if constexpr (ACT) v[i] = activate(p, v[i], (float)acc[n + FO][m][i] * (sa * sw_up[i]));
      }
      // halves of two 8-channel groups exchanged: lanes 0..31 hold the first, 32..63 the second
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[8 * j + i]), __float_as_uint(v[8 * j + 4 + i]),
                                                          false, false);
          w[i] = __uint_as_float(s[0]);
          w[4 + i] = __uint_as_float(s[1]);
        }
        const int c = cw + 16 * j + 8 * hl;
        if (t < p.T && c + 8 <= p.No) {
          if (p.add) {
            float o[8];
            load_any<8>(p.add + t * p.No + c, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] += o[i];
          }
          store_any<8>(p.out + t * p.No + c, w);
        } else if (t < p.T) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < p.No) store_one(p, t, c + i, w[i]);
        }
      }
    }
  }
}

template <int BM, int BN, int GM, int GN, int S, int KG, bool ACT>
__global__ __launch_bounds__(GM * GN * KG * 64) void gemm_i8_tile_kernel(const Gemm p, int blocks_k, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tile<BM, BN, GM, GN, S, KG, ACT>::LDS];
  int tm, tn;
  tile_of(run_of_xcd(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
  tile_body<BM, BN, GM, GN, S, KG, ACT>(p, blocks_k, tm, tn, lds);
}

// 256 x 256 tiles; those past the first `full` are taken in two halves of 128 tokens each, so that
// a last round that would leave half of the CUs idle takes half as long.
template <bool ACT>
__global__ __launch_bounds__(512) void gemm_i8_big_kernel(const Gemm p, int blocks_k, int tiles_m, int tiles_n, int full) {
  using Half = Tile<128, 256, 2, 4, 3, 1, ACT>;
  static_assert(Half::LDS >= Tile<256, 256, 2, 4, 2, 1, ACT>::LDS, "both shapes share the LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Half::LDS];
  int tm, tn;
  if ((int)blockIdx.x < full) {
    tile_of(run_of_xcd(blockIdx.x, full), tiles_m, tiles_n, tm, tn);
    tile_body<256, 256, 2, 4, 2, 1, ACT>(p, blocks_k, tm, tn, lds);
  } else {
    const int h = run_of_xcd(blockIdx.x - full, gridDim.x - full);
    tile_of(full + (h >> 1), tiles_m, tiles_n, tm, tn);
    tm = 2 * tm + (h & 1);
    if (tm * 128 < p.T) tile_body<128, 256, 2, 4, 3, 1, ACT>(p, blocks_k, tm, tn, lds);
  }
}

template <bool ACT>
int64_t tiles(const Gemm& p, int bm, int bn) {
  const int cols = ACT ? bn / 2 : bn;
  return (int64_t)((p.T + bm - 1) / bm) * ((p.No + cols - 1) / cols);
}

template <int BM, int BN, int GM, int GN, int S, int KG, bool ACT>
void tile(const Gemm& p, int blocks_k, hipStream_t s) {
  using T = Tile<BM, BN, GM, GN, S, KG, ACT>;
  const int tm = (p.T + BM - 1) / BM;
  const int64_t n = tiles<ACT>(p, BM, BN);
  gemm_i8_tile_kernel<BM, BN, GM, GN, S, KG, ACT><<<(unsigned)n, T::THREADS, 0, s>>>(p, blocks_k, tm, (int)(n / tm));
}

// Up to 16 tokens the weights are streamed; beyond, the smallest tiles that one round of CUS
// workgroups holds (they take K in more groups), then the largest of which there is more than a
// round.  Measured, us, chosen ones in brackets, in the order 32 x 64 in four groups, 64 x 64 in two, 64 x 64,
// 128 x 128, 256 x 256 (with halves):
//   K 512:   64 x 7168 [4.1] 4.6 4.4 5.9 8.1    256 x 3584 6.6 [4.7] 4.6 6.3 8.8    256 x 7168 11.6 7.8 [5.5] 6.5 9.0
//           384 x 7168 16.6 10.9 8.1 [6.8] 9.2   1024 x 7168 37.4 23.5 15.4 12.5 [11.0]
//   K 1456:  64 x 7168 [6.7] 8.2 7.7 10.6 15.4   256 x 3584 9.3 [6.7] 6.9 10.1 14.7   256 x 7168 19.8 13.7 [11.6] 12.4 17.8
//           384 x 7168 25.2 18.6 15.3 [12.6] 17.8   1024 x 7168 69.1 44.2 31.0 25.2 [20.0]
//   K 3584:  64 x 7168 [10.2] 12.6 12.1 17.6 27   256 x 3584 16.4 [11.5] 11.8 19.1 28.7   256 x 7168 31 21.7 [18.5] 20.4 29.7
//           384 x 7168 38.6 29.6 26.1 [20.7] 30   1024 x 7168 104 68 57 41.5 [33.8]
//   K 7168:  64 x 7168 [17.1] 21.5 20.9 30.6 47.6   256 x 3584 27.3 [19.5] 20.1 34.3 51.5   256 x 7168 51 36.7 [32.6] 35.3 52
//           384 x 7168 64.8 50.4 46.4 [35.4] 51.9   1024 x 7168 176 117 100 72.3 [59.6]
// Streamed at more tokens: 64 x 7168 (gate, up), K 3584: 15.6.
template <bool ACT>
void run(const Gemm& p, int blocks_k, hipStream_t s) {
  constexpr int CUS = 256;
  if (p.T <= 16) {
    const int steps = (p.K + 63) / 64, waves = (steps + STREAM_U - 1) / STREAM_U;
    gemm_i8_stream_kernel<ACT><<<(unsigned)((p.No + 15) / 16), (waves < STREAM_WAVES ? waves : STREAM_WAVES) * 64, 0, s>>>(p, blocks_k);
  } else if (tiles<ACT>(p, 32, 64) <= CUS) {
    tile<32, 64, 1, ACT ? 1 : 2, 3, 4, ACT>(p, blocks_k, s);  // with ACT a wave holds a gate and an up operand
  } else if (tiles<ACT>(p, 64, 64) <= CUS) {
    tile<64, 64, 2, ACT ? 1 : 2, 3, 2, ACT>(p, blocks_k, s);
  } else if (2 * tiles<ACT>(p, 128, 128) <= CUS) {
    tile<64, 64, 2, ACT ? 1 : 2, 4, 1, ACT>(p, blocks_k, s);
  } else if (tiles<ACT>(p, 128, 128) <= CUS) {
    tile<128, 128, 4, 2, 4, 1, ACT>(p, blocks_k, s);
  } else {
    const int64_t n = tiles<ACT>(p, 256, 256);
    const int tm = (p.T + 255) / 256, rest = (int)(n % CUS), full = (int)(2 * rest <= CUS ? n - rest : n);
    gemm_i8_big_kernel<ACT><<<(unsigned)(full + 2 * (n - full)), 512, 0, s>>>(p, blocks_k, tm, (int)(n / tm), full);
  }
}

}  // namespace

hipError_t launch_quant_i8(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* q, float* scale, hipStream_t s) {
  int64_t waves = (cols + 511) / 512;
  if (waves > 16) waves = 16;
  const int64_t slice = MAX_ITEMS / (waves * 64);
  for (int64_t r = 0; r < rows; r += slice) {
    const int64_t n = rows - r < slice ? rows - r : slice;
    quant_i8_kernel<<<(unsigned)n, (unsigned)waves * 64, 0, s>>>(x + r * cols, (int)cols, q + r * cols, scale + r);
  }
  return hipGetLastError();
}

hipError_t launch_pack_i8(const uint8_t* w, int N, int K, uint8_t* out, hipStream_t s) {
  const int blocks_k = (int)(moe_i8_packed_k(K) / 64);
  const int64_t pieces = (int64_t)moe_i8_packed_bytes(N, K) / 16;
  pack_i8_kernel<<<(unsigned)((pieces + 255) / 256), 256, 0, s>>>(w, N, K, blocks_k, pieces, out);
  return hipGetLastError();
}

hipError_t launch_gemm_i8(const GemmI8Args& a, hipStream_t s) {
  Gemm p;
  p.a = a.a;
  p.sa = a.sa;
  p.w = a.w;
  p.sw = a.sw;
  p.add = a.add;
  p.out = a.out;
  p.T = a.T;
  p.N = a.N;
  p.K = a.K;
  p.No = a.act >= 0 ? a.N / 2 : a.N;
  p.set(a.act, a.beta, a.linear_beta);
  const int blocks_k = (int)(moe_i8_packed_k(a.K) / 64);
  if (a.act >= 0) run<true>(p, blocks_k, s);
  else run<false>(p, blocks_k, s);
  return hipGetLastError();
}

}  // namespace moe
