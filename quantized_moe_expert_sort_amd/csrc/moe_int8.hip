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
#include "moe_rows.h"

#pragma clang diagnostic ignored "-Winline-asm"   // m0 is written by the load-to-LDS copies

namespace moe {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------- coding of rows

// One row per workgroup of up to 16 waves; 8 elements per lane and step, rows of up to 8 * 1024
// * 2 elements stay in registers between the maximum and the codes, longer ones are read again.
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

struct Gemm {
  const uint8_t* a;        // [T, K]
  const float* sa;         // [T]
  const uint8_t* w;        // packed
  const float* sw;         // [N]
  const uint16_t* add;     // [T, No] or null
  uint16_t* out;           // [T, No]
  int T, N, K, No, act;    // No = N, or N / 2 with an activation
  float beta, inv_beta, lb, inv_lb;
};

__device__ __forceinline__ float activate(const Gemm& p, float g, float u) {
  return p.act == MOE_ACT_SITUV2 ? situv2(g, u, p.beta, p.inv_beta, p.lb, p.inv_lb) : silu_mul(g, u);
}

// One output, channel c of token t.
__device__ __forceinline__ void store_one(const Gemm& p, int64_t t, int c, float v) {
  if (p.add) v += __uint_as_float((uint32_t)p.add[t * p.No + c] << 16);
  p.out[t * p.No + c] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// ---------------------------------------------------------------- few tokens: weights streamed
//
// A workgroup takes one 16-channel block (with an activation the gate block and the up block of
// the same outputs) and up to 16 * MT tokens; its waves split K and add their sums through LDS.
// The weights are read once, from packed blocks of whole lines, straight into the operand
// registers.  Bound by the weights' bytes.

template <int MT, bool ACT>
__global__ __launch_bounds__(1024) void gemm_i8_stream_kernel(const Gemm p, int blocks_k) {
  constexpr int NB = ACT ? 2 : 1;
  extern __shared__ __align__(16) uint8_t lds[];
  v4i* const sums = reinterpret_cast<v4i*>(lds);              // [waves][NB * MT][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.y * 16 * MT;
  const uint8_t* wp[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
    wp[b] = p.w + ((int64_t)blockIdx.x + (b ? p.No / 16 : 0)) * blocks_k * 1024 + lane * 16;
  const uint8_t* ap[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) ap[m] = p.a + (int64_t)min(t0 + 16 * m + r, p.T - 1) * p.K;
  v4i acc[NB][MT];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[b][m] = v4i{0, 0, 0, 0};
  const int per = (blocks_k + waves - 1) / waves;
  const int s1 = min((wave + 1) * per, blocks_k);
#pragma unroll 4
  for (int s = wave * per; s < s1; ++s) {
    uint4 wv[NB], av[MT];
#pragma unroll
    for (int b = 0; b < NB; ++b) wv[b] = ldw16(wp[b] + (int64_t)s * 1024);
    const int k = min(s * 64 + g * 16, p.K - 16);             // past K the weights are zero
#pragma unroll
    for (int m = 0; m < MT; ++m) av[m] = *reinterpret_cast<const uint4*>(ap[m] + k);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        acc[b][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, wv[b]), __builtin_bit_cast(v4i, av[m]),
                                                          acc[b][m], 0, 0, 0);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int m = 0; m < MT; ++m) sums[(wave * NB * MT + b * MT + m) * 64 + lane] = acc[b][m];
  __syncthreads();
  // wave m finishes token tile m: lane (g, r) has channels 4 g .. 4 g + 3 of token r
  for (int m = wave; m < MT; m += waves) {
    v4i tot[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      tot[b] = v4i{0, 0, 0, 0};
      for (int w = 0; w < waves; ++w) tot[b] += sums[(w * NB * MT + b * MT + m) * 64 + lane];
    }
    const int64_t t = t0 + 16 * m + r;
    if (t < p.T) {
      const float sa = p.sa[t];
      const int c0 = blockIdx.x * 16 + 4 * g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + i;
        if (c < p.No) {
          float v = (float)tot[0][i] * (sa * p.sw[c]);
          if constexpr (ACT) v = activate(p, v, (float)tot[1][i] * (sa * p.sw[p.No + c]));
          store_one(p, t, c, v);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- many tokens: LDS tiles
//
// Tiles of BM tokens x BN weight rows, K in steps of 128 bytes through two LDS buffers filled by
// the load-to-LDS copies.  Four waves in a 2 x 2 grid, each BM/2 x BN/2 with 32x32x32 MFMAs; LDS
// holds the operands as the same 1 KB blocks of 16 rows x 64 bytes in lane order, so a copy
// instruction fills a block and an operand read is two runs of 256 consecutive bytes per half wave.
// The operands of the next quarter step are read while the matrix cores work on the present one,
// also across the barrier between two steps.

__device__ __forceinline__ void copy16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory", "m0");
}

template <int BM, int BN, bool ACT>
__global__ __launch_bounds__(256) void gemm_i8_tile_kernel(const Gemm p, int blocks_k, int tiles_m, int tiles_n) {
  constexpr int WM = BM / 2, WN = BN / 2;                     // one wave's tokens and weight rows
  constexpr int FM = WM / 32, FN = WN / 32;                   // its 32-row operands
  constexpr int A_BYTES = BM * 128, BUF = (BM + BN) * 128;
  constexpr int QA = BM / 16 * 2 / 4, QB = BN / 16 * 2 / 4;   // copy instructions of a wave and step
  static_assert(!ACT || FN % 2 == 0, "gate and up operands in pairs");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * BUF];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;

  // Workgroup b runs on XCD b % 8.  Each XCD takes a run of consecutive tiles, in columns of GM
  // tiles down the tokens, so that the tiles it works on at one time share rows in its L2.
  constexpr int GM = 4;
  const int tiles = tiles_m * tiles_n;
  int id;
  {
    const int x = blockIdx.x & 7, i = blockIdx.x >> 3, q = tiles >> 3, rem = tiles & 7;
    id = x * q + min(x, rem) + i;
  }
  const int per_group = GM * tiles_n, grp = id / per_group, in = id - grp * per_group;
  const int gm = min(GM, tiles_m - grp * GM);
  const int tm = grp * GM + in % gm, tn = in / gm;
  const int t0 = tm * BM;
  const int c0 = ACT ? tn * (BN / 2) : tn * BN;               // first output channel
  const int last_f = (p.N + 15) / 16 - 1;

  // per-lane source offsets of this wave's copies
  const int r = lane & 15, g = lane >> 4;
  const uint8_t* a_base = p.a + (int64_t)t0 * p.K;
  uint32_t a_off[QA], b_off[QB];
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int blk = wave + 4 * q;                             // (16-row group, half step)
    a_off[q] = (uint32_t)min((blk >> 1) * 16 + r, p.T - 1 - t0) * (uint32_t)p.K + (blk & 1) * 64 + g * 16;
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) {
    const int blk = wave + 4 * q, rg = blk >> 1;              // 16-row group of the tile
    int f;
    if (ACT) {                                                // each wave's rows: its gate rows, then the up rows
      const int w = rg / (WN / 16), i = rg % (WN / 16), half = WN / 32;
      const int gf = min(c0 / 16 + w * half + i % half, p.No / 16 - 1);
      f = i < half ? gf : p.No / 16 + gf;
    } else {
      f = min(c0 / 16 + rg, last_f);
    }
    b_off[q] = (uint32_t)f * (uint32_t)blocks_k * 1024u + (blk & 1) * 1024 + lane * 16;
  }
  const int steps = blocks_k / 2;
  const auto fetch = [&](int ks) {
    const uint32_t buf = lds0 + (ks & 1) * BUF;
    const uint8_t* ab = a_base + ks * 128;
    const uint8_t* bb = p.w + (int64_t)ks * 2048;
    const bool tail = ks * 128 + 128 > p.K;
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      const int blk = wave + 4 * q;
      uint32_t off = a_off[q];
      // past K the weights are zero: read the row's last 16 bytes instead
      if (tail) off -= max((blk & 1) * 64 + g * 16 + 16 - (p.K - ks * 128), 0);
      copy16(ab, off, buf + blk * 1024);
    }
#pragma unroll
    for (int q = 0; q < QB; ++q) copy16(bb, b_off[q], buf + A_BYTES + (wave + 4 * q) * 1024);
  };

  v16i acc[FN][FM];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[n][m][i] = 0;

  // operand (16-row groups 2 k, 2 k + 1), quarter step ss: lane l holds row l % 32
  const int frag = ((lane >> 4) & 1) * 2048 + ((lane >> 5) * 16 + r) * 16;
  const uint8_t* const fa = lds + wm * (WM / 16) * 2048 + frag;
  const uint8_t* const fb = lds + A_BYTES + wn * (WN / 16) * 2048 + frag;
  v4i av[2][FM], bv[2][FN];
  const auto read = [&](int set, int ks, int ss) {
    const int at = (ks & 1) * BUF + (ss >> 1) * 1024 + (ss & 1) * 512;
#pragma unroll
    for (int n = 0; n < FN; ++n) bv[set][n] = *reinterpret_cast<const v4i*>(fb + at + n * 4096);
#pragma unroll
    for (int m = 0; m < FM; ++m) av[set][m] = *reinterpret_cast<const v4i*>(fa + at + m * 4096);
  };
  const auto mul = [&](int set) {
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int m = 0; m < FM; ++m)
        acc[n][m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bv[set][n], av[set][m], acc[n][m], 0, 0, 0);
  };
  // every copy of this wave has landed and its LDS reads are done; then meet the other waves
  const auto meet = [&]() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

  fetch(0);
  meet();
  if (steps > 1) fetch(1);
  read(0, 0, 0);
  for (int ks = 0; ks < steps; ++ks) {
    read(1, ks, 1);
    mul(0);
    read(0, ks, 2);
    mul(1);
    read(1, ks, 3);
    mul(0);
    if (ks + 1 < steps) {
      meet();                                                 // buffer ks + 1 is filled, buffer ks is free
      if (ks + 2 < steps) fetch(ks + 2);
      read(0, ks + 1, 0);
    }
    mul(1);
  }

  // epilogue: register i of lane l is weight row 8 (i / 4) + 4 (l / 32) + i % 4, token l % 32
  constexpr int FO = ACT ? FN / 2 : FN;                       // 32-channel groups of outputs
  const int hl = lane >> 5;
  const bool wide = p.No % 8 == 0 && !(((uintptr_t)p.out | (uintptr_t)p.add) & 15);
#pragma unroll
  for (int n = 0; n < FO; ++n) {
    const int cw = c0 + wn * (FO * 32) + n * 32;              // first channel of the group
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const int64_t t = t0 + wm * WM + m * 32 + (lane & 31);
      const float sa = t < p.T ? p.sa[t] : 0.0f;
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int c = min(cw + 8 * (i / 4) + 4 * hl + i % 4, p.No - 1);
        v[i] = (float)acc[n][m][i] * (sa * p.sw[c]);
        if constexpr (ACT) v[i] = activate(p, v[i], (float)acc[n + FO][m][i] * (sa * p.sw[p.No + c]));
      }
      if (wide) {
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
          if (t < p.T && c < p.No) {
            if (p.add) {
              float o[8];
              load_row<8>(p.add + t * p.No + c, o);
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] += o[i];
            }
            store_row<8>(p.out + t * p.No + c, w);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = cw + 8 * (i / 4) + 4 * hl + i % 4;
          if (t < p.T && c < p.No) store_one(p, t, c, v[i]);
        }
      }
    }
  }
}

template <int MT, bool ACT>
void stream(const Gemm& p, int blocks_k, hipStream_t s) {
  const unsigned nb = (unsigned)((p.No + 15) / 16);
  const int waves = blocks_k >= 32 ? 8 : blocks_k >= 8 ? 4 : 2;
  const size_t lds = (size_t)waves * (ACT ? 2 : 1) * MT * 1024;
  gemm_i8_stream_kernel<MT, ACT><<<dim3(nb, (unsigned)((p.T + 16 * MT - 1) / (16 * MT))), waves * 64, lds, s>>>(p, blocks_k);
}

template <int BM, int BN, bool ACT>
void tile(const Gemm& p, int blocks_k, hipStream_t s) {
  const int tm = (p.T + BM - 1) / BM, cols = ACT ? BN / 2 : BN, tn = (p.No + cols - 1) / cols;
  gemm_i8_tile_kernel<BM, BN, ACT><<<(unsigned)(tm * tn), 256, 0, s>>>(p, blocks_k, tm, tn);
}

template <bool ACT>
void run(const Gemm& p, int blocks_k, hipStream_t s) {
  if (p.T <= 16) stream<1, ACT>(p, blocks_k, s);
  else if (p.T <= 32) stream<2, ACT>(p, blocks_k, s);
  else if (p.T <= 64) stream<4, ACT>(p, blocks_k, s);
  else {
    const int64_t big = (int64_t)((p.T + 255) / 256) * ((p.N + 255) / 256);
    if (big >= 192) tile<256, 256, ACT>(p, blocks_k, s);
    else tile<128, 128, ACT>(p, blocks_k, s);
  }
}

}  // namespace

hipError_t launch_quant_i8(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* q, float* scale, hipStream_t s) {
  int64_t waves = (cols + 511) / 512;
  if (waves > 16) waves = 16;
  quant_i8_kernel<<<(unsigned)rows, (unsigned)waves * 64, 0, s>>>(x, (int)cols, q, scale);
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
  p.act = a.act;
  p.No = a.act >= 0 ? a.N / 2 : a.N;
  p.beta = a.beta;
  p.lb = a.linear_beta;
  p.inv_beta = a.act == MOE_ACT_SITUV2 ? 1.0f / a.beta : 0.0f;
  p.inv_lb = a.act == MOE_ACT_SITUV2 ? 1.0f / a.linear_beta : 0.0f;
  const int blocks_k = (int)(moe_i8_packed_k(a.K) / 64);
  if (a.act >= 0) run<true>(p, blocks_k, s);
  else run<false>(p, blocks_k, s);
  return hipGetLastError();
}

}  // namespace moe
