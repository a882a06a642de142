// What the dense products share (moe_int8.hip, moe_mx_gemm.hip): the activations of their epilogues (the
// routed layer of a few tokens has the same), the load-to-LDS copies and the order of tiles.
#pragma once

#include "moe_device.h"
#include "moe_kernels.h"

namespace moe {

namespace {

struct ActArgs {
  int act;                 // < 0: none
  float beta, inv_beta, lb, inv_lb;
  float bl;                // beta lb
  bool apart;              // where that is large and tanh(g / beta) tanh(u / lb) may be below 2^-126: bl is 1, and
                           // beta and lb go to their own factors
  // beta tanh(g / beta) is g from beta = 2^100 on (|g| < 2^88), and beta with g's sign up to beta = 2^-100
  // (|g| > 2^-96): there neither beta nor its inverse grows further, so that nothing leaves fp32's range.
  __host__ __device__ void set(int a, float b, float l) {
    act = a;
    beta = __builtin_fminf(b, 0x1p100f);
    lb = __builtin_fminf(l, 0x1p100f);
    inv_beta = a == MOE_ACT_SITUV2 ? __builtin_fminf(1.0f / beta, 0x1p100f) : 0.0f;
    inv_lb = a == MOE_ACT_SITUV2 ? __builtin_fminf(1.0f / lb, 0x1p100f) : 0.0f;
    apart = beta * lb >= 0x1p40f;
    bl = apart ? 1.0f : beta * lb;
  }
};

// 1 - 2^s for s <= 0.  Near 0 the difference would keep only what 2^s holds beside 1 (1% at s = -1e-5); there
// the first two terms of its series, off by s^2 / 12.5 < 2^-17 of it, beyond them 2^-24 of at least 2^-7.5.
__device__ __forceinline__ float one_minus_exp2(float s) {
  constexpr float LN2 = 0.6931471805599453f;
  const float near = s * __builtin_fmaf(s, -0.5f * LN2 * LN2, -LN2);
  return s > -0x1p-7f ? near : 1.0f - __builtin_amdgcn_exp2f(s);
}
// As situv2, with each tanh to a bf16's last place however small its argument.
__device__ __forceinline__ float situv2_small(float g, float u, const ActArgs& p) {
  constexpr float LOG2E = 1.4426950408889634f;
  const float ag = __builtin_fabsf(g), au = __builtin_fabsf(u);
  const float a = one_minus_exp2(ag * (-2.0f * LOG2E * p.inv_beta));
  const float b = __builtin_amdgcn_exp2f(ag * -LOG2E);
  const float c = one_minus_exp2(au * (-2.0f * LOG2E * p.inv_lb));
  const float d = 2.0f - a, den = __builtin_fmaf(d, b, d) * (2.0f - c);
  float ba = a, bc = c;
  if (p.apart) {
    asm volatile("");                                         // a scalar branch: as selects 2% of a large product
    ba *= p.beta;
    bc *= p.lb;
  }
  const float y = p.bl * (ba * bc * (g < 0.0f ? b : 1.0f)) * __builtin_amdgcn_rcpf(den);
  return __builtin_copysignf(y, __uint_as_float(__float_as_uint(g) ^ __float_as_uint(u)));
}
__device__ __forceinline__ float activate(const ActArgs& p, float g, float u) {
  return p.act == MOE_ACT_SITUV2 ? situv2_small(g, u, p) : silu_mul(g, u);
}

__device__ __forceinline__ void copy16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
// 4 bytes per lane, from any address that is a multiple of 4.
__device__ __forceinline__ void copy4(const void* from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(from) : "memory", "m0");
}

// Tile number `id` of tiles_m x tiles_n: in columns of four tiles down the tokens, so that
// neighbouring numbers share rows.
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int ROWS = 4;
  const int per_group = ROWS * tiles_n, grp = id / per_group, in = id - grp * per_group;
  const int rows = min(ROWS, tiles_m - grp * ROWS);
  tm = grp * ROWS + in % rows;
  tn = in / rows;
}
// Workgroup b runs on XCD b % 8: gives each XCD a run of consecutive numbers out of n, so that the
// tiles it works on at one time share rows in its L2.
__device__ __forceinline__ int run_of_xcd(int b, int n) {
  const int x = b & 7, q = n >> 3, rem = n & 7;
  return x * q + min(x, rem) + (b >> 3);
}

}  // namespace

}  // namespace moe
