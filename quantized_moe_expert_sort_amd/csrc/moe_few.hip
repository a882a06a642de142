// The routed layer of a few tokens: the choice of the experts and their weights, the layout that the stages
// read, and Stage1 -- in one launch where the batch is small enough that every workgroup can make the
// choice for itself, with a launch of one workgroup before Stage1 else; then Stage2 and the sum.
//
// The stages are those of moe_stage_items.h.  They are bound by the bytes of the weights, which leaves room to
// keep what lies between them more exactly than moe_fused does: with bf16 tokens the intermediate is stored
// in two bf16 parts and both are multiplied (in one part its rounding alone is as large as the output's), the
// weighted rows are added in fp32 without a rounding of their own, and SiTUv2 is the dense products', which
// keeps its digits next to 0.
//
// The choice is the router's (moe_router_choice.h), a wave per token, from fp32 copies of the logits.  A
// token has an expert at most once and there are at most 16 tokens, so every expert that is used has one
// tile of 16 rows: tile i is the i-th used local expert in ascending order, its rows in ascending token.
//
// Measured on MI355X (medians of traced launches): 1 token, 16 of 896 experts, 3584 x 384, bf16: 12.1 us for choice,
// layout and Stage1 (Stage1 alone 8.2; a router's and a sort's launch before it 4.7 and 3.4), 6.6 for Stage2 and the sum;
// 16 tokens, fp8, sigmoid scores with a bias: 11.4 us for choice and layout (16 waves of one CU; 8.3 without the bias,
// whose keys are ranked in 64 bits; the router's kernel alone, over four CUs, 6.6), 46 Stage1 (178 different experts,
// 260 MB of weights, 5.6 TB/s), 24 Stage2 (130 MB, 5.4 TB/s), 4.6 the sum; softmax scores, 223 experts: fp8 8.6,
// 56 (5.9 TB/s), 29 (5.6 TB/s), 4.6, bf16 8.8, 50 (6.5 TB/s), 37 (4.4 TB/s: two products of each weight), 4.8.  Beyond
// 1024 experts with a bias the choice keeps 11 registers in scratch.  The choice in every workgroup of Stage1 beyond
// 4 tokens would take a wave several tokens one after the other.
//
// Beside moe_router, moe_sort and moe_fused (the second figure), us, 16 of 896 experts, softmax scores:
//   tokens                  1            2            4            8            16
//   bf16, in a graph        18.4  21.6   26.8  28.3   43.2  42.6   63.4  65.6   99.1   98.4
//   fp8, in a graph         18.7  22.0   28.5  29.9   41.9  43.7   62.8  68.5   99.7  102.2
//   fp8, called in a row    19    41     29    41     41    44     62    69     99    102
// The gain is the launches'; with many experts' weights to read there is little, or none: 16 tokens with sigmoid scores
// and a bias 88.7 and 87.0 (bf16), 88.2 and 90.6 (fp8).
#include "moe_router_choice.h"

#pragma clang diagnostic ignored "-Winline-asm"   // m0 is written by the load-to-LDS copies
#include "moe_stage2_small.h"

namespace moe {

namespace {

constexpr int MAX_T = MOE_FEW_MAX_TOKENS;

// One wave: lane k < K gets the token's expert of rank k (-1 where none is left) and its weight.
// row: E floats of LDS, cand: CAND entries of LDS, both this wave's own.
template <int NREG, bool BIAS>
__device__ __forceinline__ void route_token(const RouterArgs& a, int t, float* row, uint2* cand, int lane, int& id, float& w) {
  id = -1;
  w = 0.0f;
  if (a.valid && !a.valid[t]) return;                         // the same in every lane
  float l[NREG], best = -INFINITY;
  if (a.dt == MOE_DT_F32) {
    const float* const src = static_cast<const float*>(a.logits) + (int64_t)t * a.E;
#pragma unroll
    for (int i = 0; i < NREG; ++i) l[i] = src[min(i * 64 + lane, a.E - 1)];
  } else {
    const uint16_t* const src = static_cast<const uint16_t*>(a.logits) + (int64_t)t * a.E;
#pragma unroll
    for (int i = 0; i < NREG; ++i) l[i] = __uint_as_float((uint32_t)src[min(i * 64 + lane, a.E - 1)] << 16);
  }
#pragma unroll
  for (int i = 0; i < NREG; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < a.E ? sane(l[i]) : -INFINITY;
    if (e < a.E) row[e] = l[i];
    best = __builtin_fmaxf(best, l[i]);
  }
  wave_sync();
  const float m = wave_max(best);
  if (!(m > -INFINITY)) return;
  float z = 1.0f;
  if (a.score == MOE_SCORE_SOFTMAX && (BIAS || !a.renorm)) {
    z = 0.0f;
#pragma unroll
    for (int i = 0; i < NREG; ++i) z += exp_f(l[i] - m);
    z = wave_sum(z);
  }
  float logit;
  choose<float, 1, NREG, BIAS>(row, l, best, a.bias, a.E, a.K, a.score, m, z, cand, lane, id, logit);
  // with renorm relative to the largest chosen logit: the sum is at least half of that one's term
  float top = a.score == MOE_SCORE_SOFTMAX ? m : 0.0f;
  if (a.renorm) top = __builtin_fminf(wave_max(logit), top);
  const float s = id < 0 ? 0.0f : a.score == MOE_SCORE_SOFTMAX ? exp_f(logit - top) : sigmoid_over(logit, top);
  const float den = a.renorm ? wave_sum(s) : a.score == MOE_SCORE_SOFTMAX ? z : 1.0f;
  w = id < 0 ? 0.0f : a.scale * (s / den);
}

// What Stage1 and Stage2 read of the layout (tiles of 16 rows).
struct FewLayout {
  int32_t* sorted_ids;     // [cap, 16]
  int32_t* expert_ids;     // [cap]
  int32_t* row_of;         // [T * K]
  int cap, expert_begin, E;   // E: local experts
};
__device__ __forceinline__ int local_expert(const FewLayout& o, int id) {
  const int64_t e = (int64_t)id - o.expert_begin;
  return id >= 0 && e >= 0 && e < o.E ? (int)e : -1;
}

// ---------------------------------------------------------------- choice and layout, one workgroup
//
// A wave per token; then, over LDS, the tokens of each expert as a bit mask and the number of used experts
// before it.  One launch of one workgroup instead of a launch of the router and one of the sort.

template <int NREG, bool BIAS>
__global__ __launch_bounds__(1024) void few_route_kernel(const RouterArgs a, const FewLayout o) {
  __shared__ float rows[MAX_T][NREG * 64];
  __shared__ uint2 cand[MAX_T][CAND];
  __shared__ uint32_t tokens_of[NREG * 64];                   // bit t: token t chose the local expert
  __shared__ uint64_t used[NREG];                             // bit i of [b]: expert 64 b + i is used
  const int lane = threadIdx.x & 63, t = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = blockDim.x;
  for (int e = threadIdx.x; e < NREG * 64; e += n) tokens_of[e] = 0;
  for (int i = threadIdx.x; i < o.cap * 16; i += n) o.sorted_ids[i] = a.T * a.K;
  for (int i = threadIdx.x; i < o.cap; i += n) o.expert_ids[i] = -1;
  int id;
  float w;
  route_token<NREG, BIAS>(a, t, rows[t], cand[t], lane, id, w);
  __syncthreads();
  const int e = lane < a.K ? local_expert(o, id) : -1;
  if (lane < a.K) {
    a.ids[t * a.K + lane] = id;
    a.w[t * a.K + lane] = w;
  }
  if (e >= 0) atomicOr(&tokens_of[e], 1u << t);               // bits: in any order
  __syncthreads();
  for (int b = t; b < NREG; b += a.T) {
    const uint64_t m = __ballot(tokens_of[b * 64 + lane] != 0);
    if (lane == 0) used[b] = m;
  }
  __syncthreads();
  if (lane < a.K) {
    int pos = -1;
    if (e >= 0) {
      int tile = 0;
      for (int b = 0; b < NREG; ++b) {
        const uint64_t m = used[b];
        tile += b < (e >> 6) ? __popcll(m) : b == (e >> 6) ? __popcll(m & ((1ull << (e & 63)) - 1ull)) : 0;
      }
      const int j = __popc(tokens_of[e] & ((1u << t) - 1u));
      pos = tile * 16 + j;
      o.sorted_ids[pos] = t * a.K + lane;
      if (j == 0) o.expert_ids[tile] = e;
    }
    o.row_of[t * a.K + lane] = pos;
  }
}

// ---------------------------------------------------------------- Stage1, with or without the choice
//
// NREG > 0: at most 4 tokens and 32 routed rows; each workgroup makes the choice for all of them, a wave per
// token, and works on the tile that it finds for itself; one more workgroup writes the layout that Stage2
// reads.  NREG = 0: the layout is there.

constexpr int FUSED_T = ITEM_WAVES, FUSED_ROWS = SMALL_ROWS;

template <int ADT, int ACT, int NREG, bool BIAS>
__global__ __launch_bounds__(ITEM_THREADS, 2) void few_stage1_kernel(const FusedArgs p, const RouterArgs a, const FewLayout o, int n_nblk) {
  using C = Cfg<ADT, 16>;
  static_assert(C::KW == ITEM_WAVES, "Stage1's waves");
  constexpr int RED = (C::KW * 16 * (2 * C::NI + 1) * 4 + 15) / 16 * 16, STAGE = C::LDSA ? C::KW * AStage<ADT, C::PF1>::BYTES : 0;
  constexpr int ROUTE = FUSED_T * (CAND * 8 + NREG * 64 * 4);
  // Stage1's LDS, and before it the choice's
  __shared__ __attribute__((aligned(16))) uint8_t lds[RED + STAGE > ROUTE ? RED + STAGE : ROUTE];
  __shared__ int ids[FUSED_ROWS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // as stage1_kernel: the column blocks of a tile on one XCD; the workgroup before them writes the layout
  constexpr bool CHOOSE = NREG > 0;
  const bool writer = CHOOSE && blockIdx.x == 0;
  const int item = CHOOSE ? max((int)blockIdx.x - 1, 0) : (int)blockIdx.x, xcd = item & 7, q = item >> 3;
  const int tq = q / n_nblk, tile = tq * 8 + xcd, nb = q - tq * n_nblk;
  if (tile >= o.cap) return;
  const int TK = a.T * a.K;
  int vr[1], expert;
  if constexpr (!CHOOSE) {
    vr[0] = o.sorted_ids[tile * 16 + (lane & 15)];
    expert = o.expert_ids[tile];
    if (!MOE_DCHECK(expert < o.E, DBG_EXPERT) || expert < 0) return;   // -1: an unused tile
    dcheck_row_id(vr[0], TK);
  } else {
    if (wave < a.T) {
      int id;
      float w;
      route_token<NREG, BIAS>(a, wave, reinterpret_cast<float*>(lds + FUSED_T * CAND * 8) + wave * (NREG * 64),
                              reinterpret_cast<uint2*>(lds) + wave * CAND, lane, id, w);
      if (lane < a.K) {
        ids[wave * a.K + lane] = id;
        if (writer) {
          a.ids[wave * a.K + lane] = id;
          a.w[wave * a.K + lane] = w;
        }
      }
    }
    __syncthreads();
    // lane v: routed row v.  Its tile is the number of different local experts below its own.
    const int e = lane < TK ? local_expert(o, ids[lane]) : -1;
    int below = 0, pos = 0;
    for (int v = 0; v < TK; ++v) {
      const int x = __builtin_amdgcn_readlane(e, v);
      const uint64_t same = __ballot(e == x);
      if (x < 0) continue;
      below += (int)__builtin_ctzll(same) == v && x < e;      // counted once per expert
      pos += x == e && v < lane;
    }
    const bool local = e >= 0;
    if (writer) {
      // each entry by the thread that it falls to: no two stores to one address
      const int at = local ? below * 16 + pos : -1;
      for (int i = threadIdx.x; i < o.cap * 16; i += ITEM_THREADS) {
        int v = TK, x = -1;
        for (int k = 0; k < TK; ++k) {
          const int there = __builtin_amdgcn_readlane(at, k);
          v = there == i ? k : v;
          x = there == i ? __builtin_amdgcn_readlane(e, k) : x;
        }
        o.sorted_ids[i] = v;
        if ((i & 15) == 0) o.expert_ids[i >> 4] = x;          // a tile's first row is never padding
      }
      if (wave == 0 && lane < TK) o.row_of[lane] = at;
      return;
    }
    uint64_t mine = __ballot(local && below == tile);         // this tile's rows, in ascending order
    if (mine == 0) return;                                    // an unused tile; the same in every wave
    expert = __builtin_amdgcn_readlane(e, (int)__builtin_ctzll(mine));
    vr[0] = TK;
#pragma unroll
    for (int j = 0; j < FUSED_T; ++j) {                       // a token has an expert at most once
      if (mine == 0) break;
      const int v = (int)__builtin_ctzll(mine);
      mine &= mine - 1;
      vr[0] = (lane & 15) == j ? v : vr[0];
    }
  }
  stage1_rows<ADT, 16, C::NI, C::KW, C::PF1, ACT, false, C::LDSA, ADT == DT_BF16, true>(
      p, tile, nb, vr, expert, reinterpret_cast<float (*)[16][2 * C::NI + 1]>(lds), lds + RED);
}

// ---------------------------------------------------------------- Stage2 and the sum, more than SMALL_ROWS rows

template <int SDT, bool LDSA>
__global__ __launch_bounds__(ITEM_THREADS, 2) void few_stage2_kernel(const FusedArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t astage[LDSA ? S2Stage<SDT, 16>::BYTES : 16];
  using C = Cfg<SDT, 16>;
  auto none = [] {};
  stage2_item<SDT, 16, C::NF2, C::PF2, false, decltype(none)&, LDSA, true>(p, blockIdx.x % p.cap_tiles, blockIdx.x / p.cap_tiles, none,
                                                                          astage);
}

// Thread = four consecutive columns of one token: its rows added in ascending k.
__global__ __launch_bounds__(256) void few_sum_kernel(const FusedArgs p) {
  const int groups = p.D / 4, idx = blockIdx.x * 256 + threadIdx.x;
  if (idx >= p.T * groups) return;
  const int t = idx / groups, c = (idx - t * groups) * 4;
  const float* const rows = reinterpret_cast<const float*>(p.rowout) + c;
  v4f_ sum = {0.f, 0.f, 0.f, 0.f};
  constexpr int KG = 8;
  for (int k0 = 0; k0 < p.topk; k0 += KG) {
    int r[KG];
    token_rows<KG>(p, t, k0, r);
    v4f_ v[KG];
#pragma unroll
    for (int u = 0; u < KG; ++u) v[u] = r[u] >= 0 ? *reinterpret_cast<const v4f_*>(rows + (size_t)r[u] * p.D) : v4f_{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < KG; ++u) sum += v[u];
  }
  *reinterpret_cast<uint2*>(p.out + (size_t)t * p.D + c) = uint2{bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3])};
}

// ---------------------------------------------------------------- launches

template <int NREG, bool BIAS>
hipError_t route(const RouterArgs& a, const FewLayout& o, hipStream_t s) {
  few_route_kernel<NREG, BIAS><<<1, a.T * 64, 0, s>>>(a, o);
  return hipGetLastError();
}

template <int ADT, int ACT, int NREG, bool BIAS>
void stage1(const FusedArgs& p, const RouterArgs& a, const FewLayout& o, hipStream_t s) {
  const int n1 = p.I / Cfg<ADT, 16>::NI;
  const unsigned grid = (unsigned)((int64_t)(o.cap + 7) / 8 * 8 * n1) + (NREG > 0 ? 1 : 0);
  few_stage1_kernel<ADT, ACT, NREG, BIAS><<<grid, ITEM_THREADS, 0, s>>>(p, a, o, n1);
}
template <int ADT, int ACT>
void stage1(const FusedArgs& p, const RouterArgs& a, const FewLayout& o, bool fused, hipStream_t s) {
  if (!fused) stage1<ADT, ACT, 0, false>(p, a, o, s);
  else if (a.E <= 1024) a.bias ? stage1<ADT, ACT, 16, true>(p, a, o, s) : stage1<ADT, ACT, 16, false>(p, a, o, s);
  else a.bias ? stage1<ADT, ACT, 32, true>(p, a, o, s) : stage1<ADT, ACT, 32, false>(p, a, o, s);
}
template <int ADT>
hipError_t stages(const FusedArgs& p, const RouterArgs& a, const FewLayout& o, bool fused, hipStream_t s) {
  if (p.act == ACT_SITUV2) stage1<ADT, ACT_SITUV2>(p, a, o, fused, s);
  else stage1<ADT, ACT_SILU>(p, a, o, fused, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int SDT = ADT == DT_BF16 ? DT_BF16X2 : ADT;       // what the intermediate is stored as
  const int rows = a.T * a.K;
  if (rows <= SMALL_ROWS) {
    const unsigned grid = (unsigned)(p.D / 16);
    if (rows <= 16) stage2_small_kernel<SDT, 16, 16, 1, true><<<grid, 16 * WAVE, 0, s>>>(p);
    else stage2_small_kernel<SDT, 16, 16, 2, true><<<grid, 16 * WAVE, 0, s>>>(p);
    return hipGetLastError();
  }
  using C = Cfg<SDT, 16>;
  const int n2 = (p.D + ITEM_WAVES * C::NF2 * 16 - 1) / (ITEM_WAVES * C::NF2 * 16);
  const unsigned grid = (unsigned)(p.cap_tiles * n2);
  if (p.I <= S2_I_MAX && p.I <= 128 * C::PF2) few_stage2_kernel<SDT, true><<<grid, ITEM_THREADS, 0, s>>>(p);
  else few_stage2_kernel<SDT, false><<<grid, ITEM_THREADS, 0, s>>>(p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  few_sum_kernel<<<(unsigned)((p.T * (p.D / 4) + 255) / 256), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_routed_few(const FusedArgs& p, const RouterArgs& a, int expert_begin, int32_t* sorted_ids, int32_t* expert_ids,
                             int32_t* row_of, hipStream_t s) {
  const FewLayout o{sorted_ids, expert_ids, row_of, p.cap_tiles, expert_begin, p.E};
  hipError_t e = hipSuccess;
  const bool fused = a.T <= FUSED_T && a.T * a.K <= FUSED_ROWS;
  if (!fused)
    e = a.E <= 1024 ? (a.bias ? route<16, true>(a, o, s) : route<16, false>(a, o, s))
                    : (a.bias ? route<32, true>(a, o, s) : route<32, false>(a, o, s));
  if (e != hipSuccess) return e;
  if (p.a_dtype == DT_BF16) return stages<DT_BF16>(p, a, o, fused, s);
  return p.a_dtype == DT_FP8 ? stages<DT_FP8>(p, a, o, fused, s) : stages<DT_FP4>(p, a, o, fused, s);
}

MOE_DEBUG_READER(few)

}  // namespace moe
