// The routed layer of a few tokens: the choice of the experts and their weights, the layout that the stages
// read, and Stage1 -- in one launch where the batch is small enough that every workgroup can make the
// choice for itself, with a launch of one workgroup before Stage1 else; then Stage2 and the sum.
//
// The choice is the router's (moe_router_choice.h), a wave per token, from fp32 copies of the logits.  A
// token has an expert at most once and there are at most 16 tokens, so every expert that is used has one
// tile of 16 rows: tile i is the i-th used local expert in ascending order, its rows in ascending token.
#include "moe_router_choice.h"

#pragma clang diagnostic ignored "-Winline-asm"   // m0 is written by the load-to-LDS copies
#include "moe_stage_items.h"

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

// ---------------------------------------------------------------- choice, layout and Stage1
//
// At most 4 tokens and 32 routed rows: each workgroup makes the choice for all of them, a wave per token,
// and works on the tile that it finds for itself; one more workgroup writes the layout that Stage2 reads.

constexpr int FUSED_T = ITEM_WAVES, FUSED_ROWS = 32;

template <int ADT, int ACT, int NREG, bool BIAS>
__global__ __launch_bounds__(ITEM_THREADS, 2) void few_stage1_kernel(const FusedArgs p, const RouterArgs a, const FewLayout o, int n_nblk) {
  using C = Cfg<ADT, 16>;
  static_assert(C::KW == ITEM_WAVES, "Stage1's waves");
  constexpr int RED = C::KW * 16 * (2 * C::NI + 1) * 4, STAGE = C::LDSA ? C::KW * AStage<ADT, C::PF1>::BYTES : 0;
  constexpr int RED16 = (RED + 15) / 16 * 16;
  constexpr int ROUTE = FUSED_T * (CAND * 8 + NREG * 64 * 4);
  // Stage1's LDS, and before it the choice's
  __shared__ __attribute__((aligned(16))) uint8_t lds[RED16 + STAGE > ROUTE ? RED16 + STAGE : ROUTE];
  __shared__ int ids[FUSED_ROWS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // as stage1_kernel: the column blocks of a tile on one XCD; the workgroup before them writes the layout
  const bool writer = blockIdx.x == 0;
  const int item = max((int)blockIdx.x - 1, 0), xcd = item & 7, q = item >> 3;
  const int tq = q / n_nblk, tile = tq * 8 + xcd, nb = q - tq * n_nblk;
  if (tile >= o.cap) return;
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
  const int TK = a.T * a.K;
  const int e = lane < TK ? local_expert(o, ids[lane]) : -1;
  int below = 0, pos = 0;
  for (int v = 0; v < TK; ++v) {
    const int x = __builtin_amdgcn_readlane(e, v);
    const uint64_t same = __ballot(e == x);
    if (x < 0) continue;
    const bool head = (int)__builtin_ctzll(same) == v;        // counted once per expert
    below += head && x < e;
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
      if ((i & 15) == 0) o.expert_ids[i >> 4] = x;            // a tile's first row is never padding
    }
    if (wave == 0 && lane < TK) o.row_of[lane] = at;
    return;
  }
  uint64_t mine = __ballot(local && below == tile);           // this tile's rows, in ascending order
  if (mine == 0) return;                                      // an unused tile; the same in every wave
  const int expert = __builtin_amdgcn_readlane(e, (int)__builtin_ctzll(mine));
  int vr[1] = {TK};
#pragma unroll
  for (int j = 0; j < FUSED_T; ++j) {                         // a token has an expert at most once
    if (mine == 0) break;
    const int v = (int)__builtin_ctzll(mine);
    mine &= mine - 1;
    vr[0] = (lane & 15) == j ? v : vr[0];
  }
  stage1_rows<ADT, 16, C::NI, C::KW, C::PF1, ACT, false, C::LDSA>(
      p, tile, nb, vr, expert, reinterpret_cast<float (*)[16][2 * C::NI + 1]>(lds), lds + RED16);
}

template <int NREG, bool BIAS>
hipError_t route(const RouterArgs& a, const FewLayout& o, hipStream_t s) {
  few_route_kernel<NREG, BIAS><<<1, a.T * 64, 0, s>>>(a, o);
  return hipGetLastError();
}

template <int ADT, int ACT, int NREG, bool BIAS>
hipError_t route_and_stage1(const FusedArgs& p, const RouterArgs& a, const FewLayout& o, hipStream_t s) {
  const int n1 = p.I / Cfg<ADT, 16>::NI;
  const unsigned grid = (unsigned)((int64_t)(o.cap + 7) / 8 * 8 * n1 + 1);
  few_stage1_kernel<ADT, ACT, NREG, BIAS><<<grid, ITEM_THREADS, 0, s>>>(p, a, o, n1);
  return hipGetLastError();
}
template <int ADT, int ACT>
hipError_t route_and_stage1(const FusedArgs& p, const RouterArgs& a, const FewLayout& o, hipStream_t s) {
  if (a.E <= 1024) return a.bias ? route_and_stage1<ADT, ACT, 16, true>(p, a, o, s) : route_and_stage1<ADT, ACT, 16, false>(p, a, o, s);
  return a.bias ? route_and_stage1<ADT, ACT, 32, true>(p, a, o, s) : route_and_stage1<ADT, ACT, 32, false>(p, a, o, s);
}
template <int ADT>
hipError_t route_and_stage1(const FusedArgs& p, const RouterArgs& a, const FewLayout& o, hipStream_t s) {
  return p.act == ACT_SITUV2 ? route_and_stage1<ADT, ACT_SITUV2>(p, a, o, s) : route_and_stage1<ADT, ACT_SILU>(p, a, o, s);
}

}  // namespace

hipError_t launch_routed_few(const FusedArgs& p, const RouterArgs& a, int expert_begin, int32_t* sorted_ids, int32_t* expert_ids,
                             int32_t* row_of, hipStream_t s) {
  const FewLayout o{sorted_ids, expert_ids, row_of, p.cap_tiles, expert_begin, p.E};
  FusedArgs rest = p;
  hipError_t e;
  if (a.T <= FUSED_T && a.T * a.K <= FUSED_ROWS) {
    e = p.a_dtype == DT_BF16 ? route_and_stage1<DT_BF16>(p, a, o, s)
        : p.a_dtype == DT_FP8 ? route_and_stage1<DT_FP8>(p, a, o, s)
                              : route_and_stage1<DT_FP4>(p, a, o, s);
    rest.stages = MOE_STAGE_2;
  } else {
    e = a.E <= 1024 ? (a.bias ? route<16, true>(a, o, s) : route<16, false>(a, o, s))
                    : (a.bias ? route<32, true>(a, o, s) : route<32, false>(a, o, s));
  }
  return e != hipSuccess ? e : launch_fused(rest, s);
}

MOE_DEBUG_READER(few)

}  // namespace moe
