// Stage2 and the combine in one kernel, for at most SMALL_ROWS routed rows (moe_gemm.hip, moe_few.hip).
#pragma once

#include "moe_stage_items.h"

namespace moe {

namespace {

// ---------------------------------------------------------------- Stage2 + combine, small batches
//
// For at most SMALL_ROWS routed rows (decode), one kernel does Stage2 and the combine: workgroup
// nb owns output columns [16 nb, 16 nb + 16) of every token.  Its sixteen waves take the layout's
// tiles round robin, TPW tiles each (a non-empty expert has at least one routed row per tile, so
// at most T*topk tiles are in use; tiles past num_tiles carry expert -1, so num_tiles itself is
// never read).  A wave issues all of its memory traffic before its first MFMA: it copies the
// intermediate rows of its tiles' routed rows into LDS (one slot per flat row index t*topk + k,
// written and read by this wave only) and loads the weight bytes and scales of all its tiles into
// registers, for SMALL_PS K steps at a time.  For each tile it then computes the 16 x 16 block
// (tile rows x the block's columns) with the MFMA sequence of stage2_item (same operands, K steps
// ascending) and keeps the fp32 sums in LDS.  The token sums run over k ascending: each routed
// row's sum times its router weight, rounded to bf16 as stage2_item stores it, and nothing for
// rows of non-local experts, as the combine kernel adds them: the output has the same bits as
// Stage2 + combine, without the per-row buffer or the extra launch.

constexpr int SMALL_ROWS = MOE_FEW_SMALL_ROWS;
constexpr int SMALL_PS = 3;                           // K steps per pass (inter_dim 384: one pass)

// wait_vm<STEP * n> for a wave-uniform n in [0, 1] (the loads of n later tiles still in flight)
template <int STEP>
__device__ __forceinline__ void wait_vm_n(int n) {
  if (n == 0) wait_vm<0>();
  else wait_vm<STEP>();
}

// s_barrier without the vector-memory wait that __syncthreads adds (loads stay in flight)
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
}

// NW waves of TPW tiles each (16 x 1 or 16 x 2).  More rows per workgroup measured slower than
// the per-tile Stage2 + combine: at 64 routed rows (dec-4) 16 x 4 took 17.8 us and 8 x 8 20.6 us
// against 15.9 (each workgroup then streams 16-column slices of 64 experts' weights).
// WIDE: the weighted rows are not rounded before they are added.
template <int ADT, int BM, int NW, int TPW, bool WIDE>
__global__ __launch_bounds__(NW * WAVE) void stage2_small_kernel(FusedArgs p) {
  static_assert(TPW <= 2, "wait_vm_n covers two tiles per wave");
  constexpr int MF = BM / 16;
  constexpr int SMALL_WAVES = NW, SMALL_THREADS = NW * WAVE;
  constexpr int NR = SMALL_WAVES * TPW;                                    // rows handled
  constexpr int SB = 128 * row_bytes_num<ADT>() / row_bytes_den<ADT>();   // bytes of one K step
  constexpr int SLOT = SMALL_PS * SB;
  static_assert(SLOT % 16 == 0, "whole copies");
  __shared__ float vals[NR][16];
  __shared__ float wsh[NR];
  __shared__ int written[NR];
  __shared__ __attribute__((aligned(16))) uint8_t arows[NR * SLOT + SB];   // + one zero step
  const int nb = blockIdx.x;
  const int lane = threadIdx.x & (WAVE - 1);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / WAVE);   // wave-uniform
  const int r16 = lane & 15, g = lane >> 4;
  const int TK = p.T * p.topk, D = p.D, I = p.I, S = I / 128;
  uint8_t* const zero_step = arows + NR * SLOT;

  // router weight of routed row threadIdx.x: requested first, needed only for the token sums
  const float wmine = (int)threadIdx.x < TK ? p.topk_w[threadIdx.x] : 0.f;
  // expert ids and row ids of every tile of this wave, requested together
  int eid[TPW], vr[TPW][MF];
#pragma unroll
  for (int q = 0; q < TPW; ++q) {   // unconditional loads (a tile past cap reads the last)
    const int tile = min(wave + SMALL_WAVES * q, p.cap_tiles - 1);
    eid[q] = p.expert_ids[tile];
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      vr[q][f] = p.sorted_ids[tile * BM + 16 * f + r16];
      dcheck_row_id(vr[q][f], TK);
    }
  }
  if ((int)threadIdx.x < NR) written[threadIdx.x] = 0;
  if ((int)threadIdx.x < SB / 4) reinterpret_cast<uint32_t*>(zero_step)[threadIdx.x] = 0u;
  lds_barrier();

  bool tv[TPW];   // wave-uniform: the tile has a local expert
  int ew[TPW];    // its expert, or expert 0 (whose rows then serve as in-bounds stand-ins)
#pragma unroll
  for (int q = 0; q < TPW; ++q) {
    const int tile = wave + SMALL_WAVES * q;
    const int e = __builtin_amdgcn_readfirstlane(eid[q]);
    tv[q] = tile < p.cap_tiles && e >= 0 && e < p.E;
    ew[q] = tv[q] ? e : 0;
  }
  const size_t a_row = (size_t)I * row_bytes_num<ADT>() / row_bytes_den<ADT>();
  const uint32_t lds_rows = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)arows);
  v4f acc[TPW][MF];
#pragma unroll
  for (int q = 0; q < TPW; ++q)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[q][f] = v4f{0.f, 0.f, 0.f, 0.f};

  auto pass = [&](int s0, auto full) {
    constexpr bool FULL = decltype(full)::value;
    const int n_s = FULL ? SMALL_PS : S - s0;
    // intermediate rows: one copy per routed row, lanes [0, n_s * SB / 16) of the wave
#pragma unroll
    for (int q = 0; q < TPW; ++q) {
      if (!tv[q]) continue;
      const int tile = wave + SMALL_WAVES * q;
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        uint64_t m = __ballot((unsigned)vr[q][f] < (unsigned)TK) & 0xFFFFull;   // lanes 0..15: rows 0..15
        while (m) {
          const int l = __ffsll((unsigned long long)m) - 1;
          m &= m - 1ull;
          const int v = __builtin_amdgcn_readlane(vr[q][f], l);
          const uint32_t off = (uint32_t)((size_t)(tile * BM + 16 * f + l) * a_row) + (uint32_t)(s0 * SB + 16 * lane);
#pragma unroll
          for (int c = 0; c < SLOT; c += 16 * WAVE)
            if (c + 16 * lane < n_s * SB) dma16_lds(p.inter, off + c, lds_rows + (uint32_t)(v * SLOT + c));
        }
      }
    }
    // scales, then the weights of every tile slot and step, tile after tile; a slot without a
    // local expert loads expert 0's bytes (the same lines for every such slot, served by the L2)
    // so that every wave issues the same loads and a tile's wait below is a fixed count
    ScaleQuads<SMALL_PS> bsq[TPW];
    ScaleQuads<SMALL_PS> asq[TPW][MF];
    uint4 bq[TPW][SMALL_PS];
#pragma unroll
    for (int q = 0; q < TPW; ++q) {
      const size_t wr = (size_t)ew[q] * D + nb * 16 + r16;
      bsq[q].load(p.w2s + wr * (I / 32), s0, s0 + n_s, g, tv[q]);
#pragma unroll
      for (int f = 0; f < MF; ++f)
        if (scaled<ADT>()) {
          const size_t R = (size_t)(wave + SMALL_WAVES * q) * BM + 16 * f + r16;
          asq[q][f].load(p.inter_s + R * (I / 32), s0, s0 + n_s, g, tv[q] && (unsigned)vr[q][f] < (unsigned)TK);
        }
    }
#pragma unroll
    for (int q = 0; q < TPW; ++q) {
      const uint8_t* brow = p.w2 + ((size_t)ew[q] * D + nb * 16) * (I / 2) + 16 * lane;   // packed w2
#pragma unroll
      for (int i = 0; i < SMALL_PS; ++i)
        if (FULL || i < n_s) bq[q][i] = ldw16(brow + (s0 + i) * 1024);
    }
    __builtin_amdgcn_sched_barrier(0);
    auto tile_mfmas = [&](int q) {
      const uint8_t* abase[MF];
      int astep[MF];
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const int v = vr[q][f];
        const bool in = (unsigned)v < (unsigned)TK;
        abase[f] = in ? arows + v * SLOT : zero_step;
        astep[f] = in ? SB : 0;
      }
#pragma unroll
      for (int i = 0; i < SMALL_PS; ++i) {
        if (FULL || i < n_s) {
          const uint32_t bs = bsq[q].get(i, r16, g);
#pragma unroll
          for (int f = 0; f < MF; ++f) {
            AOperand<ADT> A;
            A.load_lds(abase[f] + i * astep[f], g);
            const uint32_t as = !scaled<ADT>() ? 0u : asq[q][f].get(i, r16, g);
            acc[q][f] = A.mma(bq[q][i], bs, as, acc[q][f]);
          }
        }
      }
    };
    // loads complete in order: once at most the later tiles' weight loads are outstanding, the
    // copies, the scales and this tile's weights have arrived
    if constexpr (FULL) {
#pragma unroll
      for (int q = 0; q < TPW; ++q) {
        wait_vm_n<SMALL_PS>(TPW - 1 - q);
        if (tv[q]) tile_mfmas(q);
      }
    } else {
      wait_vm<0>();
#pragma unroll
      for (int q = 0; q < TPW; ++q)
        if (tv[q]) tile_mfmas(q);
    }
    // every LDS read of this pass is done before the next pass's copies replace the rows
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  int s0 = 0;
  for (; s0 + SMALL_PS <= S; s0 += SMALL_PS) pass(s0, std::true_type{});
  if (s0 < S) pass(s0, std::false_type{});

  // fp32 sums of the routed rows: element i of lane (r16, g) is row 4 g + i of the fragment
#pragma unroll
  for (int q = 0; q < TPW; ++q)
#pragma unroll
    for (int f = 0; f < MF; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = __shfl(vr[q][f], 4 * g + i, WAVE);
        if (tv[q] && (unsigned)v < (unsigned)TK) {
          vals[v][r16] = acc[q][f][i];
          if (r16 == 0) written[v] = 1;
        }
      }
  if ((int)threadIdx.x < TK) wsh[threadIdx.x] = wmine;
  __syncthreads();
  for (int idx = threadIdx.x; idx < p.T * 16; idx += SMALL_THREADS) {
    const int t = idx >> 4, c = idx & 15;
    float sum = 0.f;
    for (int k = 0; k < p.topk; ++k) {
      const int v = t * p.topk + k;
      const float o = vals[v][c] * wsh[v];
      if (written[v]) sum += WIDE ? o : __uint_as_float((uint32_t)f32_to_bf16_rne(o) << 16);
    }
    p.out[(size_t)t * D + nb * 16 + c] = f32_to_bf16_rne(sum);
  }
}

}  // namespace

}  // namespace moe
