// Per-stage kernels of the fused MXFP4 MoE (one launch per stage) and the dispatch between
// them, the large-batch tiled stages and the single-launch kernel.  The work items themselves
// (Stage1 with the SiTUv2 / SiLU epilogue, Stage2 with the router-weight scaling, the combine)
// are the shared device functions of moe_stage_items.h.
//
// Combine kernel: thread = 8 consecutive columns of one token; it sums that token's routed-row
// outputs (found through the sort's inverse map row_of) in ascending k and rounds to bf16.  Each
// per-row output is read once, a wave reading 1 KB of one row, with the non-temporal hint
// (ldw16): 16% faster at 8192 tokens.
#include <type_traits>

#include "moe_kernels.h"

#pragma clang diagnostic ignored "-Winline-asm"   // m0 is written by the load-to-LDS copies
#include "moe_stage2_small.h"

namespace moe {

namespace {

constexpr int THREADS = ITEM_THREADS;
constexpr int NWAVES = ITEM_WAVES;

// ---------------------------------------------------------------- Stage1

// Workgroup b runs on XCD b % 8 (workgroups are dealt to the eight XCDs round robin).  With
// r = b / 8, it takes column block r % n_nblk of tile (r / n_nblk) * 8 + b % 8: the column blocks
// of a tile are consecutive workgroups of one XCD, so the tile's gathered activation rows are
// fetched into one L2 and re-read from there.  The grid covers cap_tiles rounded up to 8.
template <int ADT, int BM, int NI, int KW, int PF, int MINW, int ACT, bool LDSA>
__global__ __launch_bounds__(KW * WAVE, MINW) void stage1_kernel(FusedArgs p, int n_nblk) {
  __shared__ float red[KW][BM][2 * NI + 1];
  __shared__ __attribute__((aligned(16))) uint8_t astage[LDSA ? KW * AStage<ADT, PF>::BYTES : 16];
  const int xcd = blockIdx.x & 7, r = blockIdx.x >> 3;
  const int tq = r / n_nblk;
  const int tile = tq * 8 + xcd, nb = r - tq * n_nblk;
  if (tile >= p.cap_tiles) return;
  stage1_item<ADT, BM, NI, KW, PF, ACT, false, LDSA>(p, tile, nb, red, astage);
}

// ---------------------------------------------------------------- Stage2
//
// Workgroup (tile, column block nb): blockIdx = nb * cap + tile, so the tiles of one column
// block run together.

template <int ADT, int BM, int NF, int PF, int MINW, bool LDSA>
__global__ __launch_bounds__(THREADS, MINW) void stage2_kernel(FusedArgs p, int cap) {
  __shared__ __attribute__((aligned(16))) uint8_t astage[LDSA ? S2Stage<ADT, BM>::BYTES : 16];
  const int tile = blockIdx.x % cap;
  const int nb = blockIdx.x / cap;
  auto none = [] {};
  stage2_item<ADT, BM, NF, PF, false, decltype(none)&, LDSA>(p, tile, nb, none, astage);
}

// ---------------------------------------------------------------- combine
//
// out[t, c] = sum over k (ascending) of rowout[row_of[t*topk + k], c], in fp32, rounded to
// bf16.  Thread = 8 consecutive columns of one token; rows of non-local experts (-1) are skipped.
// W: the rows were stored without the router weight (grouped Stage2); each is multiplied by
// topk_w[t*topk + k] in fp32 before it is added.  hot_e (with W, may be null): when it lists hot
// experts, a token's slots in hotmask[t] were summed token-major into hot_out[t] (router weight
// applied); the sum then starts from that row and skips those slots.

template <bool W = false>
__global__ __launch_bounds__(THREADS) void combine_kernel(const uint8_t* __restrict__ rowout,
                                                          const int32_t* __restrict__ row_of,
                                                          uint16_t* __restrict__ out, int T, int topk,
                                                          int D, int64_t n_rows,
                                                          const float* __restrict__ topk_w = nullptr,
                                                          const int32_t* __restrict__ hot_e = nullptr,
                                                          const uint32_t* __restrict__ hotmask = nullptr,
                                                          const uint8_t* __restrict__ hot_out = nullptr) {
  const int groups = D / 8;
  const int64_t idx = (int64_t)blockIdx.x * THREADS + threadIdx.x;
  if (idx >= (int64_t)T * groups) return;
  const int t = (int)(idx / groups), c = (int)(idx - (int64_t)t * groups) * 8;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  uint32_t hmask = 0;
  if (W && hot_e && hot_e[MOE_HOT_MAX] > 0) {
    hmask = hotmask[t];
    if (hmask) {
      const uint4 q = ldw16(hot_out + ((size_t)t * D + c) * 2);
      const uint32_t w4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        sum[2 * h] = __uint_as_float(w4[h] << 16);
        sum[2 * h + 1] = __uint_as_float(w4[h] & 0xFFFF0000u);
      }
    }
  }
  // all row indices of a group of KG slots first, then all their row loads, then the sums
  constexpr int KG = 8;
  for (int k0 = 0; k0 < topk; k0 += KG) {
    int r[KG];
#pragma unroll
    for (int u = 0; u < KG; ++u)
      r[u] = k0 + u < topk && !((hmask >> (k0 + u)) & 1u) ? row_of[(int64_t)t * topk + k0 + u] : -1;
#pragma unroll
    for (int u = 0; u < KG; ++u)
      if (!MOE_DCHECK(r[u] >= -1 && r[u] < n_rows, DBG_COMBINE_ROW)) r[u] = -1;
    uint4 q[KG];
    float wk[KG];
#pragma unroll
    for (int u = 0; u < KG; ++u) {
      q[u] = r[u] >= 0 ? ldw16(rowout + ((size_t)r[u] * D + c) * 2) : uint4{0u, 0u, 0u, 0u};
      if (W) wk[u] = r[u] >= 0 ? topk_w[(int64_t)t * topk + k0 + u] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < KG; ++u) {
      const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (W) {
          sum[2 * h] += wk[u] * __uint_as_float(w[h] << 16);
          sum[2 * h + 1] += wk[u] * __uint_as_float(w[h] & 0xFFFF0000u);
        } else {
          sum[2 * h] += __uint_as_float(w[h] << 16);
          sum[2 * h + 1] += __uint_as_float(w[h] & 0xFFFF0000u);
        }
      }
    }
  }
  uint4 o;
  o.x = (uint32_t)f32_to_bf16_rne(sum[0]) | ((uint32_t)f32_to_bf16_rne(sum[1]) << 16);
  o.y = (uint32_t)f32_to_bf16_rne(sum[2]) | ((uint32_t)f32_to_bf16_rne(sum[3]) << 16);
  o.z = (uint32_t)f32_to_bf16_rne(sum[4]) | ((uint32_t)f32_to_bf16_rne(sum[5]) << 16);
  o.w = (uint32_t)f32_to_bf16_rne(sum[6]) | ((uint32_t)f32_to_bf16_rne(sum[7]) << 16);
  *reinterpret_cast<uint4*>(out + (size_t)t * D + c) = o;
}

template <int ADT, int BM>
hipError_t launch_stage2_small(const FusedArgs& a, hipStream_t s) {
  const int rows = a.T * a.topk;
  const dim3 grid((unsigned)(a.D / 16));
  if (rows <= 16) stage2_small_kernel<ADT, BM, 16, 1, false><<<grid, 16 * WAVE, 0, s>>>(a);
  else if (rows <= SMALL_ROWS) stage2_small_kernel<ADT, BM, 16, 2, false><<<grid, 16 * WAVE, 0, s>>>(a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

template <int ADT, int BM>
hipError_t run_stages(FusedArgs a, hipStream_t s) {
  using C = Cfg<ADT, BM>;
  const int n1 = a.I / C::NI;
  const unsigned grid1 = (unsigned)((int64_t)(a.cap_tiles + 7) / 8 * 8 * n1);
  const int n2 = (a.D + NWAVES * C::NF2 * 16 - 1) / (NWAVES * C::NF2 * 16);
  constexpr int T1 = C::KW * WAVE;
  const bool tiled = tiled_path_supported(a);
  const bool tiled1 = tiled && a.T >= TILED_MIN_TOKENS_S1, tiled2 = tiled && a.T >= TILED_MIN_TOKENS_S2;
  if (tiled1 || (tiled2 && !(a.stages & 1))) {
    FusedArgs t = a;
    t.stages = a.stages & ((tiled1 ? 1 : 0) | (tiled2 ? 2 : 0));
    hipError_t err = launch_tiled(t, a.groups, a.num_groups, s);
    if (err != hipSuccess || !(a.stages & 2)) return err;
  } else if (a.stages & 1) {
    // the staged copies address x with 32-bit offsets
    if (C::LDSA && (int64_t)a.T * a.D * 2 < ((int64_t)1 << 31)) {
      if (a.act == ACT_SITUV2)
        stage1_kernel<ADT, BM, C::NI, C::KW, C::PF1, C::MINW1, ACT_SITUV2, C::LDSA><<<grid1, T1, 0, s>>>(a, n1);
      else if (a.act == ACT_SILU)
        stage1_kernel<ADT, BM, C::NI, C::KW, C::PF1, C::MINW1, ACT_SILU, C::LDSA><<<grid1, T1, 0, s>>>(a, n1);
      else
        stage1_kernel<ADT, BM, C::NI, C::KW, C::PF1, C::MINW1, ACT_NONE, C::LDSA><<<grid1, T1, 0, s>>>(a, n1);
    } else {
      if (a.act == ACT_SITUV2)
        stage1_kernel<ADT, BM, C::NI, C::KW, C::PF1, C::MINW1, ACT_SITUV2, false><<<grid1, T1, 0, s>>>(a, n1);
      else if (a.act == ACT_SILU)
        stage1_kernel<ADT, BM, C::NI, C::KW, C::PF1, C::MINW1, ACT_SILU, false><<<grid1, T1, 0, s>>>(a, n1);
      else
        stage1_kernel<ADT, BM, C::NI, C::KW, C::PF1, C::MINW1, ACT_NONE, false><<<grid1, T1, 0, s>>>(a, n1);
    }
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (!(a.stages & 2) || a.act == ACT_NONE) return hipSuccess;
  // the small kernel's copies address the intermediate with 32-bit offsets
  if ((int64_t)a.T * a.topk <= SMALL_ROWS && a.D % 16 == 0 &&
      (int64_t)a.cap_tiles * BM * a.I * 2 < ((int64_t)1 << 31))
    return launch_stage2_small<ADT, BM>(a, s);
  if (!tiled2) {
    const unsigned grid2 = (unsigned)((int64_t)a.cap_tiles * n2);
    // staged intermediate rows: the whole K in one chunk, 32-bit copy offsets
    const int64_t rb = (int64_t)a.I * row_bytes_num<ADT>() / row_bytes_den<ADT>();
    if (a.I <= S2_I_MAX && a.I <= 128 * C::PF2 && (int64_t)a.cap_tiles * BM * rb < ((int64_t)1 << 31))
      stage2_kernel<ADT, BM, C::NF2, C::PF2, C::MINW2, true><<<grid2, THREADS, 0, s>>>(a, a.cap_tiles);
    else
      stage2_kernel<ADT, BM, C::NF2, C::PF2, C::MINW2, false><<<grid2, THREADS, 0, s>>>(a, a.cap_tiles);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  const int64_t nthreads = (int64_t)a.T * (a.D / 8);
  const int64_t n_rows = (int64_t)a.cap_tiles * a.block_m;
  const unsigned gridc = (unsigned)((nthreads + THREADS - 1) / THREADS);
  if (tiled2)   // grouped Stage2 rows carry no router weight
    combine_kernel<true><<<gridc, THREADS, 0, s>>>(a.rowout, a.row_of, a.out, a.T, a.topk, a.D, n_rows, a.topk_w,
                                                   hot_path(a) ? a.hot_e : nullptr, a.hotmask, a.hot_out);
  else
    combine_kernel<false><<<gridc, THREADS, 0, s>>>(a.rowout, a.row_of, a.out, a.T, a.topk, a.D, n_rows);
  return hipGetLastError();
}

template <int ADT>
hipError_t run_dtype(const FusedArgs& a, hipStream_t s) {
  return a.block_m == 16 ? run_stages<ADT, 16>(a, s) : run_stages<ADT, 32>(a, s);
}

}  // namespace

hipError_t launch_fused(const FusedArgs& a, hipStream_t s) {
  return a.a_dtype == DT_BF16 ? run_dtype<DT_BF16>(a, s)
         : a.a_dtype == DT_FP8 ? run_dtype<DT_FP8>(a, s)
                               : run_dtype<DT_FP4>(a, s);
}

MOE_DEBUG_READER(gemm)

}  // namespace moe
