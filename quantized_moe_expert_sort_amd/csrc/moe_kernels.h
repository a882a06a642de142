// Internal interface between the C-ABI entry points (moe_api.hip) and the kernel launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_mi355x.h"

namespace moe {

struct SortLayout {
  int32_t* sorted_ids;
  float* sorted_w;        // may be null
  int32_t* expert_ids;
  int32_t* num_tiles;
  int32_t* row_of;        // may be null
  int32_t* sync;          // may be null; zeroed when given
  int64_t sync_words;
  int64_t cap_tiles;
};

constexpr int MAX_SORT_EXPERTS = MOE_SORT_MAX_EXPERTS;

// ---------------------------------------------------------------- debug checks
//
// Built with -DMOE_DEBUG_CHECKS (the separate library libmoe_mi355x_debug.so), the kernels check
// index invariants they otherwise take from the sort and the host checks: the positions the
// sort writes, the row ids and expert ids the stages read from the layout, the tile ranges of
// the grouped stages and the rows the combine gathers.  A failed check does not trap: it sets
// its bit in the violation word of its source file and the access it guards is skipped (a row
// id outside the layout reads as padding), so the launch ends normally.  Every entry point of
// the debug library then waits for the device, collects and clears the words and returns
// MOE_ERR_DEBUG_CHECK if a bit was set.  In the normal build MOE_DCHECK is `true` and adds no
// code.
enum : uint32_t {
  DBG_SORT_POS = 1u,      // a sorted position past cap_tiles * block_m
  DBG_LAYOUT_ROW = 2u,    // a layout row id outside [0, T*topk] (T*topk marks padding)
  DBG_EXPERT = 4u,        // a tile's expert id >= num_local_experts
  DBG_GROUP = 8u,         // a tile group outside [0, cap_tiles)
  DBG_COMBINE_ROW = 16u,  // a row_of entry outside [-1, cap_tiles * block_m)
};
#ifdef MOE_DEBUG_CHECKS
static __device__ uint32_t dbg_word;   // one per source file
#define MOE_DCHECK(cond, bit) ((cond) ? true : (atomicOr(&::moe::dbg_word, (uint32_t)(bit)), false))
// host side: the word of one source file, cleared after it is read
#define MOE_DEBUG_READER(name)                                                         \
  hipError_t debug_take_##name(uint32_t* v) {                                          \
    const uint32_t z = 0;                                                              \
    hipError_t e = hipMemcpyFromSymbol(v, HIP_SYMBOL(dbg_word), sizeof(uint32_t));     \
    return e != hipSuccess ? e : hipMemcpyToSymbol(HIP_SYMBOL(dbg_word), &z, sizeof(uint32_t)); \
  }
hipError_t debug_take_sort(uint32_t* v);
hipError_t debug_take_gemm(uint32_t* v);
hipError_t debug_take_grouped(uint32_t* v);
hipError_t debug_take_single(uint32_t* v);
hipError_t debug_take_few(uint32_t* v);
#else
#define MOE_DCHECK(cond, bit) true
#define MOE_DEBUG_READER(name)
#endif
// a layout row id (T*topk marks padding; the stages read anything else as padding too)
__device__ __forceinline__ void dcheck_row_id(int v, int TK) { (void)MOE_DCHECK((unsigned)v <= (unsigned)TK, DBG_LAYOUT_ROW); }
// a tile's expert id for a weight address: -1 never reaches here; an id past E reads expert 0
__device__ __forceinline__ int dcheck_expert(int e, int E) { return MOE_DCHECK((unsigned)e < (unsigned)E, DBG_EXPERT) ? e : 0; }

hipError_t launch_sort(const int32_t* topk_ids, const float* topk_w, int64_t n, int expert_begin,
                       int E, int block_m, const SortLayout& L, void* ws, hipStream_t s);

hipError_t launch_quant_act(const uint16_t* x, int64_t rows, int64_t cols, int dt, void* q,
                            uint8_t* scale, hipStream_t s);

struct FusedArgs {
  const uint8_t* x;        // activations (bf16 / fp8 / fp4x2 bytes)
  const uint8_t* xs;       // activation scales or null
  const uint8_t* w1;
  const uint8_t* w1s;
  const uint8_t* w2;
  const uint8_t* w2s;
  const float* topk_w;
  const int32_t* sorted_ids;
  const int32_t* expert_ids;
  const int32_t* num_tiles;
  const int32_t* row_of;   // [T*topk] position of each routed row or -1
  uint8_t* rowout;         // [cap*bm, D] stage2 rows (bf16)
  uint8_t* inter;          // [cap*bm, I] intermediate codes
  uint8_t* inter_s;        // [cap*bm, I/32] intermediate scales (fp8 / fp4)
  int2* groups;            // [cap] tile groups (large-batch path)
  int32_t* num_groups;     // [1]
  int2* cgroups;           // [cap] the groups of experts not taken token-major by Stage2
  int32_t* num_cgroups;    // [1]
  int32_t* tile_hot;       // [cap] hot index of each tile's expert, or -1
  int32_t* hot_e;          // [MOE_HOT_MAX] hot experts, then their count at [MOE_HOT_MAX]
  int32_t* hotpos;         // [T, MOE_HOT_MAX] layout row of (token, hot expert) or the zero row
  float* hotw;             // [T, MOE_HOT_MAX] router weight of (token, hot expert) or 0
  uint32_t* hotmask;       // [T] slots whose expert is hot
  uint8_t* hot_out;        // [T, D] bf16 router-weighted sum of the token's hot-expert rows
  float* dbg;              // [cap*bm, 2I] raw gate/up sums (NONE_TEST) or null
  int32_t* sync;           // completion counters of the single-launch path or null
  uint16_t* out;           // [T, D] bf16
  int T, topk, E, D, I, cap_tiles, block_m, a_dtype, act;
  float beta, linear_beta;
  int stages;              // bit 0: stage1, bit 1: stage2 + finalize
};

hipError_t launch_fused(const FusedArgs& a, hipStream_t s);

// Large-batch stages (moe_gemm_grouped.hip): tile groups of one expert, LDS-tiled GEMMs.
// The tile groups are built with Stage1, so Stage2 takes the grouped path only where Stage1 does.
bool tiled_path_supported(const FusedArgs& a);
// Whether the large-batch Stage2 takes the hot experts token-major (then the combine adds hot_out).
bool hot_path(const FusedArgs& a);
hipError_t launch_tiled(const FusedArgs& a, int2* groups, int32_t* ngroups, hipStream_t s);
constexpr int TILED_MIN_TOKENS_S1 = 2048;   // Stage1 from this batch size
constexpr int TILED_MIN_TOKENS_S2 = 2048;   // Stage2 from this batch size
static_assert(TILED_MIN_TOKENS_S1 <= TILED_MIN_TOKENS_S2, "Stage2 reads Stage1's tile groups");

// Stage1 weights [E, 2I, D/2] and Stage2 weights [E, D, I/2] row-major -> the packed layout of
// moe_pack.hip (same size).
hipError_t launch_pack_w1(const uint8_t* w1, uint8_t* out, int E, int D, int I, hipStream_t s);
hipError_t launch_pack_w2(const uint8_t* w2, uint8_t* out, int E, int D, int I, hipStream_t s);

// Single-launch path (moe_single.hip): Stage1, Stage2 and the combine in one grid whose
// workgroups signal each other through the layout's sync words.
hipError_t launch_single(const FusedArgs& a, hipStream_t s);

// Block norms (moe_norm.hip).  Pointers and options as in moe_block_norm_t; null = not given.
struct NormArgs {
  const void* x;           // [T, D] bf16 or fp32
  const uint16_t* y;       // [T, D] bf16 or null
  const float* w_post;     // [D] or null
  const void* gate;        // by gate_kind
  const float* w_pre;      // [D] or null
  void* h;                 // [T, D] as x, or null
  uint16_t* n;             // [T, D] bf16 or null
  void* q;                 // codes or null
  void* q_scale;
  float* rstd_y;           // [T] 1/rms(y), or null
  float* rstd_h;           // [T] 1/rms(h), or null
  int T, D, x_dt, gate_kind, gate_act, q_dt;
  float scale, eps;
};
struct NormBackwardArgs {
  NormArgs f;              // x, y, w_post, gate, w_pre, rstd and the options of the forward call
  const void* dh;          // [T, D] as x, or null
  const uint16_t* dn;      // [T, D] bf16 or null
  void* dx;                // [T, D] as x
  uint16_t* dy;            // [T, D] bf16 or null
  void* dgate;             // by gate_kind
  float* dw_post;          // [D] or null
  float* dw_pre;           // [D] or null
  float* part;             // [MOE_NORM_PARTS, 3, D] partial sums
};
hipError_t launch_block_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_block_norm_backward(const NormBackwardArgs& a, hipStream_t s);

// Layer norm (moe_layer_norm.hip).  Pointers and options as in moe_layer_norm_t; null = not given.
struct LayerNormArgs {
  const void* x;           // [T, D] bf16 or fp32
  const uint16_t* y;       // [T, D] bf16 or null
  const float* w;          // [D] or null
  const float* b;          // [D] or null
  void* h;                 // [T, D] as x, or null
  uint16_t* n;             // [T, D] bf16 or null
  void* q;                 // codes or null
  void* q_scale;
  float* mean;             // [T], or null
  float* rstd;             // [T], with mean
  int T, D, x_dt, q_dt;
  float eps;
};
struct LayerNormBackwardArgs {
  LayerNormArgs f;         // x, y, w, mean, rstd of the forward call
  const void* dh;          // [T, D] as x, or null
  const uint16_t* dn;      // [T, D] bf16
  void* dx;                // [T, D] as x
  uint16_t* dy;            // [T, D] bf16 or null
  float* dw;               // [D] or null
  float* db;               // [D] or null
  float* part;             // [MOE_NORM_PARTS, 2, D] partial sums
};
hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s);
hipError_t launch_layer_norm_backward(const LayerNormBackwardArgs& a, hipStream_t s);

// Router and balance loss (moe_router.hip), as moe_router_t and moe_balance_t.
struct RouterArgs {
  const void* logits;      // [T, E] bf16 or fp32
  const float* bias;       // [E] or null
  const uint8_t* valid;    // [T] or null
  int32_t* ids;            // [T, K]
  float* w;                // [T, K] (forward)
  int T, E, K, dt, score, renorm;
  float scale;
};
struct BalanceArgs {
  float coef, z_coef;
  int32_t* counts;         // [E]
  float* mean_prob;        // [E]
  float* loss;             // [2]
  int32_t* num_valid;      // [1]
};
hipError_t launch_router(const RouterArgs& a, const BalanceArgs* b, void* ws, hipStream_t s);
hipError_t launch_router_backward(const RouterArgs& a, const BalanceArgs* b, const float* dw, const float* dloss,
                                  void* dlogits, hipStream_t s);

// The routed layer of a few tokens (moe_few.hip): p as for launch_fused with tiles of 16 rows, its layout
// pointers the ones that are written here, topk_w the router's weights.
hipError_t launch_routed_few(const FusedArgs& p, const RouterArgs& a, int expert_begin, int32_t* sorted_ids, int32_t* expert_ids,
                             int32_t* row_of, hipStream_t s);

// Products in 8-bit integers (moe_int8.hip).
struct GemmI8Args {
  const uint8_t* a;        // [T, K] int8
  const float* sa;         // [T]
  const uint8_t* w;        // packed by launch_pack_i8
  const float* sw;         // [N]
  const uint16_t* add;     // [T, No] bf16 or null
  uint16_t* out;           // [T, No] bf16
  int T, N, K, act;        // act < 0: none, No = N; else No = N / 2
  float beta, linear_beta;
};
hipError_t launch_quant_i8(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* q, float* scale, hipStream_t s);
hipError_t launch_pack_i8(const uint8_t* w, int N, int K, uint8_t* out, hipStream_t s);
hipError_t launch_gemm_i8(const GemmI8Args& a, hipStream_t s);

// Microscaled coding and product (moe_mx.hip, moe_mx_gemm.hip), as moe_quant_mx_t and moe_gemm_mx.
struct QuantMxArgs {
  const void* x;           // [rows, cols] bf16 or fp32
  const uint8_t* noise;    // [rows, cols] or null
  void* q;                 // codes of the rows, or null
  uint8_t* q_scale;
  void* t;                 // codes of the transpose's rows, or null
  uint8_t* t_scale;
  int rows, cols, x_dt, q_dt, q_packed, t_dt, t_packed;
};
struct GemmMxArgs {
  const uint8_t* a;        // [T, K] fp8 or [T, K / 2] fp4x2
  const uint8_t* as;       // [T, K / 32]
  const uint8_t* w;        // packed
  const uint8_t* ws;       // packed
  const void* add;         // [T, No] of the output's type, or null
  void* out;               // [T, No] bf16 or fp32
  int T, N, K, a_dt, act, out_dt;   // act < 0: none, No = N; else No = N / 2
  float beta, linear_beta;
};
hipError_t launch_quant_mx(const QuantMxArgs& a, hipStream_t s);
hipError_t launch_pack_mx(const uint8_t* w, const uint8_t* ws, int N, int K, uint8_t* out, uint8_t* out_scale, hipStream_t s);
hipError_t launch_gemm_mx(const GemmMxArgs& a, hipStream_t s);
hipError_t launch_gemm_mx_fp8(const GemmMxArgs& a, hipStream_t s);    // of fp8 tokens, bf16 results
hipError_t launch_gemm_mx_wide(const GemmMxArgs& a, hipStream_t s);   // of fp8 tokens, fp32 results

// Word offsets inside the sync array.  Every counter has a 64-byte line of its own: device-scope
// atomics on one line are serialized (about 11 ns each on gfx950), whatever word they touch.
//   line 0               word 0: sticky timeout flag
//   lines 1 .. cap       Stage1 items finished, per tile
//   next cap lines       Stage2 items finished, per tile
//   next 16*T lines      (row, column block) pairs finished, per (token, column class)
constexpr int64_t SYNC_LINE = 16;
constexpr int64_t SYNC_ERR = 0;
__host__ __device__ inline int64_t sync_done1(int64_t cap, int64_t tile) { (void)cap; return SYNC_LINE * (1 + tile); }
__host__ __device__ inline int64_t sync_done2(int64_t cap, int64_t tile) { return SYNC_LINE * (1 + cap + tile); }
__host__ __device__ inline int64_t sync_token(int64_t cap, int64_t t, int cls) {
  return SYNC_LINE * (1 + 2 * cap + (int64_t)MOE_SYNC_CLASSES * t + cls);
}

}  // namespace moe
