// Router: scores of a token's experts, the K chosen ones and their weights (what moe_sort and
// moe_fused read), with the balance loss, the z loss and the per-expert counts of the batch taken
// in the same pass over the logits; and the gradient of all of it for the logits.
//
// Row t, expert i:  s = softmax(l) or sigmoid(l);  key = l, or s + bias;  the K largest keys in
// descending order, equal keys by ascending expert;  w = scale s (/ sum of the chosen s).
//   p = softmax(l), or s / sum(s);  P_i = mean_t p_ti;  c_i = how often i was chosen;
//   loss[0] = coef sum_i (c_i E / (K Tv)) P_i;  loss[1] = z_coef mean_t logsumexp(l_t)^2
// over the Tv counted rows.  A logit of -inf or NaN masks its expert, +inf counts as the largest
// finite value; a row whose logits are all masked, or that `valid` leaves out, chooses nothing
// (ids -1, weights 0) and is not counted.
//
// One wave takes a row; each lane keeps up to 32 logits in registers, so the row is read once.
// Choosing K of E: a bound that at least K keys reach is found among the 64 lane maxima (a search
// over the bits of the key, one ballot a bit), the keys at or above it (K to K + a few of 896)
// are compacted to one per lane through LDS, and every lane counts how many of them come before
// its own.  Rows where more than 64 keys reach the bound (a large K, long runs of equal keys) take those
// from the K-th largest key on instead, of experts equal to it the lowest.  With a bias the keys are sums
// whose order could depend on rounding, so the compacted candidates (taken with a margin for the fp32
// error) are ranked by keys in 64 bits; where more than 64 keys lie within that error of the K-th, K
// maxima over the wave choose.
//
// Measured on MI355X (medians of traced launches): 16384 x 896 bf16, K 16: 15 us (29 MB, 6 us at a copy's
// 4.9 TB/s): bound by its instructions and their latency (ordered integer keys and the rare paths in
// registers: 22 us); 16 rows with a bias 6.3 us, 8192 x 896 fp32 with one 26.  8192 x 896 fp32 with the balance
// statistics 17 us and 5.4 for the sums of the workgroups' parts (29 MB); its backward pass 16 us (59 MB, 12 us),
// bound by the bytes.  Of all its kernels only those for more than 1024 experts that 8 does not divide, with a
// bias and statistics, spill registers (61; 3040 x 1177 43 us, 24 without statistics).
#include "moe_kernels.h"
#include "moe_rows.h"

#include <type_traits>

namespace moe {

namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float BIG = 3.402823466e38f;
constexpr int CAND = 64;                      // candidates of a row, at most one per lane
constexpr int HAND = 4;                       // rows of LDS in which waves hand over their sums
constexpr int TURNS = 64;                     // rows that a wave adds up in fp32

// LDS written by some lanes of a wave is read by others of the same wave after this.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * LOG2E); }

// sigmoid(x) e^-m for m <= 0: with m the smaller of 0 and the largest logit, quotients of sigmoids do
// not underflow however negative all of them are.
__device__ __forceinline__ float sigmoid_over(float x, float m) {
  return exp_f(__builtin_fminf(x, 0.0f) - m) * __builtin_amdgcn_rcpf(1.0f + exp_f(-__builtin_fabsf(x)));
}

// The order of the keys as unsigned integers; 0 is left for masked experts.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);               // -0 and +0 are equal keys
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Column of a lane's register i: chunks of 64 * VEC columns, VEC consecutive ones per lane.
template <int VEC>
__device__ __forceinline__ int column(int i, int lane) { return ((i / VEC) * 64 + lane) * VEC + i % VEC; }

// -inf for a masked logit (-inf or NaN: fmaxf returns its other operand), at most `top` otherwise.
__device__ __forceinline__ float sane(float v, float top = BIG) { return __builtin_fminf(__builtin_fmaxf(v, -INFINITY), top); }

// A row's logits as they are in memory (a row ahead of the one that is worked on), and their values;
// lanes past the row read its end, and columns past E hold -inf.
template <class LT, int VEC, int NREG>
struct Row {
  typedef std::conditional_t<sizeof(LT) == 4, float, uint32_t> word;
  static constexpr bool PAIRS = sizeof(LT) == 2 && VEC > 1;   // two bf16 per register
  word raw[PAIRS ? NREG / 2 : NREG];
  __device__ __forceinline__ void load(const LT* row, int E, int lane) {
#pragma unroll
    for (int c = 0; c < NREG / VEC; ++c) {
      const LT* const p = row + min((c * 64 + lane) * VEC, E - VEC);   // E % VEC == 0
      if constexpr (VEC == 8) {
        constexpr int n = PAIRS ? 1 : 2;                      // 16-byte loads
#pragma unroll
        for (int k = 0; k < n; ++k) {
          typedef word word4 __attribute__((ext_vector_type(4)));
          const word4 q = reinterpret_cast<const word4*>(p)[k];
#pragma unroll
          for (int j = 0; j < 4; ++j) raw[(c * n + k) * 4 + j] = q[j];
        }
      } else {
        raw[c] = (word)*p;
      }
    }
  }
  __device__ __forceinline__ void values(int E, int lane, float (&l)[NREG]) const {
#pragma unroll
    for (int i = 0; i < NREG; ++i) {
      const float top = ((i / VEC) * 64 + lane) * VEC < E ? BIG : -INFINITY;
      if constexpr (sizeof(LT) == 4) l[i] = sane(raw[i], top);
      else if constexpr (PAIRS) l[i] = sane(__uint_as_float(i % 2 ? raw[i / 2] & 0xFFFF0000u : raw[i / 2] << 16), top);
      else l[i] = sane(__uint_as_float(raw[i] << 16), top);
    }
  }
};

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, WAVE);
  return v;
}
__device__ __forceinline__ float readlane_f(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ double readlane_d(double v, int l) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), l), __builtin_amdgcn_readlane(__double2loint(v), l));
}

// The selection key in 64 bits.  m, zd: the row's largest logit and sum of exp(l - m) (softmax).
__device__ __forceinline__ double exact_key(float l, float bias, int score, float m, double zd) {
  const double x = (double)l;
  const double e = exp(score == MOE_SCORE_SOFTMAX ? x - (double)m : x < 0.0 ? x : -x);
  const double s = score == MOE_SCORE_SOFTMAX ? e / zd : (x < 0.0 ? e : 1.0) / (1.0 + e);
  return s + (double)bias;
}

// The rare paths read the row again, in loops that are not unrolled: they take no registers from the
// ordinary one.
// The sum of exp(l - m) in 64 bits.
template <class LT>
__device__ __forceinline__ double exact_sum(const LT* row, int E, float m, int lane) {
  double s = 0.0;
#pragma unroll 1
  for (int e = lane; e < E; e += 64) {
    float v[1];
    load_row<1>(row + e, v);
    const float l = sane(v[0]);
    if (l > -INFINITY) s += exp((double)l - (double)m);
  }
  return wave_sum_f64(s);
}
// With a bias: K maxima over the wave, each over every key that is left, in 64 bits.
template <class LT>
__device__ __forceinline__ void choose_in_rounds(const LT* row, const float* bias, int E, int K, int score, float m,
                                                 int lane, int& id, float& logit) {
  const double zd = score == MOE_SCORE_SOFTMAX ? exact_sum(row, E, m, lane) : 1.0;
  uint32_t taken = 0;                                         // E <= 64 * 32
#pragma unroll 1
  for (int r = 0; r < K; ++r) {
    double wk = -INFINITY;
    int wc = 0x7FFFFFFF;
    float wl = -INFINITY;
#pragma unroll 1
    for (int i = 0, e = lane; e < E; e += 64, ++i) {
      float v[1];
      load_row<1>(row + e, v);
      const float l = sane(v[0]);
      if (!(l > -INFINITY) || !(bias[e] > -INFINITY) || ((taken >> i) & 1)) continue;
      const double k = exact_key(l, __builtin_fminf(bias[e], BIG), score, m, zd);
      if (wc == 0x7FFFFFFF || k > wk) { wk = k; wc = e; wl = l; }
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const double ok = __shfl_xor(wk, d, WAVE);
      const int oc = __shfl_xor(wc, d, WAVE);
      const float ol = __shfl_xor(wl, d, WAVE);
      if (oc != 0x7FFFFFFF && (wc == 0x7FFFFFFF || ok > wk || (ok == wk && oc < wc))) { wk = ok; wc = oc; wl = ol; }
    }
    if (wc == 0x7FFFFFFF) break;                              // the same in every lane
    if ((wc & 63) == lane) taken |= 1u << (wc >> 6);
    if (lane == r) { id = wc; logit = wl; }
  }
}

// The fp32 keys with a bias are off by less than half of this: a score by 4e-6 at most (the rounding
// of the exponents, of the sum of up to 2048 exponentials and of the quotient), the sum of score and
// bias by 2^-24 of itself.  So every expert among the K largest exact keys has an fp32 key of at least
// bound - key_margin(bound), where K fp32 keys reach the bound.
__device__ __forceinline__ float key_margin(float bound) { return 1e-5f * (1.0f + __builtin_fabsf(bound)); }

// The candidates of a row that has more than CAND experts above the ordinary bound (many ties, a K near
// half the lanes): those that reach the K-th largest key, of experts with the same logit and bias as it
// only the K with the lowest numbers (the others cannot be chosen).  Returns how many; the first CAND
// of them are in cand.  Without a bias they are fewer than 2 K <= CAND.
// 3400 x 2048 fp32, K 32 (about one row in 50 comes here) 24 us, 172 with K maxima over the whole row
// instead; 16384 x 896 of zeros (every row comes here) 33 us.
template <class LT, int VEC, int NREG, bool BIAS>
__device__ __forceinline__ int collect_from_kth(const LT* row, const float (&l)[NREG], const float (&keys)[BIAS ? NREG : 1],
                                                const float* bias, int E, int K, int score, float m, float z,
                                                float best, uint2* cand, int lane) {
  const auto key = [&](int i) { return BIAS ? keys[i] : l[i]; };
  const auto reach = [&](float v) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < NREG; ++i) n += __popcll(__ballot(key(i) >= v));
    return n;
  };
  // The largest key where K have it (rows of equal logits); else from the top bit down, until just K
  // reach it.
  float kth = wave_max(best);
  if (reach(kth) < K) {
    uint32_t t = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
      const int n = reach(unordered(t | (1u << bit)));
      if (n >= K) t |= 1u << bit;
      if (n == K) break;
    }
    kth = unordered(t);
  }
  const float bound = BIAS ? __builtin_fmaxf(kth - key_margin(kth), -BIG) : kth;
  bool ties = !BIAS;                                          // whether an expert with this very key was found
  float tied_l = kth, tied_b = 0.0f;
  if constexpr (BIAS) {
#pragma unroll
    for (int i = 0; i < NREG; ++i) {
      const uint64_t mask = __ballot(keys[i] == kth);
      if (mask && !ties) {
        const int from = __builtin_ctzll(mask);
        ties = true;
        tied_l = readlane_f(l[i], from);
        tied_b = __builtin_fminf(bias[column<VEC>(i, from)], BIG);
      }
    }
  }
  int n = 0, same = 0;
#pragma unroll 1
  for (int e = lane; e - lane < E; e += 64) {                 // in the experts' order
    const int at = min(e, E - 1);
    float v[1];
    load_row<1>(row + at, v);
    const float x = e < E ? sane(v[0]) : -INFINITY;
    float k = x, b = 0.0f;
    if constexpr (BIAS) {
      const bool left = x > -INFINITY && bias[at] > -INFINITY;
      b = __builtin_fminf(bias[at], BIG);
      k = left ? (score == MOE_SCORE_SOFTMAX ? exp_f(x - m) / z : fast_sigmoid(x)) + b : -INFINITY;
    }
    const bool tied = ties && k > -INFINITY && x == tied_l && b == tied_b;
    const uint64_t all = __ballot(tied);
    const int before = same + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
    same += __popcll(all);
    const bool in = tied ? before < K : k >= bound;
    const uint64_t mask = __ballot(in);
    const int p = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
    if (in && p < CAND) cand[p] = uint2{__float_as_uint(x), (uint32_t)e};
    n += __popcll(mask);
  }
  return n;
}

// One wave's row: on return lane r < K holds the expert of rank r (ascending rank) and its logit, or
// -1 / -inf where none is left.  cand: CAND entries of this wave.  best: the lane's largest logit.
template <class LT, int VEC, int NREG, bool BIAS>
__device__ __forceinline__ void choose(const LT* row, const float (&l)[NREG], float best, const float* bias, int E, int K, int score,
                                       float m, float z, uint2* cand, int lane, int& id, float& logit) {
  id = -1;
  logit = -INFINITY;
  float keys[BIAS ? NREG : 1];
  if constexpr (BIAS) {
    best = -INFINITY;
    const float inv_z = 1.0f / z;
#pragma unroll
    for (int c = 0; c < NREG / VEC; ++c) {
      float b[VEC];
      load_row<VEC>(bias + min((c * 64 + lane) * VEC, E - VEC), b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int i = c * VEC + j;
        const float s = score == MOE_SCORE_SOFTMAX ? exp_f(l[i] - m) * inv_z : fast_sigmoid(l[i]);
        keys[i] = l[i] > -INFINITY && b[j] > -INFINITY ? s + __builtin_fminf(b[j], BIG) : -INFINITY;
        best = __builtin_fmaxf(best, keys[i]);
      }
    }
  }
  const auto key = [&](int i) { return BIAS ? keys[i] : l[i]; };
  // A bound that at least K lane maxima reach, or the lowest number if fewer lanes have one: found
  // from the top bit of the ordered keys down, until few enough reach it.
  const uint32_t ob = best > -INFINITY ? ordered(best) : 0u;
  uint32_t t = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t up = t | (1u << bit);
    const int n = __popcll(__ballot(ob >= up));
    if (n >= K) {
      t = up;
      if (n <= K + 3) break;
    }
  }
  float bound = t ? unordered(t) : -BIG;
  if constexpr (BIAS) {
    bound = __builtin_fmaxf(bound - key_margin(bound), -BIG);
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < NREG; ++i) {
    const bool in = key(i) >= bound;
    const uint64_t mask = __ballot(in);
    if (mask) {
      const int p = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
      if (in && p < CAND) cand[p] = uint2{__float_as_uint(l[i]), (uint32_t)column<VEC>(i, lane)};
      n += __popcll(mask);
    }
  }
  wave_sync();
  if (n > CAND) {
    n = collect_from_kth<LT, VEC, NREG, BIAS>(row, l, keys, bias, E, K, score, m, z, best, cand, lane);
    wave_sync();
  }
  if constexpr (BIAS) {
    if (n > CAND) {                                           // keys closer than their error
      choose_in_rounds(row, bias, E, K, score, m, lane, id, logit);
      return;
    }
  }
  const bool have = lane < n;
  const uint2 c = have ? cand[lane] : uint2{0xFF800000u, 0x7FFFFFFFu};
  const float cl = __uint_as_float(c.x);
  int rank = 0;
  if constexpr (BIAS) {
    const float b = have ? __builtin_fminf(bias[c.y], BIG) : 0.0f;
    double k = 0.0, zd = 1.0;
    bool done = false;
    if (score == MOE_SCORE_SOFTMAX) {
      // fp32 keys decide unless two of them are close: the sum in 64 bits costs more than the rest
      const float k32 = exp_f(cl - m) / z + b;
      bool close = false;
      for (int j = 0; j < n; ++j) {
        const float o = readlane_f(k32, j);
        rank += o > k32;
        close |= j != lane && __builtin_fabsf(o - k32) <= 1e-5f * (1.0f + __builtin_fabsf(k32));
      }
      done = __ballot(have && close) == 0;
      if (!done) zd = exact_sum(row, E, m, lane);
    }
    if (!done) {
      rank = 0;
      if (have) k = exact_key(cl, b, score, m, zd);
      for (int j = 0; j < n; ++j) {
        const double o = readlane_d(k, j);
        const int oc = __builtin_amdgcn_readlane((int)c.y, j);
        rank += o > k || (o == k && oc < (int)c.y);
      }
    }
  } else if constexpr (sizeof(LT) == 2) {
    // bf16: the upper half of the ordered key says it all (rounded up, so that a clamped +inf, the one
    // value that is no bf16, stays above the largest bf16), the column goes below it
    const uint32_t k = ((ordered(cl) + 0xFFFFu) & 0xFFFF0000u) | (0xFFFFu - (c.y & 0xFFFFu));
    for (int j = 0; j < n; ++j) rank += (uint32_t)__builtin_amdgcn_readlane((int)k, j) > k;
  } else {
    const uint64_t k = ((uint64_t)ordered(cl) << 32) | (0xFFFFFFFFu - c.y);
    for (int j = 0; j < n; ++j) {
      const uint64_t o = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), j) << 32) |
                         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, j);
      rank += o > k;
    }
  }
  // to the lane of its rank (ranks of the candidates are 0 .. n - 1, each once)
  wave_sync();
  if (have) cand[rank] = c;
  wave_sync();
  if (lane < min(n, K)) {
    const uint2 r = cand[lane];
    id = (int)r.y;
    logit = __uint_as_float(r.x);
  }
  wave_sync();
}

// ws of the balance statistics: [256] a ticket, [parts] Tv, [parts] z sums, [ceil(E / 64)] loss
// parts, then counts [parts, E] and probability sums [parts, E].
struct BalanceParts {
  int32_t* ticket;
  int32_t* tv;
  float* z;
  float* loss;
  int32_t* counts;
  float* psum;
};
__host__ __device__ inline BalanceParts balance_parts(void* ws, int E) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  BalanceParts b;
  b.ticket = reinterpret_cast<int32_t*>(p);
  b.tv = reinterpret_cast<int32_t*>(p + 256);
  b.z = reinterpret_cast<float*>(p + 256 + 4 * MOE_ROUTER_PARTS);
  b.loss = reinterpret_cast<float*>(p + 256 + 8 * MOE_ROUTER_PARTS);
  b.counts = reinterpret_cast<int32_t*>(p + 256 + 8 * MOE_ROUTER_PARTS + 256);
  b.psum = reinterpret_cast<float*>(b.counts + (size_t)MOE_ROUTER_PARTS * E);
  return b;
}

// Waves of a workgroup: with the balance statistics as many as their registers allow.
template <int NREG, bool BIAS, bool BAL>
constexpr int router_waves() { return !BAL ? 4 : BIAS || NREG > 16 ? 8 : 16; }

// Rows wave, wave + waves of the grid, ...
template <class LT, int VEC, int NREG, bool BIAS, bool BAL>
__global__ __launch_bounds__((64 * router_waves<NREG, BIAS, BAL>())) void router_kernel(const RouterArgs a, void* ws) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane0 = threadIdx.x & 63, lane = lane0, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  uint2* const cand = reinterpret_cast<uint2*>(lds) + wave * CAND;
  double* const zsums = reinterpret_cast<double*>(lds + (size_t)waves * CAND * sizeof(uint2));    // BAL: [waves]
  double* const total = zsums + waves;                                                            // BAL: [E]
  int32_t* const hist = reinterpret_cast<int32_t*>(total + a.E);                                  // BAL: [E]
  float* const handed = reinterpret_cast<float*>(hist + a.E);                                     // BAL: [HAND, E]
  float psum[BAL ? NREG : 1];
  float zsum = 0.0f;
  int tv = 0;
  if constexpr (BAL) {
#pragma unroll
    for (int i = 0; i < NREG; ++i) psum[i] = 0.0f;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *balance_parts(ws, a.E).ticket = 0;
    __syncthreads();
  }
  const int64_t step = (int64_t)gridDim.x * waves;
  int64_t t = (int64_t)blockIdx.x * waves + wave;
  Row<LT, VEC, NREG> ahead;
  if (t < a.T) ahead.load(static_cast<const LT*>(a.logits) + t * a.E, a.E, lane);
  const auto take = [&](const int64_t t) {
    const LT* const row = static_cast<const LT*>(a.logits) + t * a.E;
    // opaque where it is short of registers: the columns' addresses and masks would be kept over the rows
    // and spill (3040 x 1177 with a bias 24 us, 41 with them kept)
    int lane = lane0;
    if constexpr ((BIAS || BAL) && NREG > (VEC == 1 ? 4 : 16)) asm volatile("" : "+v"(lane));
    int id = -1;
    float w = 0.0f;
    float l[NREG];
    ahead.values(a.E, lane, l);
    if (BAL && t + step < a.T) ahead.load(row + step * a.E, a.E, lane);
    if (!a.valid || a.valid[t]) {
      float best = -INFINITY;
#pragma unroll
      for (int i = 0; i < NREG; ++i) best = __builtin_fmaxf(best, l[i]);
      const float m = wave_max(best);
      if (m > -INFINITY) {
        float z = 1.0f;
        if (BAL || (a.score == MOE_SCORE_SOFTMAX && (BIAS || !a.renorm))) {
          z = 0.0f;
          float ex[NREG];
#pragma unroll
          for (int i = 0; i < NREG; ++i) { ex[i] = exp_f(l[i] - m); z += ex[i]; }
          z = wave_sum(z);
          if constexpr (BAL) {
            ++tv;
            const float lse = m + LN2 * __builtin_amdgcn_logf(z);
            zsum += lse * lse;
            if (a.score == MOE_SCORE_SOFTMAX) {
              const float inv = 1.0f / z;
#pragma unroll
              for (int i = 0; i < NREG; ++i) psum[i] += ex[i] * inv;
            } else {
              float s = 0.0f;
#pragma unroll
              for (int i = 0; i < NREG; ++i) { ex[i] = sigmoid_over(l[i], __builtin_fminf(m, 0.0f)); s += ex[i]; }
              const float inv = 1.0f / wave_sum(s);           // at least half of one term
#pragma unroll
              for (int i = 0; i < NREG; ++i) psum[i] += ex[i] * inv;
            }
          }
        }
        float logit;
        choose<LT, VEC, NREG, BIAS>(row, l, best, a.bias, a.E, a.K, a.score, m, z, cand, lane, id, logit);
        // with renorm relative to the largest chosen logit: the sum is at least half of that one's term
        float top = a.score == MOE_SCORE_SOFTMAX ? m : 0.0f;
        if (a.renorm) top = __builtin_fminf(wave_max(logit), top);
        const float s = id < 0 ? 0.0f : a.score == MOE_SCORE_SOFTMAX ? exp_f(logit - top) : sigmoid_over(logit, top);
        const float den = a.renorm ? wave_sum(s) : a.score == MOE_SCORE_SOFTMAX ? z : 1.0f;
        w = id < 0 ? 0.0f : a.scale * (s / den);
        if constexpr (BAL)
          if (id >= 0) atomicAdd(&hist[id], 1);
      }
    }
    if (lane < a.K) {
      a.ids[t * a.K + lane] = id;
      a.w[t * a.K + lane] = w;
    }
  };
  if constexpr (!BAL) {
    for (; t < a.T; t += step) take(t);
  } else {
    // The waves' probability sums of TURNS rows each, HAND waves at a time through LDS; each thread adds
    // its columns in the order of the waves.  Where a wave has more rows, these sums are added in 64 bits:
    // the rounding of the statistics does not grow with the number of rows.
    constexpr int COLS = (64 * NREG + 64 * router_waves<NREG, BIAS, BAL>() - 1) / (64 * router_waves<NREG, BIAS, BAL>());
    const int64_t top = (int64_t)blockIdx.x * waves;
    float sum[COLS];
    for (int64_t from = top;; from += TURNS * step) {
      const int64_t end = min((int64_t)a.T, t + TURNS * step);
      for (; t < end; t += step) take(t);
#pragma unroll
      for (int c = 0; c < COLS; ++c) sum[c] = 0.0f;
      int me = threadIdx.x;                                   // opaque: addresses kept over the rows would spill
      asm volatile("" : "+v"(me));
      for (int base = 0; base < waves; base += HAND) {
        __syncthreads();
        if (wave >= base && wave < base + HAND) {
#pragma unroll
          for (int c = 0; c < NREG / VEC; ++c) {
            const int col = (c * 64 + (me & 63)) * VEC;
            float v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) { v[j] = psum[c * VEC + j]; psum[c * VEC + j] = 0.0f; }
            if (col < a.E) store_row<VEC>(handed + (wave - base) * a.E + col, v);
          }
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
          const int col = min(c * (int)blockDim.x + me, a.E - 1);
#pragma unroll
          for (int k = 0; k < HAND; ++k) sum[c] += handed[k * a.E + col];
        }
      }
      const bool first = from == top, last = from + TURNS * step >= a.T;   // the same for every wave
      if (first && last) break;
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        const int col = c * (int)blockDim.x + me;
        if (col < a.E) {
          total[col] = (first ? 0.0 : total[col]) + sum[c];
          sum[c] = (float)total[col];
        }
      }
      if (lane == 0) zsums[wave] = (first ? 0.0 : zsums[wave]) + zsum;
      zsum = 0.0f;
      if (last) {
        if (lane == 0) zsum = (float)zsums[wave];
        break;
      }
    }
    const BalanceParts b = balance_parts(ws, a.E);
    int* const small = reinterpret_cast<int*>(handed);        // tv and z of each wave
    __syncthreads();
    if (lane == 0) { small[2 * wave] = tv; small[2 * wave + 1] = __float_as_int(zsum); }
    __syncthreads();
    if (threadIdx.x == 0) {
      int n = 0;
      float q = 0.0f;
      for (int i = 0; i < waves; ++i) { n += small[2 * i]; q += __int_as_float(small[2 * i + 1]); }
      b.tv[blockIdx.x] = n;
      b.z[blockIdx.x] = q;
    }
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) b.counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      const int col = c * blockDim.x + threadIdx.x;
      if (col < a.E) b.psum[(int64_t)blockIdx.x * a.E + col] = sum[c];
    }
  }
}

// The batch's statistics from the workgroups' partial sums, 64 experts per workgroup: 16 row
// classes add their partial rows in order, then the classes are added in order.  The workgroup
// that takes the last ticket adds the workgroups' loss parts, in the order of a wave's reduction.
__global__ __launch_bounds__(1024) void balance_finish_kernel(const RouterArgs a, const BalanceArgs o, void* ws, int parts) {
  __shared__ float ps[16][64];
  __shared__ int cs[16][64];
  __shared__ int s_tv;
  __shared__ float s_z;
  const BalanceParts b = balance_parts(ws, a.E);
  const int lane = threadIdx.x & 63, rc = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  float p = 0.0f;
  int c = 0;
  {
    const int at = min(e, a.E - 1);
#pragma unroll 8
    for (int i = rc; i < parts; i += 16) {
      p += b.psum[(int64_t)i * a.E + at];
      c += b.counts[(int64_t)i * a.E + at];
    }
  }
  ps[rc][lane] = p;
  cs[rc][lane] = c;
  if (rc == 0) {
    int n = 0;
    float q = 0.0f;
    for (int i = lane; i < parts; i += 64) { n += b.tv[i]; q += b.z[i]; }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) n += __shfl_xor(n, d, WAVE);
    q = wave_sum(q);
    if (lane == 0) { s_tv = n; s_z = q; }
  }
  __syncthreads();
  if (rc != 0) return;
  for (int i = 1; i < 16; ++i) { p += ps[i][lane]; c += cs[i][lane]; }
  const int tv = s_tv;
  const float mean = tv > 0 ? p / (float)tv : 0.0f;
  float part = 0.0f;
  if (e < a.E) {
    o.counts[e] = c;
    o.mean_prob[e] = mean;
    part = (float)c * mean;
  }
  part = wave_sum(part);
  float total = part;
  if (gridDim.x > 1) {
    int ticket = 0;
    if (lane == 0) {
      __hip_atomic_store(&b.loss[blockIdx.x], part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      ticket = __hip_atomic_fetch_add(b.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(ticket) != (int)gridDim.x - 1) return;
    // at most MOE_ROUTER_MAX_EXPERTS / 64 parts: one per lane, in one round trip
    total = wave_sum(lane < (int)gridDim.x ? __hip_atomic_load(&b.loss[lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0f);
  }
  if (lane != 0) return;
  o.num_valid[0] = tv;
  o.loss[0] = tv > 0 ? o.coef * total * ((float)a.E / ((float)a.K * (float)tv)) : 0.0f;
  o.loss[1] = tv > 0 && o.z_coef != 0.0f ? o.z_coef * s_z / (float)tv : 0.0f;   // s_z may be infinite
}

// d_logits of one row per wave.  With t_k the gradient that reaches the chosen expert k through
// its weight (times ds/dl), a_i = d_loss[0] coef c_i E / (K Tv^2):
//   softmax: dl_i = t_i - p_i sum t + p_i (a_i - sum a p);  sigmoid: t_i + p_i s(-l_i) (a_i - sum a p)
// plus d_loss[1] z_coef 2 lse / Tv softmax(l)_i.  t is spread over the row through LDS; an expert
// that the ids name twice gets the sum.
template <class LT, int VEC, int NREG>
__global__ __launch_bounds__(256) void router_backward_kernel(const RouterArgs a, const BalanceArgs o,
                                                              const float* __restrict__ dw,
                                                              const float* __restrict__ dloss,
                                                              LT* __restrict__ dlogits) {
  extern __shared__ __attribute__((aligned(16))) float spread[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  float* const f = spread;                                    // [E] a_i
  float* const t_row = spread + (1 + wave) * a.E;             // [E] of this wave
  for (int e = lane; e < a.E; e += 64) t_row[e] = 0.0f;
  const int64_t step = (int64_t)gridDim.x * waves;
  int64_t t = (int64_t)blockIdx.x * waves + wave;
  Row<LT, VEC, NREG> ahead;
  if (t < a.T) ahead.load(static_cast<const LT*>(a.logits) + t * a.E, a.E, lane);
  const int tv = o.counts ? *o.num_valid : 0;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  const float db = o.counts && tv > 0 ? (dloss ? dloss[0] : 1.0f) * o.coef : 0.0f;
  const float dz = o.counts && tv > 0 ? (dloss ? dloss[1] : 1.0f) * o.z_coef * 2.0f / (float)tv : 0.0f;
  {
    const float k = tv > 0 ? db * (float)a.E / ((float)a.K * (float)tv * (float)tv) : 0.0f;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) f[e] = o.counts ? k * (float)o.counts[e] : 0.0f;
  }
  __syncthreads();
  // this lane's a_i of chunk c
  const auto balance = [&](int c, float (&v)[VEC]) { load_row<VEC>(f + min((c * 64 + lane) * VEC, a.E - VEC), v); };
  for (; t < a.T; t += step) {
    const LT* const row = static_cast<const LT*>(a.logits) + t * a.E;
    LT* const out = dlogits + t * a.E;
    // the chosen experts' ids, gradients and logits are asked for before anything waits
    int id = -1;
    float g = 0.0f, one[1] = {-INFINITY};
    if (dw && lane < a.K) {
      id = a.ids[t * a.K + lane];
      g = a.scale * dw[t * a.K + lane];
    }
    if ((unsigned)id >= (unsigned)a.E) id = -1;
    if (id >= 0) load_row<1>(row + id, one);
    float l[NREG];
    ahead.values(a.E, lane, l);
    if (t + step < a.T) ahead.load(row + step * a.E, a.E, lane);
    float m = -INFINITY;
    if (!a.valid || a.valid[t]) {
#pragma unroll
      for (int i = 0; i < NREG; ++i) m = __builtin_fmaxf(m, l[i]);
      m = wave_max(m);
    }
    if (!(m > -INFINITY)) {                                   // a row that chose nothing
#pragma unroll
      for (int i = 0; i < NREG; ++i) l[i] = 0.0f;
    } else {
      // softmax: ex = exp(l - m); sigmoid: ex = the sigmoid times e^-top, l stays
      const float top = __builtin_fminf(m, 0.0f);
      float ex[NREG];
      float z = 1.0f, inv_z = 1.0f;
      if (softmax) {
        if (o.counts || !a.renorm) {
          z = 0.0f;
#pragma unroll
          for (int i = 0; i < NREG; ++i) { ex[i] = exp_f(l[i] - m); z += ex[i]; }
          z = wave_sum(z);
          inv_z = 1.0f / z;
        } else {
#pragma unroll
          for (int i = 0; i < NREG; ++i) ex[i] = 0.0f;
        }
      } else if (dz != 0.0f) {
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < NREG; ++i) z += exp_f(l[i] - m);
        z = wave_sum(z);
        inv_z = 1.0f / z;
      }
      // the chosen experts' part
      float tsum = 0.0f;
      if (dw) {
        const float lk = sane(one[0]);
        if (id < 0) g = 0.0f;
        const float v = id < 0 ? 0.0f : softmax ? exp_f(lk - m) * inv_z : fast_sigmoid(lk);
        float tk;
        if (a.renorm) {
          const float top = __builtin_fminf(wave_max(lk), softmax ? m : 0.0f);
          const bool on = lk > -INFINITY;
          const float e = !on ? 0.0f : softmax ? exp_f(lk - top) : sigmoid_over(lk, top);
          const float total = wave_sum(e);
          const float w = on ? e / total : 0.0f;
          const float mean = wave_sum(w * g);
          tk = w * (g - mean);                                // softmax: sums to 0 over the chosen
        } else {
          tk = v * g;
          tsum = softmax ? wave_sum(tk) : 0.0f;
        }
        if (!softmax) tk *= fast_sigmoid(-lk);                // 1 - v would cancel
        if (id >= 0) atomicAdd(&t_row[id], tk);
        wave_sync();
      }
      const float lse = m + LN2 * __builtin_amdgcn_logf(z);
      const float kz = dz != 0.0f ? dz * lse * inv_z : 0.0f;
      if (softmax) {
        float mean = 0.0f;
        if (o.counts) {
#pragma unroll
          for (int c = 0; c < NREG / VEC; ++c) {
            float v[VEC];
            balance(c, v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) mean += v[j] * ex[c * VEC + j];
          }
          mean = wave_sum(mean) * inv_z;
        }
        const float base = mean + tsum;
#pragma unroll
        for (int c = 0; c < NREG / VEC; ++c) {
          float v[VEC];
          balance(c, v);
#pragma unroll
          for (int j = 0; j < VEC; ++j) l[c * VEC + j] = ex[c * VEC + j] * (inv_z * (v[j] - base) + kz);
        }
      } else {
        float s = 1.0f, mean = 0.0f;
        if (o.counts) {
          s = 0.0f;
#pragma unroll
          for (int c = 0; c < NREG / VEC; ++c) {
            float v[VEC];
            balance(c, v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              const int i = c * VEC + j;
              ex[i] = sigmoid_over(l[i], top);
              s += ex[i];
              mean += v[j] * ex[i];
            }
          }
          s = wave_sum(s);
          mean = wave_sum(mean);
        }
        const float inv_s = 1.0f / s;                         // at least half of one term
        mean *= inv_s;
#pragma unroll
        for (int c = 0; c < NREG / VEC; ++c) {
          float v[VEC];
          balance(c, v);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int i = c * VEC + j;
            float d = 0.0f;
            if (o.counts) d = ex[i] * fast_sigmoid(-l[i]) * (v[j] - mean) * inv_s;
            if (kz != 0.0f) d += kz * exp_f(l[i] - m);
            l[i] = d;
          }
        }
      }
      if (dw) {
#pragma unroll
        for (int c = 0; c < NREG / VEC; ++c) {
          float v[VEC];
          load_row<VEC>(t_row + min((c * 64 + lane) * VEC, a.E - VEC), v);
#pragma unroll
          for (int j = 0; j < VEC; ++j) l[c * VEC + j] += v[j];
        }
      }
      if (dw) {
        wave_sync();
        if (id >= 0) t_row[id] = 0.0f;
        wave_sync();
      }
    }
#pragma unroll
    for (int c = 0; c < NREG / VEC; ++c) {
      const int col = (c * 64 + lane) * VEC;
      if (col < a.E) {
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = l[c * VEC + j];
        store_row<VEC>(out + col, v);
      }
    }
  }
}

// 8 consecutive logits per lane (16-byte accesses) for rows that allow it and fill most lanes;
// one per lane otherwise (rows of up to 256 experts leave too few lanes a maximum to bound the
// choice with, and are short anyway).
bool wide_rows(int E, const void* p, const void* q) {
  return E > 256 && E % 8 == 0 && !(((uintptr_t)p | (uintptr_t)q) & 15);
}

template <class LT, int VEC, int NREG, bool BIAS, bool BAL>
int forward_rows(const RouterArgs& a, void* ws, hipStream_t s) {
  constexpr int waves = router_waves<NREG, BIAS, BAL>();
  const size_t lds = waves * CAND * sizeof(uint2) + (BAL ? waves * 8 + (size_t)(3 + HAND) * a.E * 4 + 256 : 0);
  if constexpr (BAL) {
    const int64_t groups = ((int64_t)a.T + waves - 1) / waves;
    const int grid = (int)(groups < 1 ? 1 : groups < MOE_ROUTER_PARTS ? groups : MOE_ROUTER_PARTS);
    router_kernel<LT, VEC, NREG, BIAS, BAL><<<(unsigned)grid, waves * 64, lds, s>>>(a, ws);
    return grid;
  } else {
    RouterArgs part = a;
    constexpr int64_t slice = MAX_ITEMS / 64;                 // a wave per row; keeps the alignment of the rows
    for (int64_t t = 0; t < a.T; t += slice) {
      part.T = (int)(a.T - t < slice ? a.T - t : slice);
      part.logits = static_cast<const LT*>(a.logits) + t * a.E;
      part.valid = a.valid ? a.valid + t : nullptr;
      part.ids = a.ids + t * a.K;
      part.w = a.w + t * a.K;
      router_kernel<LT, VEC, NREG, BIAS, BAL><<<(unsigned)((part.T + waves - 1) / waves), waves * 64, lds, s>>>(part, ws);
    }
    return 0;
  }
}
// Returns the number of partial sums of the balance statistics.
template <class LT, int VEC, int NREG>
int forward_rows(const RouterArgs& a, bool bal, void* ws, hipStream_t s) {
  if (bal) return a.bias ? forward_rows<LT, VEC, NREG, true, true>(a, ws, s) : forward_rows<LT, VEC, NREG, false, true>(a, ws, s);
  return a.bias ? forward_rows<LT, VEC, NREG, true, false>(a, ws, s) : forward_rows<LT, VEC, NREG, false, false>(a, ws, s);
}

template <class LT>
int forward(const RouterArgs& a, bool bal, void* ws, hipStream_t s) {
  if (wide_rows(a.E, a.logits, a.bias)) {
    if (a.E <= 512) return forward_rows<LT, 8, 8>(a, bal, ws, s);
    else if (a.E <= 1024) return forward_rows<LT, 8, 16>(a, bal, ws, s);
    else return forward_rows<LT, 8, 32>(a, bal, ws, s);
  } else {
    if (a.E <= 256) return forward_rows<LT, 1, 4>(a, bal, ws, s);
    else if (a.E <= 1024) return forward_rows<LT, 1, 16>(a, bal, ws, s);
    else return forward_rows<LT, 1, 32>(a, bal, ws, s);
  }
}

template <class LT>
void backward(const RouterArgs& a, const BalanceArgs& o, const float* dw, const float* dloss, void* dlogits, hipStream_t s) {
  const unsigned groups = (unsigned)(((int64_t)a.T + 3) / 4);
  const unsigned grid = groups < 1024u ? groups : 1024u;
  const size_t lds = (size_t)5 * a.E * 4;
  LT* const d = static_cast<LT*>(dlogits);
  if (wide_rows(a.E, a.logits, dlogits)) {
    if (a.E <= 512) router_backward_kernel<LT, 8, 8><<<grid, 256, lds, s>>>(a, o, dw, dloss, d);
    else if (a.E <= 1024) router_backward_kernel<LT, 8, 16><<<grid, 256, lds, s>>>(a, o, dw, dloss, d);
    else router_backward_kernel<LT, 8, 32><<<grid, 256, lds, s>>>(a, o, dw, dloss, d);
  } else {
    if (a.E <= 256) router_backward_kernel<LT, 1, 4><<<grid, 256, lds, s>>>(a, o, dw, dloss, d);
    else if (a.E <= 1024) router_backward_kernel<LT, 1, 16><<<grid, 256, lds, s>>>(a, o, dw, dloss, d);
    else router_backward_kernel<LT, 1, 32><<<grid, 256, lds, s>>>(a, o, dw, dloss, d);
  }
}

}  // namespace

hipError_t launch_router(const RouterArgs& a, const BalanceArgs* b, void* ws, hipStream_t s) {
  const int parts = a.dt == MOE_DT_F32 ? forward<float>(a, b != nullptr, ws, s) : forward<uint16_t>(a, b != nullptr, ws, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !b) return e;
  balance_finish_kernel<<<(unsigned)((a.E + 63) / 64), 1024, 0, s>>>(a, *b, ws, parts);
  return hipGetLastError();
}

hipError_t launch_router_backward(const RouterArgs& a, const BalanceArgs* b, const float* dw, const float* dloss,
                                  void* dlogits, hipStream_t s) {
  BalanceArgs none = {};
  if (a.dt == MOE_DT_F32) backward<float>(a, b ? *b : none, dw, dloss, dlogits, s);
  else backward<uint16_t>(a, b ? *b : none, dw, dloss, dlogits, s);
  return hipGetLastError();
}

}  // namespace moe
