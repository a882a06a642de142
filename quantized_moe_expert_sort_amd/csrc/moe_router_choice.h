// The choice of a token's experts, shared by the router (moe_router.hip) and the routed layer of a few
// tokens (moe_few.hip): one wave takes a row of logits.
#pragma once

#include <type_traits>

#include "moe_kernels.h"
#include "moe_rows.h"

namespace moe {

namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float BIG = 3.402823466e38f;
constexpr int CAND = 64;                      // candidates of a row, at most one per lane

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

}  // namespace

}  // namespace moe
