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
#include "moe_router_choice.h"

namespace moe {

namespace {

constexpr int HAND = 4;                       // rows of LDS in which waves hand over their sums
constexpr int TURNS = 64;                     // rows that a wave adds up in fp32

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
