// Losses over token log-probabilities grouped into sequences: the preference
// loss over paired sequences and the clipped policy loss with a KL term, each
// with its gradient in the token log-probabilities.
//
// Both are bound by memory (a handful of operations per token and array), and
// by launch latency below a few hundred thousand tokens.  Both have two phases:
// the first sums what the second has to divide by or compare with (a
// sequence's log ratio, the mask), the second reads the tokens, writes the
// gradient and reduces the scalars.  The gradient thus comes with the loss,
// in one reading of everything but the mask.  A policy loss that is averaged
// per sequence, with a team for each whole sequence, needs no first phase: the
// team sums its sequence's mask and finds it in L1 when it reads it again.
//
// Up to kOneLaunchTokens tokens, when all items find a team at once, the phases
// are one cooperative launch (which CUDA starts only when all of its blocks are
// resident) with a grid barrier between them, else two launches (the second waits
// for the first's end only where it needs the sums).
// One launch saves the host 2.5 us, and costs the GPU 3 us with 256 blocks:
// calls back to back take 20.3 against 22.6 us (preference, 190 thousand
// tokens), 21.7 against 24.2 (policy, half a million), 41.3 against 34.8
// (preference, 7.7 million).
//
// Work is cut into items: a sequence, or one of `splits` ranges of it when the
// sequences are few and long.  A team (a warp for short sequences, a block
// otherwise) walks an item's tokens four at a time on 16-byte boundaries of
// the arrays, so a sequence may begin and end anywhere.  Sums are kept in
// 64 bits and joined in a fixed order: no result depends on the order in
// which blocks run.
#pragma once

#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "kd_launch.cuh"

namespace kd {
namespace seq {

constexpr int kThreads = 256;
constexpr int kSumBlocks = 1184;     // blocks of the first launch at most (8 per SM): partial totals to join
constexpr int kLossBlocks = 4736;    // blocks of the second launch at most (32 per SM, several of them in turn)
constexpr int kResident = 4;         // blocks of the loss phase that an SM holds (64 registers a thread)
constexpr int kSumUnroll = 2;        // groups of four tokens whose loads a thread of the first launch has in flight
constexpr int64_t kOneLaunchTokens = int64_t(1) << 20;
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - (int64_t(1) << 16);   // token indices fit an int, a stride past the end too

// The sequences of an array of N tokens: sequence s is [offsets[s],
// offsets[s + 1]), or row s of S rows of L tokens when offsets is null.
// Offsets are clamped to [0, N], so that no value of theirs leads outside
// the arrays.
struct Sequences {
  const void* offsets;
  int offsets_i64;
  int64_t S, N, L;
  int splits;          // items per sequence
};

__device__ __forceinline__ int seq_offset(const Sequences& q, int64_t s) {
  if (!q.offsets) return (int)(s * q.L);
  int64_t o = q.offsets_i64 ? static_cast<const int64_t*>(q.offsets)[s]
                            : (int64_t)static_cast<const int32_t*>(q.offsets)[s];
  return (int)(o < 0 ? 0 : (o > q.N ? q.N : o));
}

// Tokens [lo, hi) of item k of sequence s.
__device__ __forceinline__ void item_range(const Sequences& q, int64_t s, int k, int& lo, int& hi) {
  const int b = seq_offset(q, s), e = seq_offset(q, s + 1);
  lo = b;
  hi = e;
  if (q.splits > 1) {
    const int a = b & ~3;
    const int per = e > b ? ((e - a + q.splits - 1) / q.splits + 3) & ~3 : 0;
    const int64_t start = a + (int64_t)k * per;        // past hi for the last ranges of a short sequence
    if (start > lo) lo = start < hi ? (int)start : hi;
    if (start + per < hi) hi = (int)(start + per);
  }
  if (hi < lo) hi = lo;
}

// Four tokens of an array from t0 (a multiple of 4): those of [lo, hi), zeros
// for the others.  ONCE: not read again, so not worth keeping in L2 (the mask is).
template <bool VEC, bool ONCE = true>
__device__ __forceinline__ void load4(const float* __restrict__ p, int t0, int lo, int hi, float (&v)[4]) {
  if (VEC && t0 >= lo && t0 + 4 <= hi) {
    const float4* q = reinterpret_cast<const float4*>(p + t0);
    const float4 f = ONCE ? __ldcs(q) : *q;
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (t0 + j >= lo && t0 + j < hi) ? p[t0 + j] : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store4(float* __restrict__ p, int t0, int lo, int hi, const float (&v)[4]) {
  if (VEC && t0 >= lo && t0 + 4 <= hi) {
    __stcs(reinterpret_cast<float4*>(p + t0), make_float4(v[0], v[1], v[2], v[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t0 + j >= lo && t0 + j < hi) p[t0 + j] = v[j];
  }
}

// The four tokens' weights: the mask, or one, inside [lo, hi); 0 outside.
template <bool VEC>
__device__ __forceinline__ void load_mask4(const float* __restrict__ mask, int t0, int lo, int hi,
                                           float (&m)[4]) {
  if (mask) {
    load4<VEC, false>(mask, t0, lo, hi, m);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = (t0 + j >= lo && t0 + j < hi) ? 1.f : 0.f;
  }
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over a team, the same on every thread of it.  `red`: kThreads / 32
// doubles of shared memory, free again when the call returns.
template <int TEAM>
__device__ __forceinline__ double team_sum(double v, double* red) {
  v = warp_sum64(v);
  if constexpr (TEAM > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < TEAM / 32; ++w) v += red[w];
    __syncthreads();
  }
  return v;
}

// Calls body(team, item, lo, hi, thread in the team) for the block's items; every
// thread of a team calls together.  Among short sequences one that is long is
// left to the whole block: a warp would still be at it when all others are done
// (32,768 tokens among 2,000 sequences of 150: policy loss 92 us, by warps alone
// 480; 200,000 sequences of 100 tokens pay 3% for the question).
constexpr int kWarpItemTokens = 2048;

template <int T>
struct Team {
  static constexpr int threads = T;
};

template <int TEAM, class Body>
__device__ __forceinline__ void for_items(const Sequences& q, Body&& body) {
  const int64_t items = q.S * q.splits;
  auto range = [&](int64_t it, int& lo, int& hi) {
    const int64_t s = it / q.splits;
    item_range(q, s, (int)(it - s * q.splits), lo, hi);
  };
  if constexpr (TEAM == kThreads) {
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
      int lo, hi;
      range(it, lo, hi);
      body(Team<kThreads>{}, it, lo, hi, (int)threadIdx.x);
    }
  } else {
    constexpr int kTeams = kThreads / TEAM;
    const int64_t first = (int64_t)blockIdx.x * kTeams, step = (int64_t)gridDim.x * kTeams;
    bool left = false;
    for (int64_t it = first + threadIdx.x / TEAM; it < items; it += step) {
      int lo, hi;
      range(it, lo, hi);
      if (hi - lo <= kWarpItemTokens) body(Team<TEAM>{}, it, lo, hi, (int)(threadIdx.x % TEAM));
      else left = true;
    }
    if (__syncthreads_or(left))               // after the short ones: no warp waits for another on the way
      for (int64_t base = first; base < items; base += step)
        for (int64_t it = base; it < base + kTeams && it < items; ++it) {
          int lo, hi;
          range(it, lo, hi);
          if (hi - lo > kWarpItemTokens) body(Team<kThreads>{}, it, lo, hi, (int)threadIdx.x);
        }
  }
}

// Sum of n values, by the lanes of one warp in a fixed order.
__device__ __forceinline__ double warp_sum_array(const double* p, int64_t n, int stride) {
  double v = 0.0;
  for (int64_t i = threadIdx.x & 31; i < n; i += 32) v += p[i * stride];
  return warp_sum64(v);
}

// The last block of a launch to get here (by `counter`, zeroed beforehand)
// sums the blocks' partials in block order; every thread of it gets true.
__device__ __forceinline__ bool last_block(unsigned int* counter) {
  __shared__ bool last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(counter, 1u) == gridDim.x - 1;
  __syncthreads();
  if (last) __threadfence();
  return last;
}

// Tokens in no sequence (before the first, behind the last) have no gradient.
__device__ __forceinline__ void zero_outside(const Sequences& q, float* __restrict__ out) {
  if (!q.offsets) return;
  const int b = seq_offset(q, 0), e = seq_offset(q, q.S);
  const int64_t step = (int64_t)gridDim.x * blockDim.x, i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t t = i0; t < b; t += step) out[t] = 0.f;
  for (int64_t t = e + i0; t < q.N; t += step) out[t] = 0.f;
}

// ---------------------------------------------------------------- preference loss
//
// Sequences s and P + s (P = S / 2) are pair s's chosen and rejected answer.
// With r_s = sum_t m_t (logp_t - ref_t), divided by sum_t m_t when averaged
// (0 for a sequence without tokens),
//   D = beta (r_s - r_{P+s}) - margin
//   sigmoid: -(1 - e) log sigma(D) - e log sigma(-D)
//   hinge:   max(0, 1 - D)
//   ipo:     (r_s - r_{P+s} - margin - 1 / (2 beta))^2
// the loss is the mean over the pairs and
//   dlogp_t = +- g (dl/dD) (dD/dr) m_t / P  [/ sum m].
// The difference of policy and reference is taken per token, so that the sum
// holds the small log ratio and not two large log-probabilities.

enum { kSigmoid = 0, kHinge = 1, kIpo = 2 };

struct PrefArgs {
  Sequences q;
  const float *logp, *ref, *mask, *grad_loss;
  double beta, smoothing, margin;
  int kind, average;
  double* sums;            // [S * splits][2]: sum m (logp - ref), sum m
  double* part;            // [blocks] pair losses
  unsigned int* counter;
  float *loss, *chosen, *rejected, *dlogp;
};

template <int TEAM, bool VEC>
__device__ __forceinline__ void pref_sums(const PrefArgs& A, double* red) {
  for_items<TEAM>(A.q, [&](auto team, int64_t it, int lo, int hi, int tid) {
    constexpr int T = decltype(team)::threads;
    double r = 0.0, n = 0.0;
    for (int t0 = ((lo >> 2) + tid) << 2; t0 < hi; t0 += 4 * T * kSumUnroll) {
      float m[kSumUnroll][4], lp[kSumUnroll][4], rf[kSumUnroll][4];
#pragma unroll
      for (int u = 0; u < kSumUnroll; ++u) {
        const int t = t0 + 4 * T * u;
        load_mask4<VEC>(A.mask, t, lo, hi, m[u]);
        load4<VEC>(A.logp, t, lo, hi, lp[u]);
        if (A.ref) load4<VEC>(A.ref, t, lo, hi, rf[u]);
      }
#pragma unroll
      for (int u = 0; u < kSumUnroll; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (m[u][j] != 0.f) {               // a masked place may hold anything, NaN included
            r += (double)m[u][j] * ((double)lp[u][j] - (A.ref ? (double)rf[u][j] : 0.0));
            n += (double)m[u][j];
          }
    }
    r = team_sum<T>(r, red);
    n = team_sum<T>(n, red);
    if (tid == 0) {
      A.sums[2 * it] = r;
      A.sums[2 * it + 1] = n;
    }
  });
}

// Sequence s's log ratio and the factor of its tokens' weights (a whole warp calls).
__device__ __forceinline__ void seq_ratio(const PrefArgs& A, int64_t s, double& r, double& w) {
  const double* p = A.sums + 2 * s * A.q.splits;
  r = warp_sum_array(p, A.q.splits, 2);
  w = 1.0;
  if (A.average) {
    const double n = warp_sum_array(p + 1, A.q.splits, 2);
    w = n != 0.0 ? 1.0 / n : 0.0;
  }
  r *= w;
}

// w v, and 0 for w = 0 whatever v (a pair so far apart that v is infinite).
__device__ __forceinline__ double share(double w, double v) { return w != 0.0 ? w * v : 0.0; }

__device__ __forceinline__ double softplus64(double v) { return (v > 0.0 ? v : 0.0) + log1p(exp(-fabs(v))); }

// The second phase, up to the block's partial loss.
template <int TEAM, bool VEC>
__device__ __forceinline__ void pref_losses(const PrefArgs& A, double* red) {
  __shared__ float s_coef;
  const int64_t P = A.q.S / 2;
  const double g = A.grad_loss ? (double)*A.grad_loss : 1.0;
  double mine = 0.0;                          // pair losses of this thread's teams
  for_items<TEAM>(A.q, [&](auto team, int64_t it, int lo, int hi, int tid) {
    constexpr int T = decltype(team)::threads;
    const int64_t s = it / A.q.splits;
    const int k = (int)(it - s * A.q.splits);
    float m[kSumUnroll][4];                   // the first groups' masks arrive while the coefficient is worked out
    if (A.dlogp)
#pragma unroll
      for (int u = 0; u < kSumUnroll; ++u)
        load_mask4<VEC>(A.mask, (((lo >> 2) + tid) << 2) + 4 * T * u, lo, hi, m[u]);
    float coef = 0.f;
    wait_previous();                          // for the sums
    if (tid < 32) {
      const bool is_chosen = s < P;
      double r, w, ro, wo;
      seq_ratio(A, s, r, w);
      seq_ratio(A, is_chosen ? s + P : s - P, ro, wo);
      const double diff = is_chosen ? r - ro : ro - r;
      const double D = A.beta * diff - A.margin;
      double slope;                           // the pair loss's derivative in r_chosen
      const double e = diff - A.margin - 0.5 / A.beta;
      if (A.kind == kSigmoid) slope = A.beta * (1.0 / (1.0 + exp(-D)) - (1.0 - A.smoothing));
      else if (A.kind == kHinge) slope = D < 1.0 ? -A.beta : (D >= 1.0 ? 0.0 : D);       // NaN stays NaN
      else slope = 2.0 * e;
      coef = (float)((is_chosen ? slope : -slope) * w * g / (double)P);
      if (tid == 0 && k == 0) {
        if (is_chosen) {
          if (A.kind == kSigmoid) mine += share(1.0 - A.smoothing, softplus64(-D)) + share(A.smoothing, softplus64(D));
          else if (A.kind == kHinge) mine += D < 1.0 ? 1.0 - D : (D >= 1.0 ? 0.0 : D);
          else mine += e * e;
          A.chosen[s] = (float)(A.beta * r);
        } else {
          A.rejected[s - P] = (float)(A.beta * r);
        }
      }
    }
    if (!A.dlogp) return;
    if constexpr (T > 32) {
      if (threadIdx.x == 0) s_coef = coef;
      __syncthreads();
      coef = s_coef;
      __syncthreads();
    }
    for (int t0 = ((lo >> 2) + tid) << 2; t0 < hi; t0 += 4 * T * kSumUnroll) {
      float d[kSumUnroll][4];
#pragma unroll
      for (int u = 0; u < kSumUnroll; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[u][j] = m[u][j] != 0.f ? coef * m[u][j] : 0.f;
#pragma unroll
      for (int u = 0; u < kSumUnroll; ++u)
        load_mask4<VEC>(A.mask, t0 + 4 * T * (u + kSumUnroll), lo, hi, m[u]);
#pragma unroll
      for (int u = 0; u < kSumUnroll; ++u) {
        const int t = t0 + 4 * T * u;
        if (t < hi) store4<VEC>(A.dlogp, t, lo, hi, d[u]);
      }
    }
  });
  wait_previous();                            // a block without an item, too: the counter is the first launch's
  if (A.dlogp) zero_outside(A.q, A.dlogp);
  mine = team_sum<kThreads>(mine, red);
  if (threadIdx.x == 0) A.part[blockIdx.x] = mine;
}

// The blocks' partial losses, joined in block order by one block.
__device__ __forceinline__ void pref_join(const PrefArgs& A, double* red) {
  const int64_t P = A.q.S / 2;
  double v = 0.0;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kThreads) v += __ldcg(A.part + i);
  v = team_sum<kThreads>(v, red);
  if (threadIdx.x == 0) *A.loss = P > 0 ? (float)(v / (double)P) : 0.f;
}

template <int TEAM, bool VEC>
__global__ void __launch_bounds__(kThreads, kResident) pref_sums_kernel(const PrefArgs A) {
  __shared__ double red[kThreads / 32];
  next_may_start();
  if (blockIdx.x == 0 && threadIdx.x == 0) *A.counter = 0u;
  pref_sums<TEAM, VEC>(A, red);
}

template <int TEAM, bool VEC>
__global__ void __launch_bounds__(kThreads, kResident) pref_loss_kernel(const PrefArgs A) {
  __shared__ double red[kThreads / 32];
  pref_losses<TEAM, VEC>(A, red);
  if (last_block(A.counter)) pref_join(A, red);
}

template <int TEAM, bool VEC>
__global__ void __launch_bounds__(kThreads, kResident) pref_one_kernel(const PrefArgs A) {
  __shared__ double red[kThreads / 32];
  pref_sums<TEAM, VEC>(A, red);
  cooperative_groups::this_grid().sync();
  pref_losses<TEAM, VEC>(A, red);
  cooperative_groups::this_grid().sync();
  if (blockIdx.x == 0) pref_join(A, red);
}

// ---------------------------------------------------------------- policy loss
//
// Per token, with x = logp - old, r = e^x and advantage A (the token's or its
// sequence's):
//   obj = min(r A, clip(r, 1 - lo, 1 + hi) A), and for A < 0 at least c A
//         when a dual clip c is given
//   kl  = y, y^2 / 2 or e^-y - 1 + y       (k1, k2, k3; y = logp - ref)
//   l   = -obj + kl_coef kl
// summed with weights w_t: m_t / sum m over all sequences, or m_t / (S sum of
// the sequence's m), 0 where that sum is 0.  The gradient
//   dlogp = g w ( [not clipped] (-A r) + kl_coef (1 | y | 1 - e^-y) )
// treats old, ref and A as constants.
//
// Whether a token is clipped is decided on the exact difference x, against
// log(1 + hi), log(1 - lo) and log c, and not on a rounded exponential.  In one
// launch, where the time is the host's, a token's terms are computed in 64 bits.
// In two, e^x and the KL term are taken in 32 (so that r or e^-y is infinite
// above 3.4e38); e^-y - 1 + y, which cancels for small y, by its series for
// |y| < 1/2.  There tokens are computed without branches, masked ones on zeros:
// four at a time in flight instead of one behind the other.  Sums are 64-bit in
// both: adding four tokens in 32 bits first would take 70.1 us instead of 71.8
// for 22 million padded tokens, and lose what terms that cancel leave.

enum { kK1 = 0, kK2 = 1, kK3 = 2, kNoKl = 3 };

struct PolicyArgs {
  Sequences q;
  const float *logp, *old, *ref, *adv, *mask, *grad_loss;
  int adv_per_seq, per_sequence;
  float hi_h, hi_l, lo_h, lo_l, dual_h, dual_l;     // log borders in two floats each (no dual clip: infinity)
  float hi1, lo1, dual_c, kl_coef;                  // 1 + hi, 1 - lo, c
  double log_hi, log_lo, log_dual, hi1_64, lo1_64, dual_64, kl_coef_64;      // the same
  double* sums;            // [S * splits] sum m; null: each team sums its own (whole) sequences' masks
  double* total;           // [kSumBlocks] the first launch's blocks' sums
  double* part;            // [blocks][3]
  unsigned int* counter;
  float *loss, *dlogp;     // loss[3]: loss, KL, clipped share
};

// A thread's share of the sum of the mask over [lo, hi).
template <int TEAM, bool VEC>
__device__ __forceinline__ double mask_sum(const float* __restrict__ mask, int lo, int hi, int tid) {
  double n = 0.0;
  for (int t0 = ((lo >> 2) + tid) << 2; t0 < hi; t0 += 4 * TEAM * kSumUnroll) {
    float m[kSumUnroll][4];
#pragma unroll
    for (int u = 0; u < kSumUnroll; ++u) load4<VEC, false>(mask, t0 + 4 * TEAM * u, lo, hi, m[u]);
#pragma unroll
    for (int u = 0; u < kSumUnroll; ++u)
      n += ((double)m[u][0] + (double)m[u][1]) + ((double)m[u][2] + (double)m[u][3]);
  }
  return n;
}

template <int TEAM, bool VEC>
__device__ __forceinline__ void policy_sums(const PolicyArgs& A, double* red) {
  double all = 0.0;
  for_items<TEAM>(A.q, [&](auto team, int64_t it, int lo, int hi, int tid) {
    constexpr int T = decltype(team)::threads;
    const double n = A.mask ? team_sum<T>(mask_sum<T, VEC>(A.mask, lo, hi, tid), red) : (double)(hi - lo);
    if (tid == 0) {
      A.sums[it] = n;
      all += n;
    }
  });
  all = team_sum<kThreads>(all, red);
  if (threadIdx.x == 0) A.total[blockIdx.x] = all;
}

// (e^x - 1 - x) / x^2 for |x| < 1/2: sum_k x^k / (k + 2)!, k = 0..8 (the next term is below 2^-31 of it).
__device__ __forceinline__ float exp_tail_series(float x) {
  float p = 1.f / 3628800.f;
  p = fmaf(p, x, 1.f / 362880.f);
  p = fmaf(p, x, 1.f / 40320.f);
  p = fmaf(p, x, 1.f / 5040.f);
  p = fmaf(p, x, 1.f / 720.f);
  p = fmaf(p, x, 1.f / 120.f);
  p = fmaf(p, x, 1.f / 24.f);
  p = fmaf(p, x, 1.f / 6.f);
  return fmaf(p, x, 0.5f);
}

// What the rounding of x = lp - old left out, exactly.
__device__ __forceinline__ float difference_rest(float lp, float old, float x) {
  const float b = __fsub_rn(x, lp);
  return __fsub_rn(__fsub_rn(lp, __fsub_rn(x, b)), __fadd_rn(old, b));
}

// One token: its loss, KL estimate, whether it is clipped, and d loss / d logp.
template <int KL>
__device__ __forceinline__ void policy_token(const PolicyArgs& A, float lp, float old, float ref, float a, float& loss,
                                             float& kl, float& clipped, float& d) {
  const float x = __fsub_rn(lp, old);
  // A rounded x above (below) the border's nearest float is an exact one above (below) the border; where they are
  // equal, the rests decide.
  bool over = x > A.hi_h, under = x < A.lo_h, far = x > A.dual_h;
  if (x == A.hi_h || x == A.lo_h || x == A.dual_h) {
    const float rest = difference_rest(lp, old, x);
    over = over || (x == A.hi_h && rest > A.hi_l);
    under = under || (x == A.lo_h && rest < A.lo_l);
    far = far || (x == A.dual_h && rest > A.dual_l);
  }
  const bool clip = a > 0.f ? over : (a < 0.f && (under || far));
  const float border = a > 0.f ? A.hi1 : (under ? A.lo1 : A.dual_c);
  const float ra = a == 0.f ? 0.f : expf(x) * a;     // A = 0: no term, whatever the ratio
  const float obj = clip ? border * a : ra;
  clipped = clip ? 1.f : 0.f;
  kl = 0.f;
  float dk = 0.f;
  if (KL != kNoKl) {
    const float y = lp - ref;
    if (KL == kK1) {
      kl = y;
      dk = 1.f;
    } else if (KL == kK2) {
      kl = 0.5f * y * y;
      dk = y;
    } else {
      const float e = expf(-y);
      const bool small = fabsf(y) < 0.5f;
      kl = small ? y * y * exp_tail_series(-y) : e - 1.f + y;      // e^-y - 1 + y
      dk = small ? y - kl : 1.f - e;                               // 1 - e^-y
    }
  }
  // kl_coef 0: the KL is reported and has no part in the loss, not even 0 times infinity
  loss = KL != kNoKl && A.kl_coef != 0.f ? fmaf(A.kl_coef, kl, -obj) : -obj;
  d = clip ? 0.f : -ra;
  if (KL != kNoKl && A.kl_coef != 0.f) d = fmaf(A.kl_coef, dk, d);
}

// The same in 64 bits.
template <int KL>
__device__ __forceinline__ void policy_token64(const PolicyArgs& A, float lp, float old, float ref, float a, double& loss,
                                               double& kl, double& clipped, double& d) {
  const double x = (double)lp - (double)old;
  const bool under = x < A.log_lo;
  const bool clip = a > 0.f ? x > A.log_hi : (a < 0.f && (under || x > A.log_dual));
  const double border = a > 0.f ? A.hi1_64 : (under ? A.lo1_64 : A.dual_64);
  const double ra = a == 0.f ? 0.0 : exp(x) * (double)a;
  clipped = clip ? 1.0 : 0.0;
  kl = 0.0;
  double dk = 0.0;
  if (KL != kNoKl) {
    const double y = (double)lp - (double)ref;
    if (KL == kK1) {
      kl = y;
      dk = 1.0;
    } else if (KL == kK2) {
      kl = 0.5 * y * y;
      dk = y;
    } else {
      dk = -expm1(-y);
      kl = y - dk;
    }
  }
  loss = -(clip ? border * (double)a : ra);
  d = clip ? 0.0 : -ra;
  if (KL != kNoKl && A.kl_coef_64 != 0.0) {   // 0: see policy_token
    loss += A.kl_coef_64 * kl;
    d += A.kl_coef_64 * dk;
  }
}

// The blocks' partial scalars, joined in block order by one block.
__device__ __forceinline__ void policy_join(const PolicyArgs& A, int blocks, double* red) {
  double v[3] = {0.0, 0.0, 0.0};
  for (int i = threadIdx.x; i < blocks; i += kThreads)
#pragma unroll
    for (int j = 0; j < 3; ++j) v[j] += __ldcg(A.part + 3 * i + j);
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    v[j] = team_sum<kThreads>(v[j], red);
    if (threadIdx.x == 0) A.loss[j] = (float)v[j];
  }
}

// The second phase, up to the block's partial scalars; sum_blocks: the first phase's blocks.
template <int TEAM, bool VEC, int KL, bool WIDE>
__device__ __forceinline__ void policy_losses(const PolicyArgs& A, int sum_blocks, double* red) {
  const float g = A.grad_loss ? *A.grad_loss : 1.f;
  double inv_total = 0.0;
  if (A.sums) wait_previous();
  if (!A.per_sequence) {
    double t = 0.0;
    for (int i = threadIdx.x; i < sum_blocks; i += kThreads) t += __ldcg(A.total + i);
    t = team_sum<kThreads>(t, red);
    inv_total = t != 0.0 ? 1.0 / t : 0.0;
  }
  double sum_l = 0.0, sum_k = 0.0, sum_c = 0.0;
  for_items<TEAM>(A.q, [&](auto team, int64_t it, int lo, int hi, int tid) {
    constexpr int T = decltype(team)::threads;
    const int64_t s = it / A.q.splits;
    double w = inv_total;
    if (A.per_sequence) {
      double n = 0.0;
      if (A.sums) {
        n = warp_sum_array(A.sums + s * A.q.splits, A.q.splits, 1);             // every warp of the team
      } else if (A.mask) {                    // the mask's second reading, below, finds it in L1
        n = team_sum<T>(mask_sum<T, VEC>(A.mask, lo, hi, tid), red);
      } else {
        n = (double)(hi - lo);
      }
      w = n != 0.0 ? 1.0 / (n * (double)A.q.S) : 0.0;
    }
    const float as = A.adv_per_seq ? A.adv[s] : 0.f;
    float next[4];                            // the next group's mask, loaded a group ahead
    load_mask4<VEC>(A.mask, ((lo >> 2) + tid) << 2, lo, hi, next);
    for (int t0 = ((lo >> 2) + tid) << 2; t0 < hi; t0 += 4 * T) {
      float m[4] = {next[0], next[1], next[2], next[3]}, d[4] = {0.f, 0.f, 0.f, 0.f};
      load_mask4<VEC>(A.mask, t0 + 4 * T, lo, hi, next);
      if (w != 0.0 && (m[0] != 0.f || m[1] != 0.f || m[2] != 0.f || m[3] != 0.f)) {     // padding costs its mask alone
        float lp[4], od[4], rf[4], a[4];
        load4<VEC>(A.logp, t0, lo, hi, lp);
        load4<VEC>(A.old, t0, lo, hi, od);
        if (KL != kNoKl) load4<VEC>(A.ref, t0, lo, hi, rf);
        if (!A.adv_per_seq) load4<VEC>(A.adv, t0, lo, hi, a);
        if constexpr (WIDE) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (m[j] != 0.f) {                // a masked place may hold anything, NaN included
              double l64, k64, c64, d64;
              policy_token64<KL>(A, lp[j], od[j], KL != kNoKl ? rf[j] : 0.f, A.adv_per_seq ? as : a[j], l64, k64, c64, d64);
              const double wm = w * (double)m[j];
              sum_l += wm * l64;
              sum_k += wm * k64;
              sum_c += wm * c64;
              d[j] = (float)((double)g * wm * d64);
            }
        } else {
          const float wg = (float)w * g;
          float l[4], k[4], c[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {         // a masked place may hold anything, NaN included
            const bool on = m[j] != 0.f;
            policy_token<KL>(A, on ? lp[j] : 0.f, on ? od[j] : 0.f, KL != kNoKl && on ? rf[j] : 0.f,
                             on ? (A.adv_per_seq ? as : a[j]) : 0.f, l[j], k[j], c[j], d[j]);
            d[j] = on ? wg * m[j] * d[j] : 0.f;
          }
          // in 64 bits, where the products are exact and terms that cancel leave what is left of them
          double tl = 0.0, tk = 0.0, tc = 0.0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const double wide = (double)m[j];
            tl = fma(wide, (double)l[j], tl);
            if (KL != kNoKl) tk = fma(wide, (double)k[j], tk);
            if (c[j] != 0.f) tc += wide;
          }
          sum_l += w * tl;
          sum_k += w * tk;
          sum_c += w * tc;
        }
      }
      if (A.dlogp) store4<VEC>(A.dlogp, t0, lo, hi, d);
    }
  });
  if (A.dlogp) zero_outside(A.q, A.dlogp);
  sum_l = team_sum<kThreads>(sum_l, red);
  sum_k = team_sum<kThreads>(sum_k, red);
  sum_c = team_sum<kThreads>(sum_c, red);
  if (threadIdx.x == 0) {
    A.part[3 * blockIdx.x] = sum_l;
    A.part[3 * blockIdx.x + 1] = sum_k;
    A.part[3 * blockIdx.x + 2] = sum_c;
  }
}

template <int TEAM, bool VEC>
__global__ void __launch_bounds__(kThreads, 8) policy_sums_kernel(const PolicyArgs A) {
  __shared__ double red[kThreads / 32];
  next_may_start();
  if (blockIdx.x == 0 && threadIdx.x == 0) *A.counter = 0u;
  policy_sums<TEAM, VEC>(A, red);
}

// Five blocks an SM, 48 registers a thread and some spills: 71.8 us against 78.0
// with four, for 22 million padded tokens (6.6 million of them unmasked).  Six take
// 71.3 there, but 53.7 against 51.4 for three million tokens in sequences of 150.
template <int TEAM, bool VEC, int KL>
__global__ void __launch_bounds__(kThreads, 5) policy_loss_kernel(const PolicyArgs A, int sum_blocks) {
  __shared__ double red[kThreads / 32];
  if (!A.sums) next_may_start();              // policy_finish_kernel
  policy_losses<TEAM, VEC, KL, false>(A, sum_blocks, red);
  if (A.sums && last_block(A.counter)) policy_join(A, gridDim.x, red);
}

// One block: the scalars of a launch that had nothing before it to zero the counter.
__global__ void __launch_bounds__(kThreads) policy_finish_kernel(const PolicyArgs A, int blocks) {
  __shared__ double red[kThreads / 32];
  wait_previous();
  policy_join(A, blocks, red);
}

template <int TEAM, bool VEC, int KL>
__global__ void __launch_bounds__(kThreads, kResident) policy_one_kernel(const PolicyArgs A) {
  __shared__ double red[kThreads / 32];
  if (A.sums) {
    policy_sums<TEAM, VEC>(A, red);
    cooperative_groups::this_grid().sync();
  }
  policy_losses<TEAM, VEC, KL, true>(A, gridDim.x, red);
  cooperative_groups::this_grid().sync();
  if (blockIdx.x == 0) policy_join(A, gridDim.x, red);
}

// out = x g, the gradient of a loss whose unit gradient x was kept; 0 where x is 0
// (a token that takes no part), also for a g that is not finite.  out may be x:
// each value is read and written by one thread.
template <bool VEC>
__global__ void __launch_bounds__(kThreads) scale_kernel(const float* x, const float* __restrict__ g, float* out, int n) {
  const float s = *g;
  for (int64_t t0 = 4 * ((int64_t)blockIdx.x * kThreads + threadIdx.x); t0 < n; t0 += 4 * (int64_t)gridDim.x * kThreads) {
    float v[4];
    load4<VEC>(x, (int)t0, 0, n, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = v[j] != 0.f ? v[j] * s : 0.f;
    store4<VEC>(out, (int)t0, 0, n, v);
  }
}

}  // namespace seq
}  // namespace kd
