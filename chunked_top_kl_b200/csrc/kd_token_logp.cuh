// Label log-probabilities of tokens under the LM head, and their gradient:
//   z = H W^T / T,  lse_n = log sum_v exp z_nv,  logp_n = z[n, y_n] - lse_n,
//   ent_n = lse_n - sum_v p_nv z_nv              (p = softmax z)
//   dZ_nv = (1/T) [ g_n (1[v = y_n] - p_nv) - h_n p_nv (log p_nv + ent_n) ]
//   dH = dZ W,  dW = dZ^T H
// for upstream gradients g of logp and h of ent.
//
// The products are the GEMM of kd_gemm.cuh with the epilogues below; as in
// the distillation loss the logits are never stored, and recomputed chunk by
// chunk for the gradient.  Both passes are bound by the tensor cores once
// there are a few hundred tokens, by the bytes of W below that (2 V d read).
//
// Only tokens that count are multiplied: a negative label (a prompt token) and,
// going back, a token whose upstream gradient is zero (masked or clipped) have
// their rows left out.  The rows that stay are listed on the device, their H
// rows gathered (N d 4 bytes of copying against 2 N d V operations), and the
// GEMMs take the row count and the schedule for it from device memory.
#pragma once

#include "kd_gemm.cuh"

namespace kd {

constexpr int kLabelThreads = 1024;
constexpr float kLn2 = 0.6931471805599453f;

// The tensor cores' fp32 accumulation truncates at every step, so a logit that
// they return is short of the exact one by a share of itself that grows with
// the number of steps.  Measured over random and drifting rows, the mean of
// (z - z_exact) / z_exact is -d 2^-23 times 0.0064 (d = 256), 0.0075 (2048),
// 0.0081 (8192), the same for small and large logits: 2.6e-6 at d = 2880, two
// fp32 steps, and always the same way, so it would add up over a sequence's
// tokens.  The logits' scale makes up for the mean.
__host__ __device__ __forceinline__ double accumulation_gain(int64_t d) { return 1.0 + 0.0077 * (double)d / 8388608.0; }

// What the label scan leaves for the kernels behind it.
struct LiveRows {
  int count;         // rows that take part
  int pad;
  Raster raster;     // forward: of all of them; backward: of the last, partly filled chunk
  DhPlan dh;         // backward: how that chunk's dH product is cut
};

struct LabelPrep {
  const void* labels;
  int labels_i64;
  int N, V;
  const float *dlogp, *dent;      // backward: upstream gradients (dent may be null); null in the forward pass
  float *logp, *lse, *ent;        // forward: outputs to clear for tokens that take no part (ent may be null)
  int32_t *rowmap, *lab;          // the live tokens in order, and their labels
  LiveRows* live;
  Status* status;
  // the schedule: rows of `chunk` at most (backward; 0: all rows), column tiles, CTA pairs
  int64_t chunk;
  int n_tiles, groups, max_splits;
  int64_t part_slots;             // forward: bounds the ranges by the partial slots (0: no bound)
  int64_t band_bytes, l2_bytes;
  unsigned int* wave;             // forward: pacing counters to clear
  // backward: the joint launch of dH and dW (see dh_plan)
  int64_t d, dw_units, part_rows;
  int joint_groups;
};

// One block lists the tokens that take part, in increasing order, with their
// labels.  Labels at or above V are counted in the status words; their
// log-probability is NaN, and they take no further part.
__global__ void __launch_bounds__(kLabelThreads) label_prep_kernel(const LabelPrep P) {
  __shared__ int s_warp[kLabelThreads / 32];
  __shared__ unsigned int s_bad;
  __shared__ unsigned long long s_best, s_dh;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  next_may_start();
  if (t == 0) {
    s_bad = 0u;
    s_best = s_dh = ~0ull;
  }
  int total = 0;
  for (int64_t base = 0; base < P.N; base += 4 * kLabelThreads) {
    const int64_t n0 = base + 4 * t;
    int lab[4], keep = 0;
    int64_t y[4];
    float g[4], h[4];
    unsigned int bad = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {             // all loads first
      const int64_t n = n0 + j;
      const bool in = n < P.N;
      y[j] = !in ? -1
                 : P.labels_i64 ? static_cast<const int64_t*>(P.labels)[n]
                                : (int64_t) static_cast<const int32_t*>(P.labels)[n];
      g[j] = in && P.dlogp ? P.dlogp[n] : 0.f;
      h[j] = in && P.dent ? P.dent[n] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + j;
      bool on = y[j] >= 0 && y[j] < P.V;
      const bool wrong = y[j] >= P.V;
      bad += wrong;
      if (P.dlogp) {
        on = on && (g[j] != 0.f || h[j] != 0.f);        // NaN stays in
      } else if (!on && n < P.N) {
        const float v = wrong ? __int_as_float(0x7fc00000) : 0.f;
        P.logp[n] = v;
        P.lse[n] = v;
        if (P.ent) P.ent[n] = v;
      }
      lab[j] = on ? (int)y[j] : -1;
      keep += on;
    }
    int scan = keep;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    __syncthreads();                       // the last tile's totals have been read
    if (lane == 31) s_warp[warp] = scan;
    if (bad) atomicAdd(&s_bad, bad);
    __syncthreads();
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += v;
    }
    const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    int o = total + (warp > 0 ? before : 0) + scan - keep;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lab[j] >= 0) {
        P.rowmap[o] = (int32_t)(n0 + j);
        P.lab[o++] = lab[j];
      }
    total += __shfl_sync(0xffffffffu, w, 31);
  }
  // The schedule of the live rows: forward_raster's search, a thread for each number of ranges.
  const int64_t rows = P.chunk > 0 ? total % P.chunk : total;
  const int64_t m_tiles = ceil_div64(rows, 256);
  int64_t most = P.max_splits;
  if (P.part_slots > 0 && rows > 0 && P.part_slots / rows < most) most = P.part_slots / rows;
  __syncthreads();
  if (rows > 0 && t + 1 <= most && t + 1 <= P.n_tiles)
    atomicMin(&s_best, ((unsigned long long)split_cost(m_tiles, P.n_tiles, P.groups, t + 1) << 32) | (unsigned)(t + 1));
  const int64_t n_cols = ceil_div64(P.d, 256);
  if (P.chunk > 0 && rows > 0 && t < 2 * kMaxDhSplits) {
    bool wide;
    int ks;
    dh_candidate(t, wide, ks);
    const int64_t c = dh_cost(m_tiles, n_cols, P.d, ceil_div64(P.V, BK), P.dw_units, ceil_div64(rows, BK),
                              P.joint_groups, wide, ks, P.part_rows);
    if (c >= 0) atomicMin(&s_dh, ((unsigned long long)c << 32) | (unsigned)t);
  }
  __syncthreads();
  Raster r{};
  if (rows > 0)
    r = split_raster(m_tiles, P.n_tiles, P.groups, (int)(unsigned)s_best, P.band_bytes, P.l2_bytes);
  if (t == 0) {
    P.live->count = total;
    P.live->raster = r;
    if (P.chunk > 0 && rows > 0) P.live->dh = dh_plan_of((int)(unsigned)s_dh, n_cols);
    P.status->bad_index = s_bad;
    P.status->timeout = 0u;
  }
  if (P.wave)
    for (int64_t i = t; i < wave_slots_bound(r.num_units, 0); i += kLabelThreads) P.wave[i] = 0u;
}

__device__ __forceinline__ float dot8(const uint4& x, const uint4& y) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
  float s[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {           // bf16 is the upper half of an fp32; products are exact
    const float lo = __uint_as_float(a[k] << 16) * __uint_as_float(b[k] << 16);
    s[k] = fmaf(__uint_as_float(a[k] & 0xffff0000u), __uint_as_float(b[k] & 0xffff0000u), lo);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// What the dZ epilogue needs of a row: dZ / scale = p (a + b u) with
// u = z zl2 - bias off the label, `label` at it.
struct RowCoef {
  float bias, a, b, label;
};

// The backward pass's share of gather_live_kernel.
struct RowScales {
  const float *lse, *ent, *dlogp, *dent;   // ent and dent null without an entropy gradient
  const float* logp;        // the forward pass's, or null
  float zs;                 // 1 / T
  RowCoef* coef;            // [C]
  float* scale;             // [C]
  uint4* scaled;            // [C][d8] H rows times their scale; null when no dW is wanted
  uint4* clear;             // dH, cleared: the rows that are left out stay 0
  int64_t clear_n;
  unsigned int* counters;   // the joint launch's pacing counters, cleared
  int64_t counters_n;
};

// Row n's factors. dZ is formed and rounded to bf16 per row as dZ / scale, with
// a scale that makes the label's entry exactly 1 or -1: it is the largest, and
// its rounding error would be a common factor of the token's whole dH row.  dH
// is multiplied by the scale in fp32, and dW = dZ^T H takes it with H, whose
// elements round independently.  With pl = p at the label:
//   without an entropy gradient  scale = -g (1 - pl) / T, dZ / scale = p / (1 - pl)
//   (1 - pl folded into the exponent), -1 at the label;
//   with one, a = -(g + h ent) / T, b = -h ln 2 / T, the label's entry
//   L = (g (1 - pl) - h pl (log pl + ent)) / T is the scale unless it is small
//   beside |g| + |h| (then that is, and L / scale is rounded as the others are).
// log pl is z_y / T - lse from the exact logit, about 1e-6 off where lse is 20
// (its rounding): below 2^-14 of 1 - pl = 1/16, but all of a 1 - pl of 1e-6.  So
// where 1 - pl is below 1/16 the forward pass's log pl is taken, which is exact
// to some 1e-5 of itself; without one (`logp` null) the 1e-6 stay.
__device__ __forceinline__ RowCoef row_coef(const RowScales& B, int n, float zy, float& scale) {
  RowCoef c;
  const float g = B.dlogp[n] * B.zs;
  float logp = fmaf(zy, B.zs, -B.lse[n]), om = -expm1f(logp);
  if (B.logp && om < 0.0625f) {
    logp = B.logp[n];
    om = -expm1f(logp);
  }
  c.bias = B.lse[n] * kLog2e;
  if (!B.dent) {
    const float room = om < 5.42e-20f ? 5.42e-20f : om;       // 2^-64, for a division; NaN stays
    scale = -g * room;
    c.bias += log2f(room);
    c.a = c.b = 0.f;
    c.label = -1.f;
    return c;
  }
  const float h = B.dent[n] * B.zs, ent = B.ent[n], base = fabsf(g) + fabsf(h);
  const float L = g * om - h * (1.f - om) * (logp + ent);
  const bool own = fabsf(L) > base * 9.77e-4f;                 // 2^-10
  scale = own ? L : base;
  if (scale == 0.f) {                          // g / T and h / T are below the smallest float
    c.a = c.b = c.label = 0.f;
    return c;
  }
  c.a = -fmaf(h, ent, g) / scale;
  c.b = -h * kLn2 / scale;
  c.label = own ? 1.f : L / scale;
  return c;
}

__device__ __forceinline__ uint32_t scale2(uint32_t x, float s) {
  const float lo = __uint_as_float(x << 16) * s, hi = __uint_as_float(x & 0xffff0000u) * s;
  return pack_bf16x2(lo, hi);
}

// Rows [row0, row0 + C) of the live list: dst[r] = src[rowmap[row0 + r]]
// (16-byte vectors, d8 per row), a warp per row.  Rows past the live ones are
// zero up to the end of the last band of 256, as far as the GEMMs read.
//
// Each row's label logit H[n] W[lab] is taken on the way, in 64-bit partial
// sums: it enters the log-probability undiminished, and the tensor cores return
// a logit of ten some 1e-5 off at d = 2880.  W's rows are read beside H's, 2 d
// more bytes a row.  The forward pass keeps it (zlab); going back, the row's
// scale and coefficients come from it.
//
// Of the first rows, kPadRows are written even when fewer are live: loads of a
// band with a row or two made the one-token product 1.4 times slower (294 us
// against 207 us at d = 2880, 1.07 GB of W) than those of 64 rows.
constexpr int kPadRows = 64;

template <bool BACKWARD>
__global__ void __launch_bounds__(256)
gather_live_kernel(const uint4* __restrict__ src, int d8, const int32_t* __restrict__ rowmap,
                   const LiveRows* __restrict__ live, int row0, int C, uint4* __restrict__ dst,
                   const uint4* __restrict__ W, const int32_t* __restrict__ lab, float* __restrict__ zlab,
                   const RowScales B) {
  next_may_start();
  wait_previous();
  if (BACKWARD) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = i0; i < B.clear_n; i += step) B.clear[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t i = i0; i < B.counters_n; i += step) B.counters[i] = 0u;
  }
  int rows = live->count - row0;
  rows = rows < 0 ? 0 : (rows > C ? C : rows);
  const int64_t room = C > kPadRows ? C : kPadRows, want = ceil_div64(rows, 256) * 256;
  const int64_t end = want < room ? want : room;
  const int lane = threadIdx.x & 31;
  for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < end; r += (int64_t)gridDim.x * 8) {
    uint4* to = dst + (size_t)r * d8;
    uint4* scaled = BACKWARD && B.scaled ? B.scaled + (size_t)r * d8 : nullptr;
    if (r >= rows) {
      for (int j = lane; j < d8; j += 32) {
        to[j] = make_uint4(0u, 0u, 0u, 0u);
        if (scaled) scaled[j] = make_uint4(0u, 0u, 0u, 0u);
      }
      continue;
    }
    const int n = rowmap[row0 + r];
    const uint4 *from = src + (size_t)n * d8, *w = W + (size_t)lab[row0 + r] * d8;
    double z = 0.0;
    for (int j = lane; j < d8; j += 32) {
      const uint4 h = from[j];
      to[j] = h;
      z += (double)dot8(h, w[j]);
    }
    z = warp_sum_d(z);
    if (!BACKWARD) {
      if (lane == 0) zlab[row0 + r] = (float)z;
      continue;
    }
    float scale;
    const RowCoef c = row_coef(B, n, (float)z, scale);
    if (lane == 0) {
      B.coef[r] = c;
      B.scale[r] = scale;
    }
    if (scaled)
      for (int j = lane; j < d8; j += 32) {
        const uint4 h = from[j];
        scaled[j] = make_uint4(scale2(h.x, scale), scale2(h.y, scale), scale2(h.z, scale), scale2(h.w, scale));
      }
  }
}

// Forward: running scaled maximum and sum-exp over the unit's vocabulary
// columns but the label's, and with ENT the sum of e u that the entropy
// needs.  In log2 units, u_v = z_v zl2 - mb with zl2 = log2(e) / T (times
// accumulation_gain) and mb = max z * zl2 as rounded: s = sum 2^u and
// t = sum 2^u u (u <= 0, so t does not cancel).  A new maximum shifts u by
// delta = mb_old - mb_new: t <- 2^delta (t + delta s), s <- 2^delta s.
// The label's own term comes in when all others are summed, from its exact
// logit (logp_merge_kernel): beside a label of probability one the others would
// be lost in an fp32 sum that holds it, and log p with them.
// Partials {mb, s, t, -} per live row and column range.  The label's column and
// columns >= V are taken as kNoLogit; the maximum starts far above it and below
// any logit, so that u is finite and 2^u 0 in a range without other columns.
constexpr float kNoLogit = -1e30f, kLeastMax = -1e29f;

template <bool ENT>
struct EpiLogp {
  static constexpr bool kStaging = false;
  struct Params {
    int V;
    float zl2;
    const int32_t* lab;
    float4* part;
  };
  float mrun, srun, trun;
  int grow, rows, label;

  __device__ __forceinline__ void begin_unit(const Params& P, int grow_, int, int, const EpiCtx& cx) {
    grow = grow_;
    rows = cx.rows_valid;
    mrun = kLeastMax;
    srun = 0.f;
    trun = 0.f;
    label = grow < rows ? P.lab[grow] : -1;
  }

  __device__ __forceinline__ void tile(const Params& P, const CUtensorMap*, int, int n, uint32_t taddr, EpiCtx&) {
    const float zl2 = P.zl2;
#pragma unroll 1
    for (int j = 0; j < BN / 64; ++j) {
      float v[64];
      __syncwarp();
      tmem_ld_32x32b_x64(taddr + j * 64, v);
      const int c0 = n * BN + j * 64;
      if (c0 + 64 > P.V) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (c0 + i >= P.V) v[i] = kNoLogit;
      }
      const int off = label - c0;
      if ((unsigned)off < 64u) {              // once per row
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (i == off) v[i] = kNoLogit;
      }
      float t[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) t[i] = fmaxf(v[i], v[i + 32]);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) t[i] = fmaxf(t[i], t[i + w]);
      const float mn = fmaxf(mrun, t[0]);
      const float mb = mn * zl2;
      if (mn > mrun) {                        // rare after the first columns
        const float delta = mrun * zl2 - mb;
        const float f = ex2_approx(delta);
        if (ENT) trun = f > 0.f ? f * fmaf(delta, srun, trun) : 0.f;
        srun *= f;
        mrun = mn;
      }
      const float2 zl2v = make_float2(zl2, zl2), nmb = make_float2(-mb, -mb);
      float2 a01 = make_float2(0.f, 0.f), a23 = a01, b01 = a01, b23 = a01;
#pragma unroll
      for (int i = 0; i < 64; i += 4) {
        const float2 u01 = __ffma2_rn(make_float2(v[i + 0], v[i + 1]), zl2v, nmb);
        const float2 u23 = __ffma2_rn(make_float2(v[i + 2], v[i + 3]), zl2v, nmb);
        const float2 e01 = make_float2(ex2_approx(u01.x), ex2_approx(u01.y));
        const float2 e23 = make_float2(ex2_approx(u23.x), ex2_approx(u23.y));
        a01 = __fadd2_rn(a01, e01);
        a23 = __fadd2_rn(a23, e23);
        if (ENT) {
          b01 = __ffma2_rn(e01, u01, b01);
          b23 = __ffma2_rn(e23, u23, b23);
        }
      }
      srun += (a01.x + a01.y) + (a23.x + a23.y);
      if (ENT) trun += (b01.x + b01.y) + (b23.x + b23.y);
    }
  }

  __device__ __forceinline__ void end_unit(const Params& P, int, int split) {
    if (grow < rows) P.part[(size_t)split * rows + grow] = make_float4(mrun * P.zl2, srun, trun, 0.f);
  }
};

// A row's state over some of the columns: m (the scaled maximum mb of
// EpiLogp), s and t.
template <bool ENT>
struct LogpState {
  float m, s, t;

  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    s = t = 0.f;
  }
  __device__ __forceinline__ void join(const LogpState& o) {
    const float top = fmaxf(m, o.m);
    const float d1 = m == top ? 0.f : m - top, d2 = o.m == top ? 0.f : o.m - top;
    const float f1 = ex2_approx(d1), f2 = ex2_approx(d2);
    if (ENT) t = (f1 > 0.f ? f1 * fmaf(d1, s, t) : 0.f) + (f2 > 0.f ? f2 * fmaf(d2, o.s, o.t) : 0.f);
    s = fmaf(f1, s, f2 * o.s);
    m = top;
  }
  // One more column's logit.
  __device__ __forceinline__ void add(float z, float zl2) {
    const float mb = fmaxf(m, z * zl2);
    if (mb > m) {
      const float delta = m - mb, f = ex2_approx(delta);
      if (ENT) t = f > 0.f ? f * fmaf(delta, s, t) : 0.f;
      s *= f;
      m = mb;
    }
    const float u = fmaf(z, zl2, -m), e = ex2_approx(u);
    s += e;
    if (ENT) t = fmaf(e, u, t);
  }
  __device__ __forceinline__ LogpState shuffled(int o) const {
    LogpState r;
    r.m = __shfl_xor_sync(0xffffffffu, m, o);
    r.s = __shfl_xor_sync(0xffffffffu, s, o);
    r.t = ENT ? __shfl_xor_sync(0xffffffffu, t, o) : 0.f;
    return r;
  }
};

__device__ __forceinline__ bool status_timed_out(const Status* s) {
  return *reinterpret_cast<const volatile unsigned int*>(&s->timeout) != 0u;
}

// Joins the column ranges' partials of a row, then takes in the label's term,
// from its exact logit z_y (see gather_live_kernel).  With M the others' scaled
// maximum, s and t their sums, and u = z_y log2(e) / T - M:
//   u < 0:  S = s + 2^u,  logp = ln 2 (u - log2 S),  lse = ln 2 (M + log2 S),
//           ent = ln 2 (log2 S - (t + 2^u u) / S)
//   u >= 0: over the label's term, r = 2^-u s (the others' sum),
//           logp = -log(1 + r),  lse = z_y / T + log(1 + r),
//           ent = log(1 + r) - ln 2 2^-u (t - u s) / (1 + r):
// a confident token's log-probability, -r as r goes to 0, keeps its relative
// precision, and with it 1 - p.  It is written a second time (`kept`, may be
// null) for the gradient: the first is the caller's to change.
//
// ROWS rows a block, LANES threads a row: 32 and 8 for the GEMM's few ranges,
// one row and 256 threads for the many of logp_few_kernel.
template <bool ENT, int ROWS, int LANES>
__global__ void __launch_bounds__(ROWS * LANES)
logp_merge_kernel(const float4* __restrict__ part, const LiveRows* __restrict__ live,
                  const int32_t* __restrict__ rowmap, const float* __restrict__ zlab, float zl2_exact,
                  float* __restrict__ logp, float* __restrict__ kept, float* __restrict__ lse, float* __restrict__ ent,
                  const Status* __restrict__ status) {
  __shared__ LogpState<ENT> s_part[LANES][ROWS];
  wait_previous();
  const int rows = live->count, splits = live->raster.splits;
  const int x = threadIdx.x % ROWS, y = threadIdx.x / ROWS;
  const int q = blockIdx.x * ROWS + x;
  LogpState<ENT> st;
  st.clear();
  if (q < rows)
    for (int k = y; k < splits; k += LANES) {
      const float4 p = part[(size_t)k * rows + q];
      st.join(LogpState<ENT>{p.x, p.y, p.z});
    }
  s_part[y][x] = st;
#pragma unroll
  for (int w = LANES / 2; w > 0; w >>= 1) {
    __syncthreads();
    if (y < w) {
      st.join(s_part[y + w][x]);
      s_part[y][x] = st;
    }
  }
  if (y == 0 && q < rows) {
    const int n = rowmap[q];
    const float zy = zlab[q] * zl2_exact, u = fmaf(zlab[q], zl2_exact, -st.m);
    float lp, ls, en;
    if (u >= 0.f) {
      const float f = exp2f(-u), r = f * st.s, l = log1pf(r);
      lp = -l;
      ls = fmaf(kLn2, zy, l);
      en = f > 0.f ? l - kLn2 * f * fmaf(-u, st.s, st.t) / (1.f + r) : l;
    } else {                                  // NaN too
      const float e = exp2f(u), s = st.s + e, l2 = log2f(s);
      lp = kLn2 * (u - l2);
      ls = kLn2 * (st.m + l2);
      en = kLn2 * (l2 - (e > 0.f ? fmaf(e, u, st.t) : st.t) / s);
    }
    if (status_timed_out(status)) lp = ls = en = __int_as_float(0x7fc00000);
    logp[n] = lp;
    lse[n] = ls;
    if (kept) kept[n] = lp;
    if (ENT) ent[n] = en;
  }
}

// ---------------------------------------------------------------- a few tokens
//
// Up to eight tokens (a single token's score, a draft to verify): the time is
// that of reading W once, 2 V d bytes, and the GEMM above, whose tiles are 256
// tokens high, reads it at 4.6 TB/s (250 us at V = 201,088, d = 2880, one token).
// Here each warp streams a contiguous range of W's rows straight into registers,
// sixteen rows at a time, as the A operand of m16n8k16 products with the tokens
// as columns: the tensor cores idle nearly all of the time, so the plain
// warp-level product serves.  A thread's 16-byte load holds eight consecutive k
// of a row where the product's layout wants two groups of two times two; as every
// k counts alike, A and B take the same eight in the same order.  H lies in shared
// memory in the order of the loads (few_smem bytes: a d that does not fit goes to
// the GEMM); read through L1 it was pushed out by the stream of W (206 us instead
// of 195 us for a token).  The running softmax state is as in EpiLogp, a thread
// holding two tokens (per eight) over the rows it meets; warps, then blocks
// (through the partials, one range per block) are joined.
//
// Measured against the GEMM's 128-row tiles (us): V = 201,088, d = 2880, up to
// eight tokens 190, nine to sixteen 223 against 205; V = 32,000, d = 2048, 31, and
// 35 against 43; V = 8,000, d = 512, 17 against 20.  So nine to sixteen tokens come
// here where W is small (kFewWideBytes) and launches are a part of the time.
//
// Every kFewBatch k blocks the products start from zero and are added up in
// fp32 with rounding: sums so short need no accumulation_gain.
constexpr int64_t kFewWideBytes = 200 << 20;
constexpr int kFewTokens = 16;
constexpr int kFewWarps = 8, kFewThreads = 32 * kFewWarps;
constexpr int kFewBatch = 4;                  // k blocks of 32 whose loads are in flight together
constexpr int kFewBlocksPerSm = 2;            // one wave: the ranges are even

// Bytes of H in shared memory for N tokens, and the most that two blocks of an SM can have.
KD_HD int64_t few_smem(int64_t N, int64_t d) { return ceil_div64(N, 8) * ceil_div64(d, 32) * 512; }
constexpr int64_t kFewSmem = 110 * 1024;

struct FewArgs {
  const uint4 *H, *W;
  const void* labels;
  int labels_i64, N, V, d8;
  float zl2;
  float *logp, *lse, *ent;
  int32_t* rowmap;
  LiveRows* live;
  Status* status;
  float* zlab;
  float4* part;
};

__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int NT, bool ENT>
__global__ void __launch_bounds__(kFewThreads, kFewBlocksPerSm) logp_few_kernel(const FewArgs A) {
  __shared__ int s_tok[kFewTokens], s_lab[kFewTokens];
  __shared__ LogpState<ENT> s_part[kFewWarps][8 * NT];
  next_may_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  // every warp finds the live tokens; block 0 says so to the merge
  int64_t y = -1;
  if (lane < A.N)
    y = A.labels_i64 ? static_cast<const int64_t*>(A.labels)[lane] : (int64_t) static_cast<const int32_t*>(A.labels)[lane];
  const bool on = y >= 0 && y < A.V;
  const unsigned live = __ballot_sync(0xffffffffu, on), wrong = __ballot_sync(0xffffffffu, y >= A.V);
  const int rows = __popc(live), q = __popc(live & ((1u << lane) - 1u));
  if (warp == 0) {
    if (on) {
      s_tok[q] = lane;
      s_lab[q] = (int)y;
    }
    if (blockIdx.x == 0) {
      if (on) A.rowmap[q] = lane;
      if (lane < A.N && !on) {
        const float v = y >= A.V ? __int_as_float(0x7fc00000) : 0.f;
        A.logp[lane] = v;
        A.lse[lane] = v;
        if (ENT) A.ent[lane] = v;
      }
      if (lane == 0) {
        A.live->count = rows;
        A.live->raster.splits = (int)gridDim.x;
        A.status->bad_index = __popc(wrong);
        A.status->timeout = 0u;
      }
    }
  }
  __syncthreads();
  if (rows == 0) return;
  // the exact label logits, a row per block (see gather_live_kernel)
  if (warp == 0)
    for (int r = blockIdx.x; r < rows; r += gridDim.x) {
      const uint4 *h = A.H + (size_t)s_tok[r] * A.d8, *w = A.W + (size_t)s_lab[r] * A.d8;
      double z = 0.0;
      for (int j = lane; j < A.d8; j += 32) z += (double)dot8(h[j], w[j]);
      z = warp_sum_d(z);
      if (lane == 0) A.zlab[r] = (float)z;
    }
  // H: for each eight tokens and k block of 32, lane (g, t)'s eight k of token g
  extern __shared__ uint4 s_h[];
  const int kblocks = (A.d8 + 3) / 4;
  for (int i = threadIdx.x; i < NT * kblocks * 32; i += kFewThreads) {
    const int nt = i / (kblocks * 32), k = (i / 32 % kblocks) * 4 + (i & 3), n = 8 * nt + ((i & 31) >> 2);
    s_h[i] = n < rows && k < A.d8 ? A.H[(size_t)s_tok[n] * A.d8 + k] : make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  int lab[2 * NT];                            // labels of the tokens whose logits it gets: 2 t and 2 t + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) lab[2 * nt + j] = 8 * nt + 2 * t + j < rows ? s_lab[8 * nt + 2 * t + j] : -1;
  }
  LogpState<ENT> st[2 * NT];
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) st[i].clear();

  const int64_t w = (int64_t)blockIdx.x * kFewWarps + warp, nw = (int64_t)gridDim.x * kFewWarps;
  const int r0 = (int)(A.V * w / nw), r1 = (int)(A.V * (w + 1) / nw);
  float z[NT][4];
  // the batch of row r, k blocks from k0; rows past the range repeat its last one, and do not count
  auto load = [&](int r, int k0, uint4 (&va)[kFewBatch], uint4 (&vb)[kFewBatch]) {
    const uint4* pa = A.W + (size_t)(r + g < r1 ? r + g : r1 - 1) * A.d8;
    const uint4* pb = A.W + (size_t)(r + g + 8 < r1 ? r + g + 8 : r1 - 1) * A.d8;
#pragma unroll
    for (int u = 0; u < kFewBatch; ++u) {
      const int k = k0 + 4 * u + t;
      va[u] = vb[u] = make_uint4(0u, 0u, 0u, 0u);
      if (k < A.d8) {
        va[u] = __ldcs(pa + k);
        vb[u] = __ldcs(pb + k);
      }
    }
  };
  auto multiply = [&](int r, int k0, const uint4 (&va)[kFewBatch], const uint4 (&vb)[kFewBatch]) {
    if (k0 == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[nt][j] = 0.f;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < kFewBatch; ++u) {
        const int kb = k0 / 4 + u;              // W is zero past d, H there is not read past its last block
        const uint4 h = s_h[(nt * kblocks + (kb < kblocks ? kb : kblocks - 1)) * 32 + lane];
        mma_m16n8k16(c, va[u].x, vb[u].x, va[u].y, vb[u].y, h.x, h.y);
        mma_m16n8k16(c, va[u].z, vb[u].z, va[u].w, vb[u].w, h.z, h.w);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) z[nt][j] += c[j];
    }
    if (k0 + 4 * kFewBatch < A.d8) return;
    const int ra = r + g, rb = r + g + 8;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        LogpState<ENT>& x = st[2 * nt + j];
        if (ra < r1 && ra != lab[2 * nt + j]) x.add(z[nt][j], A.zl2);
        if (rb < r1 && rb != lab[2 * nt + j]) x.add(z[nt][j + 2], A.zl2);
      }
  };
  auto step = [&](int& r, int& k0) {          // to the next batch
    k0 += 4 * kFewBatch;
    if (k0 >= A.d8) {
      k0 = 0;
      r += 16;
    }
  };
  // two batches in registers: one is multiplied while the other arrives
  uint4 va[kFewBatch], vb[kFewBatch], wa[kFewBatch], wb[kFewBatch];
  int r = r0, k0 = 0;
  if (r < r1) load(r, k0, va, vb);
  while (r < r1) {
    int r2 = r, k2 = k0;
    step(r2, k2);
    if (r2 < r1) load(r2, k2, wa, wb);
    multiply(r, k0, va, vb);
    if (r2 >= r1) break;
    r = r2;
    k0 = k2;
    step(r, k0);
    if (r < r1) load(r, k0, va, vb);
    multiply(r2, k2, wa, wb);
  }
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) {          // over the eight lanes with the same tokens
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) st[i].join(st[i].shuffled(o));
    if (g == 0) s_part[warp][8 * (i / 2) + 2 * t + (i & 1)] = st[i];
  }
  __syncthreads();
  const int n = threadIdx.x;
  if (n < rows) {
    LogpState<ENT> x = s_part[0][n];
    for (int k = 1; k < kFewWarps; ++k) x.join(s_part[k][n]);
    A.part[(size_t)blockIdx.x * rows + n] = make_float4(x.m, x.s, x.t, 0.f);
  }
}

// Backward, per chunk: dZ over the row's scale (see row_coef) in bf16 for the
// chunk's live rows (row-major, ldz columns), stored as EpiDz stores it.  With
// u = z zl2 - bias and p = 2^u: p itself without an entropy gradient (ENT), else
// p (a + b u); the label's entry is set, not computed.
template <bool ENT>
struct EpiDlogp {
  static constexpr bool kStaging = true;
  struct Params {
    int row0;              // live-list index of chunk row 0
    int V;
    float zl2;             // log2(e) / T (times accumulation_gain)
    const int32_t* lab;
    const RowCoef* coef;
  };
  RowCoef c;
  int label;

  __device__ __forceinline__ void begin_unit(const Params& P, int r, int, int, const EpiCtx& cx) {
    c = RowCoef{1e30f, 0.f, 0.f, 0.f};        // rows past the live ones: p = 0 and a finite u
    label = -1;
    if (r < cx.rows_valid) {
      c = P.coef[r];
      label = P.lab[P.row0 + r];
    }
  }
  __device__ __forceinline__ void end_unit(const Params&, int, int) {}

  __device__ __forceinline__ void tile(const Params& P, const CUtensorMap* out, int, int n, uint32_t taddr,
                                       EpiCtx& cx) {
    const float zl2 = P.zl2;
#pragma unroll 1
    for (int j = 0; j < BN / 64; ++j) {
      float v[64];
      __syncwarp();
      tmem_ld_32x32b_x64(taddr + j * 64, v);
      const int c0 = n * BN + j * 64;
      const float2 zl2v = make_float2(zl2, zl2), nb = make_float2(-c.bias, -c.bias);
      const float2 av = make_float2(c.a, c.a), bv = make_float2(c.b, c.b);
#pragma unroll
      for (int i = 0; i < 64; i += 2) {
        const float2 u = __ffma2_rn(make_float2(v[i], v[i + 1]), zl2v, nb);
        float2 e = make_float2(ex2_approx(u.x), ex2_approx(u.y));
        if (ENT) e = __fmul2_rn(e, __ffma2_rn(bv, u, av));
        v[i] = e.x;
        v[i + 1] = e.y;
      }
      if (c0 + 64 > P.V) {                    // last vocabulary tile: zero columns >= V
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (c0 + i >= P.V) v[i] = 0.f;
      }
      const int off = label - c0;
      if (__any_sync(0xffffffffu, (unsigned)off < 64u)) {     // a label in this group (rare)
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (i == off) v[i] = c.label;
      }
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      stage_store(cx, out, c0, cx.row_base, w, false);
    }
  }
};

// dH of a chunk's live rows, or the part of it that one K range gives: fp32
// rows of the parts' buffer (`out`: box {32, 128}, 128-byte swizzle).
struct EpiDhPart {
  static constexpr bool kStaging = true;
  struct Params {
    int unused;
  };
  __device__ __forceinline__ void begin_unit(const Params&, int, int, int, const EpiCtx&) {}
  __device__ __forceinline__ void end_unit(const Params&, int, int) {}

  __device__ __forceinline__ void tile(const Params&, const CUtensorMap* out, int, int n, uint32_t taddr, EpiCtx& cx) {
#pragma unroll 1
    for (int j = 0; j < BN / 32; ++j) {
      float v[32];
      __syncwarp();
      tmem_ld_32x32b_x32(taddr + j * 32, v);
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
      stage_store(cx, out, n * BN + j * 32, cx.row_base, w, false);
    }
  }
};

// dH[token] = bf16(scale * sum over the K ranges, in order) for the chunk's live
// rows; eight values a thread.  `full_splits` is the plan of a chunk that is live
// throughout.  When a pipeline wait of the call has given up, the last chunk's
// launch writes NaN to all of dH and dW instead (Gradients, null before the
// last): in a training step nobody reads the status words.
struct Gradients {
  uint4 *dH, *dW;           // dW null: none wanted
  int64_t dH_n, dW_n;       // 16-byte vectors
};

__global__ void __launch_bounds__(256)
dh_finish_kernel(const float4* __restrict__ part, int d8, const int32_t* __restrict__ rowmap,
                 const LiveRows* __restrict__ live, const float* __restrict__ scale, int row0, int C, int full_splits,
                 uint4* __restrict__ dH, const Status* status, const Gradients all) {
  wait_previous();
  if (status_timed_out(status)) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    const uint32_t nan = 0x7fc07fc0u;         // two bf16 NaN, and an fp32 one
    for (int64_t i = i0; i < all.dH_n; i += step) all.dH[i] = make_uint4(nan, nan, nan, nan);
    for (int64_t i = i0; i < all.dW_n; i += step) all.dW[i] = make_uint4(nan, nan, nan, nan);
    return;
  }
  int rows = live->count - row0;
  rows = rows < 0 ? 0 : (rows > C ? C : rows);
  const int splits = rows == C ? full_splits : live->dh.k_splits;
  const size_t stride = (size_t)ceil_div64(rows, 256) * 256 * d8 * 2;
  const int64_t total = (int64_t)rows * d8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int r = (int)(i / d8), j = (int)(i - (int64_t)r * d8);
    const float4* p = part + ((size_t)r * d8 + j) * 2;
    float4 a = p[0], b = p[1];
#pragma unroll 4
    for (int k = 1; k < splits; ++k) {
      const float4 x = p[k * stride], y = p[k * stride + 1];
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
      b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
    }
    const float s = scale[r];
    dH[(size_t)rowmap[row0 + r] * d8 + j] =
        make_uint4(pack_bf16x2(s * a.x, s * a.y), pack_bf16x2(s * a.z, s * a.w), pack_bf16x2(s * b.x, s * b.y),
                   pack_bf16x2(s * b.z, s * b.w));
  }
}

// dW = dZ^T H of a single chunk, rounded to bf16 and stored (`out`: dW [V][d]
// bf16, box {64, 128}, 128-byte swizzle): half the bytes of an fp32 dW, and
// no pass that converts it.  Rounded once, from the fp32 accumulator.
struct EpiDwHalf {
  static constexpr bool kStaging = true;
  struct Params {
    int unused;
  };
  __device__ __forceinline__ void begin_unit(const Params&, int, int, int, const EpiCtx&) {}
  __device__ __forceinline__ void end_unit(const Params&, int, int) {}

  __device__ __forceinline__ void tile(const Params&, const CUtensorMap* out, int, int n, uint32_t taddr, EpiCtx& cx) {
    const bool empty = cx.rows_valid == 0;    // no live rows: no MMA ran, the tile is zero
#pragma unroll 1
    for (int j = 0; j < BN / 64; ++j) {
      float v[64];
      __syncwarp();
      if (empty) {
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] = 0.f;
      } else {
        tmem_ld_32x32b_x64(taddr + j * 64, v);
      }
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      stage_store(cx, out, n * BN + j * 64, cx.row_base, w, false, kL2EvictFirst);
    }
  }
};

// out = bf16(in): the fp32 dW that several chunks added up; left as it is (NaN, see
// dh_finish_kernel) when a wait has given up.
__global__ void __launch_bounds__(256)
round_bf16_kernel(const float4* __restrict__ in, uint2* __restrict__ out, int64_t n4, const Status* status) {
  wait_previous();
  if (status_timed_out(status)) return;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
    const float4 f = in[i];
    out[i] = make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
  }
}

}  // namespace kd
