// Host side of the losses over token log-probabilities (kd_preference_loss,
// kd_policy_loss): argument checks, workspace layout, how the sequences are
// cut into items, and the launches.

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "../../include/kd_topk_kl.h"
#include "kd_sequence_losses.cuh"

using namespace kd::seq;

namespace {

constexpr int64_t kSplitItems = 592;      // items to aim at when few sequences are split: one wave, 4 blocks per SM
constexpr int64_t kTokensPerItem = 4 * kThreads;
constexpr int64_t kWarpTokens = 192;      // mean length up to which a warp takes a sequence

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// The counter, the blocks' partials, then the items' sums.  At most
// max(S, kSplitItems) items, whatever the lengths (see split_of).
struct Layout {
  size_t off_counter = 0, off_total = 0, off_part = 0, off_sums = 0, total = 0;
};

Layout make_layout(int64_t S) {
  Layout L;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t r = o; o = align256(o + bytes); return r; };
  L.off_counter = take(sizeof(unsigned int));
  L.off_total = take(sizeof(double) * kSumBlocks);
  L.off_part = take(sizeof(double) * 3 * kLossBlocks);
  L.off_sums = take(sizeof(double) * 2 * (size_t)(S > kSplitItems ? S : kSplitItems));
  L.total = o;
  return L;
}

int check_sequences(int64_t S, int64_t N, const void* offsets, int offsets_i64) {
  if (S < 0 || N < 0 || (offsets_i64 & ~1)) return KD_ERR_INVALID_ARG;
  if (S >= (int64_t(1) << 31) || N > kMaxTokens) return KD_ERR_UNSUPPORTED;
  if (!offsets && (S == 0 ? N != 0 : N % S != 0)) return KD_ERR_INVALID_ARG;
  if (offsets && !aligned(offsets, offsets_i64 ? 8 : 4)) return KD_ERR_INVALID_ARG;
  return KD_OK;
}

// A warp per sequence for short sequences, else a block, and when there are
// fewer sequences than the GPU holds blocks, several blocks (each with at
// least one pass of tokens) per sequence.
Sequences split_of(int64_t S, int64_t N, const void* offsets, int offsets_i64, int* team) {
  Sequences q{offsets, offsets_i64, S, N, S > 0 ? N / S : 0, 1};
  const int64_t mean = q.L;
  *team = mean <= kWarpTokens ? 32 : kThreads;
  if (*team == kThreads && S < kSplitItems) {
    const int64_t room = kSplitItems / S, need = (mean + kTokensPerItem - 1) / kTokensPerItem;
    q.splits = (int)(need < room ? need : room);
    if (q.splits < 1) q.splits = 1;
  }
  return q;
}

unsigned blocks_for(const Sequences& q, int team, int most) {
  const int64_t teams = kThreads / team, items = q.S * q.splits;
  const int64_t b = (items + teams - 1) / teams;
  return (unsigned)(b < 1 ? 1 : (b < most ? b : most));
}

bool all_aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p && !aligned(p, 16)) return false;
  return true;
}

void two_floats(double v, float* h, float* l) {
  *h = (float)v;
  *l = std::isfinite(v) ? (float)(v - (double)*h) : 0.f;
}

int launched() { return cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA; }

template <class K, class... A>
int next(K kernel, unsigned blocks, cudaStream_t s, A&&... args) {
  return kd::launch_next(kernel, blocks, (unsigned)kThreads, s, args...) == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}

// SMs of the current device.
int current_sms() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Whether the phases are one launch: a call whose time is the host's, every
// item of which has a team of its own among the blocks that the GPU holds at once.
bool one_launch(const Sequences& q, int team, unsigned blocks) {
  return q.N <= kOneLaunchTokens && (int64_t)blocks * (kThreads / team) >= q.S * q.splits && blocks <= (unsigned)(kResident * current_sms());
}

template <class K, class A>
int cooperative(K kernel, unsigned blocks, cudaStream_t s, const A& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess ? launched() : KD_ERR_CUDA;
}

template <int TEAM, bool VEC>
int run_preference(const PrefArgs& A, cudaStream_t s) {
  const unsigned blocks = blocks_for(A.q, TEAM, kLossBlocks);
  if (one_launch(A.q, TEAM, blocks)) return cooperative(pref_one_kernel<TEAM, VEC>, blocks, s, A);
  pref_sums_kernel<TEAM, VEC><<<blocks_for(A.q, TEAM, kSumBlocks), kThreads, 0, s>>>(A);
  if (launched() != KD_OK) return KD_ERR_CUDA;
  return next(pref_loss_kernel<TEAM, VEC>, blocks, s, A);
}

template <int TEAM, bool VEC, int KL>
int run_policy(PolicyArgs A, cudaStream_t s) {
  const unsigned blocks = blocks_for(A.q, TEAM, kLossBlocks);
  const bool own_sums = A.per_sequence && A.q.splits == 1;
  if (own_sums) A.sums = nullptr;
  if (one_launch(A.q, TEAM, blocks)) return cooperative(policy_one_kernel<TEAM, VEC, KL>, blocks, s, A);
  if (own_sums) {
    policy_loss_kernel<TEAM, VEC, KL><<<blocks, kThreads, 0, s>>>(A, 0);
    if (launched() != KD_OK) return KD_ERR_CUDA;
    return next(policy_finish_kernel, 1, s, A, (int)blocks);
  }
  const unsigned sum_blocks = blocks_for(A.q, TEAM, kSumBlocks);
  policy_sums_kernel<TEAM, VEC><<<sum_blocks, kThreads, 0, s>>>(A);
  if (launched() != KD_OK) return KD_ERR_CUDA;
  return next(policy_loss_kernel<TEAM, VEC, KL>, blocks, s, A, (int)sum_blocks);
}

template <int TEAM, bool VEC>
int run_policy_kl(int kl, const PolicyArgs& A, cudaStream_t s) {
  switch (kl) {
    case kK1: return run_policy<TEAM, VEC, kK1>(A, s);
    case kK2: return run_policy<TEAM, VEC, kK2>(A, s);
    case kK3: return run_policy<TEAM, VEC, kK3>(A, s);
    default: return run_policy<TEAM, VEC, kNoKl>(A, s);
  }
}

}  // namespace

extern "C" {

size_t kd_sequence_loss_workspace_size(int64_t S) {
  if (S < 0 || S >= (int64_t(1) << 31)) return 0;
  return make_layout(S).total;
}

int kd_preference_loss(const float* logp, const float* ref_logp, const float* mask, const void* offsets,
                       int offsets_i64, int64_t S, int64_t N, double beta, int kind, double label_smoothing,
                       double margin, int average, const float* grad_loss, float* loss, float* chosen,
                       float* rejected, float* dlogp, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_sequences(S, N, offsets, offsets_i64);
  if (st != KD_OK) return st;
  if (S % 2 != 0 || kind < 0 || kind > 2 || (average & ~1)) return KD_ERR_INVALID_ARG;
  if (!(beta > 0.0) || !std::isfinite(beta) || !std::isfinite(margin) || !(label_smoothing >= 0.0) ||
      !(label_smoothing <= 1.0))
    return KD_ERR_INVALID_ARG;
  if (!loss || !workspace || (N > 0 && !logp) || (S > 0 && (!chosen || !rejected))) return KD_ERR_INVALID_ARG;
  for (const void* p : {(const void*)logp, (const void*)ref_logp, (const void*)mask, (const void*)grad_loss,
                        (const void*)loss, (const void*)chosen, (const void*)rejected, (const void*)dlogp})
    if (!aligned(p, 4)) return KD_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return KD_ERR_INVALID_ARG;
  const Layout L = make_layout(S);
  if (workspace_bytes < L.total) return KD_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  PrefArgs A{};
  int team = 0;
  A.q = split_of(S, N, offsets, offsets_i64, &team);
  A.logp = logp;
  A.ref = ref_logp;
  A.mask = mask;
  A.grad_loss = grad_loss;
  A.beta = beta;
  A.smoothing = label_smoothing;
  A.margin = margin;
  A.kind = kind;
  A.average = average;
  A.sums = reinterpret_cast<double*>(ws + L.off_sums);
  A.part = reinterpret_cast<double*>(ws + L.off_part);
  A.counter = reinterpret_cast<unsigned int*>(ws + L.off_counter);
  A.loss = loss;
  A.chosen = chosen;
  A.rejected = rejected;
  A.dlogp = dlogp;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = all_aligned16({logp, ref_logp, mask, dlogp});
  if (team == 32) return vec ? run_preference<32, true>(A, s) : run_preference<32, false>(A, s);
  return vec ? run_preference<kThreads, true>(A, s) : run_preference<kThreads, false>(A, s);
}

int kd_policy_loss(const float* logp, const float* old_logp, const float* ref_logp, const float* advantages,
                   int advantages_per_sequence, const float* mask, const void* offsets, int offsets_i64, int64_t S,
                   int64_t N, double clip_low, double clip_high, double dual_clip, double kl_coef, int kl_kind,
                   int per_sequence, const float* grad_loss, float* loss, float* dlogp, void* workspace,
                   size_t workspace_bytes, void* stream) {
  int st = check_sequences(S, N, offsets, offsets_i64);
  if (st != KD_OK) return st;
  if (kl_kind < 0 || kl_kind > 2 || (advantages_per_sequence & ~1) || (per_sequence & ~1)) return KD_ERR_INVALID_ARG;
  if (!(clip_low >= 0.0) || !(clip_low < 1.0) || !(clip_high >= 0.0) || !std::isfinite(clip_high) ||
      !std::isfinite(kl_coef) || !(dual_clip == 0.0 || (dual_clip > 1.0 && std::isfinite(dual_clip))))
    return KD_ERR_INVALID_ARG;
  if (!loss || !workspace || (N > 0 && (!logp || !old_logp || !advantages))) return KD_ERR_INVALID_ARG;
  for (const void* p : {(const void*)logp, (const void*)old_logp, (const void*)ref_logp, (const void*)advantages,
                        (const void*)mask, (const void*)grad_loss, (const void*)loss, (const void*)dlogp})
    if (!aligned(p, 4)) return KD_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return KD_ERR_INVALID_ARG;
  const Layout L = make_layout(S);
  if (workspace_bytes < L.total) return KD_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  PolicyArgs A{};
  int team = 0;
  A.q = split_of(S, N, offsets, offsets_i64, &team);
  A.logp = logp;
  A.old = old_logp;
  A.ref = ref_logp;
  A.adv = advantages;
  A.mask = mask;
  A.grad_loss = grad_loss;
  A.adv_per_seq = advantages_per_sequence;
  A.per_sequence = per_sequence;
  A.log_hi = std::log1p(clip_high);
  A.log_lo = std::log1p(-clip_low);
  A.log_dual = dual_clip == 0.0 ? INFINITY : std::log(dual_clip);
  two_floats(A.log_hi, &A.hi_h, &A.hi_l);
  two_floats(A.log_lo, &A.lo_h, &A.lo_l);
  two_floats(A.log_dual, &A.dual_h, &A.dual_l);
  A.hi1 = (float)(A.hi1_64 = 1.0 + clip_high);
  A.lo1 = (float)(A.lo1_64 = 1.0 - clip_low);
  A.dual_64 = dual_clip;
  A.kl_coef_64 = kl_coef;
  A.dual_c = (float)dual_clip;
  A.kl_coef = (float)kl_coef;
  A.sums = reinterpret_cast<double*>(ws + L.off_sums);
  A.total = reinterpret_cast<double*>(ws + L.off_total);
  A.part = reinterpret_cast<double*>(ws + L.off_part);
  A.counter = reinterpret_cast<unsigned int*>(ws + L.off_counter);
  A.loss = loss;
  A.dlogp = dlogp;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = all_aligned16({logp, old_logp, ref_logp, advantages_per_sequence ? nullptr : advantages, mask, dlogp});
  const int kl = ref_logp ? kl_kind : kNoKl;
  if (team == 32) return vec ? run_policy_kl<32, true>(kl, A, s) : run_policy_kl<32, false>(kl, A, s);
  return vec ? run_policy_kl<kThreads, true>(kl, A, s) : run_policy_kl<kThreads, false>(kl, A, s);
}

int kd_scale_gradient(const float* x, const float* g, float* out, int64_t N, void* stream) {
  if (N < 0 || !g || (N > 0 && (!x || !out))) return KD_ERR_INVALID_ARG;
  if (N > kMaxTokens) return KD_ERR_UNSUPPORTED;
  if (!aligned(x, 4) || !aligned(g, 4) || !aligned(out, 4)) return KD_ERR_INVALID_ARG;
  if (N == 0) return KD_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t b = (N + kTokensPerItem - 1) / kTokensPerItem;
  const unsigned grid = (unsigned)(b < kLossBlocks ? b : kLossBlocks);
  if (all_aligned16({x, out})) scale_kernel<true><<<grid, kThreads, 0, s>>>(x, g, out, (int)N);
  else scale_kernel<false><<<grid, kThreads, 0, s>>>(x, g, out, (int)N);
  return launched();
}

}  // extern "C"
