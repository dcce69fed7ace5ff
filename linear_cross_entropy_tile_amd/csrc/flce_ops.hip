// Host side of the embedding and loss operators of libflce: argument checks,
// workspace layouts and kernel launches. Declarations and their documentation:
// include/flce.h.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <limits>

#include "flce.h"
#include "flce_embedding.hpp"
#include "flce_launch.hpp"
#include "flce_losses.hpp"
#include "flce_ops_plan.hpp"

namespace {

using namespace flce;

static_assert(sizeof(PolicyLoss::Share) == sum_bytes(4) &&
                  sizeof(PolicyLoss::Total) == sum_bytes(5) &&
                  sizeof(PreferenceLoss::Share) == sum_bytes(1) &&
                  sizeof(PreferenceLoss::Total) == sum_bytes(1),
              "workspace layout");

// ---- losses ----------------------------------------------------------------------

template <class Loss>
flce_status_t run_grads(const LossArgs<Loss>& a, hipStream_t st) {
  if (a.tiles == 0) return FLCE_OK;
  const int grid = (int)ceil_div(a.tiles, kLossWaves);
  return launch(K_LOSS_GRADS, st, [&] {
    if (a.rows == 1)
      loss_grads_kernel<Loss, 1><<<grid, 64 * kLossWaves, 0, st>>>(a);
    else
      loss_grads_kernel<Loss, kLossRows><<<grid, 64 * kLossWaves, 0, st>>>(a);
  });
}

// Forward (parts, sequences) and, with `grads`, the gradients. The workspace
// regions of `a` are set here; a.state is the caller's, or null.
template <class Loss>
flce_status_t run_loss(LossArgs<Loss>& a, const LossPlan& p, bool grads, void* workspace,
                       hipStream_t st) {
  a.tiles = p.tiles;
  a.rows = p.rows;
  a.parts = reinterpret_cast<typename Loss::Share*>(wsp(workspace, p.parts));
  a.seq_sum = reinterpret_cast<typename Loss::Share*>(wsp(workspace, p.seq_sum));
  a.totals = reinterpret_cast<typename Loss::Total*>(wsp(workspace, p.totals));
  a.header = reinterpret_cast<int32_t*>(workspace);
  if (p.small) {
    return launch(K_LOSS_SMALL, st, [&] {
      if (grads)
        loss_small_kernel<Loss, true><<<1, 64 * kSmallWaves, 0, st>>>(a);
      else
        loss_small_kernel<Loss, false><<<1, 64 * kSmallWaves, 0, st>>>(a);
    });
  }
  if (a.state == nullptr) a.state = reinterpret_cast<double*>(wsp(workspace, p.state));
  // What the sequences kernel's blocks found is added up by the gradients kernel if
  // there is one and a lane a block suffices.
  a.deferred = grads && a.tiles > 0 && p.seq_blocks > 1 && p.seq_blocks <= 64 ? p.seq_blocks : 0;
  // At least one block, which readies the header for the next kernel.
  const int grid = (int)ceil_div(a.tiles > 0 ? a.tiles : 1, kLossWaves);
  FLCE_TRY(launch(K_LOSS_PARTS, st, [&] {
    if (a.rows == 1)
      loss_parts_kernel<Loss, 1><<<grid, 64 * kLossWaves, 0, st>>>(a);
    else
      loss_parts_kernel<Loss, kLossRows><<<grid, 64 * kLossWaves, 0, st>>>(a);
  }));
  FLCE_TRY(launch(K_LOSS_SEQUENCES, st, [&] {
    loss_sequences_kernel<Loss><<<p.seq_blocks, kSeqThreads, 0, st>>>(a, p.seq_items);
  }));
  return grads ? run_grads(a, st) : FLCE_OK;
}

LossArgs<PolicyLoss> policy_args(const float* logprob, const float* entropy,
                                 const float* old_logprob, const float* ref_logprob,
                                 const float* advantages, const int64_t* labels,
                                 const int64_t* cu, int64_t N, int64_t B, int64_t V,
                                 const flce_policy_options_t& o) {
  const double inf = std::numeric_limits<double>::infinity();
  LossArgs<PolicyLoss> a{};
  a.in.logprob = logprob;
  a.in.old_logprob = old_logprob;
  a.in.ref_logprob = ref_logprob;
  a.in.entropy = entropy;
  a.in.advantages = advantages;
  a.in.over = 1.0 + o.clip_high;
  a.in.under = 1.0 - o.clip_low;
  a.in.dual = o.dual_clip;
  a.in.log_over = std::log1p(o.clip_high);
  a.in.log_under = o.clip_low < 1.0 ? std::log1p(-o.clip_low) : -inf;
  a.in.log_dual = o.dual_clip > 0.0 ? std::log(o.dual_clip) : inf;
  a.in.kl_coef = o.kl_coef;
  a.in.ent_coef = o.entropy_coef;
  a.in.kl = o.kl_estimator;
  a.in.by_sequence = o.level == FLCE_RATIO_SEQUENCE ? 1 : 0;
  a.in.adv_seq = o.advantages_per_sequence;
  a.in.reduction = o.reduction;
  a.labels = labels;
  a.cu = cu;
  a.N = N;
  a.B = B;
  a.V = V;
  a.ignore_index = o.ignore_index;
  a.items = B;
  return a;
}

// The pointers that every policy call reads.
flce_status_t check_policy_inputs(const float* logprob, const float* old_logprob,
                                  const float* ref_logprob, const float* advantages,
                                  const int64_t* labels, const int64_t* cu, int64_t N,
                                  const flce_policy_options_t& o) {
  if (N > 0 && (logprob == nullptr || old_logprob == nullptr || labels == nullptr))
    return FLCE_ERR_NULL_POINTER;
  if (advantages == nullptr && (N > 0 || o.advantages_per_sequence != 0))
    return FLCE_ERR_NULL_POINTER;
  if (o.kl_coef != 0.0 && N > 0 && ref_logprob == nullptr) return FLCE_ERR_NULL_POINTER;
  if (!aligned_to(logprob, 4) || !aligned_to(old_logprob, 4) || !aligned_to(ref_logprob, 4) ||
      !aligned_to(advantages, 4) || !aligned_to(labels, 8) || !aligned_to(cu, 8))
    return FLCE_ERR_MISALIGNED;
  return FLCE_OK;
}

// Forward, with gradients when grad_logprob is set; state null: the workspace's.
flce_status_t policy_impl(const float* logprob, const float* entropy, const float* old_logprob,
                          const float* ref_logprob, const float* advantages,
                          const int64_t* labels, const int64_t* cu, int64_t N, int64_t B,
                          int64_t V, const flce_policy_options_t* opt, const float* grad_loss,
                          float* loss, float* stats, double* state, bool grads, float* grad_logprob,
                          float* grad_entropy, void* workspace, size_t workspace_bytes,
                          void* stream) {
  FLCE_TRY(check_policy(N, B, V, cu != nullptr, opt));
  FLCE_TRY(check_policy_inputs(logprob, old_logprob, ref_logprob, advantages, labels, cu, N, *opt));
  if (stats == nullptr || workspace == nullptr) return FLCE_ERR_NULL_POINTER;
  if (opt->entropy_coef != 0.0 && N > 0 && entropy == nullptr) return FLCE_ERR_NULL_POINTER;
  if (grads && N > 0 && grad_logprob == nullptr) return FLCE_ERR_NULL_POINTER;
  if (!aligned_to(entropy, 4) || !aligned_to(loss, 4) || !aligned_to(stats, 4) ||
      !aligned_to(state, 8) || !aligned_to(grad_loss, 4) || !aligned_to(grad_logprob, 4) ||
      !aligned_to(grad_entropy, 4) || !aligned16(workspace))
    return FLCE_ERR_MISALIGNED;
  const LossPlan p = policy_plan(N, B);
  if (workspace_bytes < p.total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  LossArgs<PolicyLoss> a = policy_args(logprob, entropy, old_logprob, ref_logprob, advantages,
                                       labels, cu, N, B, V, *opt);
  a.out.loss = loss;
  a.out.stats = stats;
  a.out.grad_loss = grad_loss;
  a.out.grad_logprob = grad_logprob;
  a.out.grad_entropy = grad_entropy;
  a.state = state;
  return run_loss(a, p, grads, workspace, static_cast<hipStream_t>(stream));
}

LossArgs<PreferenceLoss> preference_args(const float* logprob, const float* ref_logprob,
                                         const int64_t* labels, const int64_t* cu, int64_t N,
                                         int64_t P, int64_t V,
                                         const flce_preference_options_t& o) {
  LossArgs<PreferenceLoss> a{};
  a.in.logprob = logprob;
  a.in.ref_logprob = ref_logprob;
  a.in.beta = o.beta;
  a.in.eps = o.label_smoothing;
  a.in.margin = o.margin;
  a.in.half_inv_beta = 0.5 / o.beta;
  a.in.kind = o.kind;
  a.in.normalize = o.length_normalize;
  a.in.reduction = o.reduction;
  a.labels = labels;
  a.cu = cu;
  a.N = N;
  a.B = 2 * P;
  a.V = V;
  a.ignore_index = o.ignore_index;
  a.items = P;
  return a;
}

flce_status_t preference_impl(const float* logprob, const float* ref_logprob,
                              const int64_t* labels, const int64_t* cu, int64_t N, int64_t P,
                              int64_t V, const flce_preference_options_t* opt,
                              const float* grad_loss, float* loss, float* pair_loss,
                              float* chosen, float* rejected, double* state, bool grads,
                              float* grad_logprob, void* workspace, size_t workspace_bytes,
                              void* stream) {
  FLCE_TRY(check_preference(N, P, V, opt));
  if (cu == nullptr || pair_loss == nullptr || chosen == nullptr || rejected == nullptr ||
      workspace == nullptr)
    return FLCE_ERR_NULL_POINTER;
  if (opt->reduction != FLCE_REDUCTION_NONE && loss == nullptr) return FLCE_ERR_NULL_POINTER;
  if (N > 0 && (logprob == nullptr || labels == nullptr)) return FLCE_ERR_NULL_POINTER;
  if (grads && N > 0 && grad_logprob == nullptr) return FLCE_ERR_NULL_POINTER;
  if (!aligned_to(logprob, 4) || !aligned_to(ref_logprob, 4) || !aligned_to(labels, 8) ||
      !aligned_to(cu, 8) || !aligned_to(grad_loss, 4) || !aligned_to(loss, 4) ||
      !aligned_to(pair_loss, 4) || !aligned_to(chosen, 4) || !aligned_to(rejected, 4) ||
      !aligned_to(state, 8) || !aligned_to(grad_logprob, 4) || !aligned16(workspace))
    return FLCE_ERR_MISALIGNED;
  const LossPlan p = preference_plan(N, P);
  if (workspace_bytes < p.total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  LossArgs<PreferenceLoss> a = preference_args(logprob, ref_logprob, labels, cu, N, P, V, *opt);
  a.out.loss = loss;
  a.out.pair_loss = pair_loss;
  a.out.chosen = chosen;
  a.out.rejected = rejected;
  a.out.grad_loss = grad_loss;
  a.out.grad_logprob = grad_logprob;
  a.state = state;
  return run_loss(a, p, grads, workspace, static_cast<hipStream_t>(stream));
}

// ---- embedding --------------------------------------------------------------------

TokenArgs token_args(const int64_t* tokens, int64_t N, int64_t Vs, int64_t v_begin,
                     int64_t V_total, int64_t ignore_index, void* workspace) {
  TokenArgs t{};
  t.tokens = tokens;
  t.N = N;
  t.Vs = Vs;
  t.v_begin = v_begin;
  t.V_total = V_total;
  t.ignore_index = ignore_index;
  t.header = reinterpret_cast<int32_t*>(workspace);
  return t;
}

flce_status_t clear_header(const TokenArgs& t, hipStream_t st) {
  return launch(K_FILL, st, [&] { embed_clear_kernel<<<1, 64, 0, st>>>(t.header); });
}

// Sorts the tokens to (key, perm) in the workspace and fills the header.
flce_status_t sort_tokens(const TokenArgs& t, const EmbedPlan& p, void* ws, int32_t** key,
                          int32_t** perm, hipStream_t st) {
  int32_t* k1 = reinterpret_cast<int32_t*>(wsp(ws, p.key));
  int32_t* p1 = reinterpret_cast<int32_t*>(wsp(ws, p.perm));
  const SortPlan& s = p.sort;
  *key = k1;
  *perm = p1;
  if (s.by_rank) {
    // Without a token one block still writes the header.
    const int64_t groups = ceil_div(t.N, kRankItems);
    const size_t lds = 4 * (size_t)groups * kRankItems;
    return launch(K_EMBED_SORT, st, [&] {
      embed_rank_kernel<<<(unsigned)(groups > 0 ? groups : 1), kRankThreads, lds, st>>>(t, k1, p1);
    });
  }
  int32_t* k2 = reinterpret_cast<int32_t*>(wsp(ws, p.key2));
  int32_t* p2 = reinterpret_cast<int32_t*>(wsp(ws, p.perm2));
  int32_t* totals = reinterpret_cast<int32_t*>(wsp(ws, p.totals));
  FLCE_TRY(clear_header(t, st));
  const int nd = 1 << s.bits;
  SortArgs a{};
  a.t = t;
  a.counts = reinterpret_cast<int32_t*>(wsp(ws, p.counts));
  a.pitch = s.pitch;
  a.bits = s.bits;
  for (int pass = 0; pass < s.passes; ++pass) {
    a.shift = pass * s.bits;
    a.key_in = pass == 0 ? nullptr : *key;
    a.perm_in = pass == 0 ? nullptr : *perm;
    a.key_out = (pass & 1) == 0 ? k1 : k2;
    a.perm_out = (pass & 1) == 0 ? p1 : p2;
    FLCE_TRY(launch(K_EMBED_SORT, st, [&] {
      embed_sort_count_kernel<<<(int)s.tiles, 256, 0, st>>>(a);
    }));
    FLCE_TRY(launch(K_EMBED_SORT, st, [&] {
      embed_sort_scan_kernel<<<(nd + 3) / 4, 256, 0, st>>>(a.counts, s.tiles, s.pitch, nd,
                                                           totals);
    }));
    FLCE_TRY(launch(K_EMBED_SORT, st, [&] {
      embed_sort_move_kernel<<<(int)s.tiles, 64 * kSortMoveWaves, 0, st>>>(a, totals);
    }));
    *key = a.key_out;
    *perm = a.perm_out;
  }
  return FLCE_OK;
}

// Lanes that share a row of H values, eight each.
int row_lanes(int64_t H) {
  int t = 8;
  while (t < 64 && (int64_t)t * 8 < H) t <<= 1;
  return t;
}

// Hidden values a block of the gradient takes, of `unit` at a time: all of them, or
// as few as it takes to give every CU four blocks.
int64_t grad_range(int64_t H, int64_t unit, int64_t blocks) {
  const int64_t units = ceil_div(H, unit);
  int64_t parts = ceil_div(4 * kNumCUs, blocks);
  if (parts > units) parts = units;
  return ceil_div(units, parts) * unit;
}

template <bool HF32, bool GF32, bool ACC>
void launch_grad(GradArgs a, int layout, hipStream_t st) {
  if (layout == FLCE_EMBED_VH) {
    const int64_t blocks = ceil_div(a.Vs, kGradRows);
    a.range = grad_range(a.H, (int64_t)a.lanes * (GF32 ? 4 : 8), blocks);
    const dim3 grid((unsigned)blocks, (unsigned)ceil_div(a.H, a.range));
    embed_grad_rows_kernel<HF32, GF32, ACC><<<grid, 256, 0, st>>>(a);
    return;
  }
  const dim3 grid((unsigned)ceil_div(a.Vs, kStrip), (unsigned)ceil_div(a.H, kStripH));
  if (a.Vs % 8 == 0)
    embed_grad_cols_kernel<HF32, GF32, ACC, true><<<grid, 256, 0, st>>>(a);
  else
    embed_grad_cols_kernel<HF32, GF32, ACC, false><<<grid, 256, 0, st>>>(a);
}

}  // namespace

extern "C" {

// ---- embedding --------------------------------------------------------------------

flce_status_t flce_embedding_workspace_size(int64_t N, int64_t H, int64_t Vs,
                                            const flce_embedding_options_t* opt, size_t* fwd_bytes,
                                            size_t* bwd_bytes) {
  FLCE_TRY(check_embedding(N, H, Vs, 0, Vs, opt));
  const EmbedPlan p = make_embed_plan(N, H, Vs, opt->layout);
  if (fwd_bytes) *fwd_bytes = p.f_total;
  if (bwd_bytes) *bwd_bytes = p.b_total;
  return FLCE_OK;
}

flce_status_t flce_embedding_forward(const void* weight, const int64_t* tokens, int64_t N,
                                     int64_t H, int64_t Vs, int64_t v_begin, int64_t V_total,
                                     const flce_embedding_options_t* opt, void* hidden,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  FLCE_TRY(check_embedding(N, H, Vs, v_begin, V_total, opt));
  if (workspace == nullptr) return FLCE_ERR_NULL_POINTER;
  if (N > 0 && (weight == nullptr || tokens == nullptr || hidden == nullptr))
    return FLCE_ERR_NULL_POINTER;
  if (!aligned16(weight) || !aligned16(hidden) || !aligned16(workspace) || !aligned_to(tokens, 8))
    return FLCE_ERR_MISALIGNED;
  const EmbedPlan p = make_embed_plan(N, H, Vs, opt->layout);
  if (workspace_bytes < p.f_total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  GatherArgs a{};
  a.t = token_args(tokens, N, Vs, v_begin, V_total, opt->ignore_index, workspace);
  if (N == 0) return clear_header(a.t, st);
  a.weight = static_cast<const uint16_t*>(weight);
  a.H = H;
  a.scale = (float)opt->scale;
  a.out = static_cast<uint16_t*>(hidden);
  if (opt->layout == FLCE_EMBED_HV) {
    if (p.sorted) {
      int32_t *key, *perm;
      FLCE_TRY(sort_tokens(a.t, p, workspace, &key, &perm, st));
      a.key = key;
      a.perm = perm;
    } else {
      a.count_block = 1;  // eight more blocks, the first of which counts
    }
    const int64_t blocks = ceil_div(N, kGatherTokens) + a.count_block;
    const dim3 grid((unsigned)(8 * blocks), (unsigned)ceil_div(H, 64 * 8));
    return launch(K_EMBED_GATHER, st, [&] { embed_gather_cols_kernel<<<grid, 256, 0, st>>>(a); });
  }
  // One more block, the first, counts the invalid tokens beside the copy, which takes
  // longer while the batch is small or the rows are long; otherwise every wave
  // counts its own into a cleared header, a launch more (4 us).
  a.count_block = N <= kCountBlockTokens || H >= kCountBlockHidden ? 1 : 0;
  if (a.count_block == 0) FLCE_TRY(clear_header(a.t, st));
  a.lanes = row_lanes(H);
  const dim3 grid((unsigned)(ceil_div(N, 4 * (64 / a.lanes)) + a.count_block),
                  (unsigned)ceil_div(H, (int64_t)a.lanes * 8 * kGatherLoads));
  return launch(K_EMBED_GATHER, st, [&] { embed_gather_rows_kernel<<<grid, 256, 0, st>>>(a); });
}

flce_status_t flce_embedding_backward(const void* grad_hidden, const int64_t* tokens, int64_t N,
                                      int64_t H, int64_t Vs, int64_t v_begin, int64_t V_total,
                                      const flce_embedding_options_t* opt, void* grad_weight,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  FLCE_TRY(check_embedding(N, H, Vs, v_begin, V_total, opt));
  if (workspace == nullptr || grad_weight == nullptr) return FLCE_ERR_NULL_POINTER;
  if (N > 0 && (grad_hidden == nullptr || tokens == nullptr)) return FLCE_ERR_NULL_POINTER;
  if (!aligned16(grad_hidden) || !aligned16(grad_weight) || !aligned16(workspace) ||
      !aligned_to(tokens, 8))
    return FLCE_ERR_MISALIGNED;
  const EmbedPlan p = make_embed_plan(N, H, Vs, opt->layout);
  if (workspace_bytes < p.b_total) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const TokenArgs t = token_args(tokens, N, Vs, v_begin, V_total, opt->ignore_index, workspace);
  int32_t* strips = reinterpret_cast<int32_t*>(wsp(workspace, p.strips));
  int32_t *key, *perm;
  FLCE_TRY(sort_tokens(t, p, workspace, &key, &perm, st));
  GradArgs a{};
  a.grad = grad_hidden;
  a.key = key;
  a.perm = perm;
  a.header = t.header;
  a.strips = strips;
  a.part = reinterpret_cast<float*>(wsp(workspace, p.part));
  a.N = N;
  a.H = H;
  a.Vs = Vs;
  a.scale = (float)opt->scale;
  a.out = grad_weight;
  a.lanes = row_lanes(H);
  const bool hf = opt->hidden_dtype == FLCE_GRAD_F32, gf = opt->grad_dtype == FLCE_GRAD_F32;
  const bool acc = opt->accumulate != 0;
  const int threads = H <= 256 ? 64 : (H <= 512 ? 128 : 256);
  a.strip_blocks = (int)ceil_div(ceil_div(Vs, kStrip) + 1, threads);
  a.chunks = (int)ceil_div(H, (int64_t)threads * 4);
  const int64_t blocks = a.strip_blocks + ceil_div(N, kPiece) * a.chunks;
  FLCE_TRY(launch(K_EMBED_SEGMENTS, st, [&] {
    if (hf)
      embed_segments_kernel<true><<<(unsigned)blocks, threads, 0, st>>>(a);
    else
      embed_segments_kernel<false><<<(unsigned)blocks, threads, 0, st>>>(a);
  }));
  const int64_t large = p.large_pieces;
  if (large > 0) {
    a.part2 = reinterpret_cast<float*>(wsp(workspace, p.part2));
    FLCE_TRY(launch(K_EMBED_SEGMENTS, st, [&] {
      embed_large_pieces_kernel<<<(unsigned)(large * a.chunks), threads, 0, st>>>(a);
    }));
  }
  return launch(K_EMBED_GRAD, st, [&] {
    switch ((hf ? 4 : 0) + (gf ? 2 : 0) + (acc ? 1 : 0)) {
      case 0: launch_grad<false, false, false>(a, opt->layout, st); break;
      case 1: launch_grad<false, false, true>(a, opt->layout, st); break;
      case 2: launch_grad<false, true, false>(a, opt->layout, st); break;
      case 3: launch_grad<false, true, true>(a, opt->layout, st); break;
      case 4: launch_grad<true, false, false>(a, opt->layout, st); break;
      case 5: launch_grad<true, false, true>(a, opt->layout, st); break;
      case 6: launch_grad<true, true, false>(a, opt->layout, st); break;
      default: launch_grad<true, true, true>(a, opt->layout, st); break;
    }
  });
}

// ---- policy loss --------------------------------------------------------------------

flce_status_t flce_policy_workspace_size(int64_t N, int64_t B, size_t* bytes) {
  if (N < 0 || N > kMaxN || B < 1 || B > kMaxSequences) return FLCE_ERR_BAD_SHAPE;
  if (bytes) *bytes = policy_plan(N, B).total;
  return FLCE_OK;
}

flce_status_t flce_policy_loss_forward(const float* logprob, const float* entropy,
                                       const float* old_logprob, const float* ref_logprob,
                                       const float* advantages, const int64_t* labels,
                                       const int64_t* cu_seqlens, int64_t N, int64_t B, int64_t V,
                                       const flce_policy_options_t* opt, float* loss, float* stats,
                                       double* seq_state, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  if (seq_state == nullptr) return FLCE_ERR_NULL_POINTER;
  return policy_impl(logprob, entropy, old_logprob, ref_logprob, advantages, labels, cu_seqlens,
                     N, B, V, opt, nullptr, loss, stats, seq_state, false, nullptr, nullptr,
                     workspace, workspace_bytes, stream);
}

flce_status_t flce_policy_loss_backward(const float* logprob, const float* old_logprob,
                                        const float* ref_logprob, const float* advantages,
                                        const int64_t* labels, const int64_t* cu_seqlens,
                                        int64_t N, int64_t B, int64_t V,
                                        const flce_policy_options_t* opt, const double* seq_state,
                                        const float* grad_loss, float* grad_logprob,
                                        float* grad_entropy, void* stream) {
  FLCE_TRY(check_policy(N, B, V, cu_seqlens != nullptr, opt));
  FLCE_TRY(check_policy_inputs(logprob, old_logprob, ref_logprob, advantages, labels, cu_seqlens,
                               N, *opt));
  if (seq_state == nullptr || (N > 0 && grad_logprob == nullptr)) return FLCE_ERR_NULL_POINTER;
  if (!aligned_to(seq_state, 8) || !aligned_to(grad_loss, 4) || !aligned_to(grad_logprob, 4) ||
      !aligned_to(grad_entropy, 4))
    return FLCE_ERR_MISALIGNED;
  LossArgs<PolicyLoss> a = policy_args(logprob, nullptr, old_logprob, ref_logprob, advantages,
                                       labels, cu_seqlens, N, B, V, *opt);
  const LossPlan p = policy_plan(N, B);
  a.tiles = p.tiles;
  a.rows = p.rows;
  a.state = const_cast<double*>(seq_state);  // read only by the gradients kernel
  a.out.grad_loss = grad_loss;
  a.out.grad_logprob = grad_logprob;
  a.out.grad_entropy = grad_entropy;
  return run_grads(a, static_cast<hipStream_t>(stream));
}

flce_status_t flce_policy_loss_forward_backward(
    const float* logprob, const float* entropy, const float* old_logprob, const float* ref_logprob,
    const float* advantages, const int64_t* labels, const int64_t* cu_seqlens, int64_t N, int64_t B,
    int64_t V, const flce_policy_options_t* opt, const float* grad_loss, float* loss, float* stats,
    float* grad_logprob, float* grad_entropy, void* workspace, size_t workspace_bytes,
    void* stream) {
  return policy_impl(logprob, entropy, old_logprob, ref_logprob, advantages, labels, cu_seqlens,
                     N, B, V, opt, grad_loss, loss, stats, nullptr, true, grad_logprob,
                     grad_entropy, workspace, workspace_bytes, stream);
}

// ---- preference loss ------------------------------------------------------------------

flce_status_t flce_preference_workspace_size(int64_t N, int64_t P, size_t* bytes) {
  if (N < 0 || N > kMaxN || P < 1 || P > kMaxSequences / 2) return FLCE_ERR_BAD_SHAPE;
  if (bytes) *bytes = preference_plan(N, P).total;
  return FLCE_OK;
}

flce_status_t flce_preference_loss_forward(const float* logprob, const float* ref_logprob,
                                           const int64_t* labels, const int64_t* cu_seqlens,
                                           int64_t N, int64_t P, int64_t V,
                                           const flce_preference_options_t* opt, float* loss,
                                           float* pair_loss, float* chosen_reward,
                                           float* rejected_reward, double* seq_state,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  if (seq_state == nullptr) return FLCE_ERR_NULL_POINTER;
  return preference_impl(logprob, ref_logprob, labels, cu_seqlens, N, P, V, opt, nullptr, loss,
                         pair_loss, chosen_reward, rejected_reward, seq_state, false, nullptr,
                         workspace, workspace_bytes, stream);
}

flce_status_t flce_preference_loss_backward(const int64_t* labels, const int64_t* cu_seqlens,
                                            int64_t N, int64_t P, int64_t V,
                                            const flce_preference_options_t* opt,
                                            const double* seq_state, const float* grad_loss,
                                            float* grad_logprob, void* stream) {
  FLCE_TRY(check_preference(N, P, V, opt));
  if (cu_seqlens == nullptr || seq_state == nullptr) return FLCE_ERR_NULL_POINTER;
  if (N > 0 && (labels == nullptr || grad_logprob == nullptr)) return FLCE_ERR_NULL_POINTER;
  if (!aligned_to(labels, 8) || !aligned_to(cu_seqlens, 8) || !aligned_to(seq_state, 8) ||
      !aligned_to(grad_loss, 4) || !aligned_to(grad_logprob, 4))
    return FLCE_ERR_MISALIGNED;
  LossArgs<PreferenceLoss> a =
      preference_args(nullptr, nullptr, labels, cu_seqlens, N, P, V, *opt);
  const LossPlan p = preference_plan(N, P);
  a.tiles = p.tiles;
  a.rows = p.rows;
  a.state = const_cast<double*>(seq_state);  // read only by the gradients kernel
  a.out.grad_loss = grad_loss;
  a.out.grad_logprob = grad_logprob;
  return run_grads(a, static_cast<hipStream_t>(stream));
}

flce_status_t flce_preference_loss_forward_backward(
    const float* logprob, const float* ref_logprob, const int64_t* labels,
    const int64_t* cu_seqlens, int64_t N, int64_t P, int64_t V,
    const flce_preference_options_t* opt, const float* grad_loss, float* loss, float* pair_loss,
    float* chosen_reward, float* rejected_reward, float* grad_logprob, void* workspace,
    size_t workspace_bytes, void* stream) {
  return preference_impl(logprob, ref_logprob, labels, cu_seqlens, N, P, V, opt, grad_loss, loss,
                         pair_loss, chosen_reward, rejected_reward, nullptr, true, grad_logprob,
                         workspace, workspace_bytes, stream);
}

}  // extern "C"
