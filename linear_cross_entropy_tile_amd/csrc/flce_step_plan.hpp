// Host planner of the operators at the two ends of a training step (logits to
// sample from, their processing, the gradients' norm and the AdamW update):
// limits, argument checks, workspace layouts and the split of the work over
// blocks. Host-only C++ without HIP, so that it also builds on its own for
// sanitizer checks.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "flce.h"
#include "flce_layout.hpp"
#include "flce_plan.hpp"

namespace flce {

inline bool at_multiple(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool known_dtype(int d) { return d == FLCE_GRAD_BF16 || d == FLCE_GRAD_F32; }
inline size_t dtype_bytes(int d) { return d == FLCE_GRAD_F32 ? 4 : 2; }

// ---- logits ------------------------------------------------------------------------

constexpr int64_t kMaxLogitRows = 1024;
constexpr int kLogitStrip = 128;     // vocabulary columns a block takes

// How a product is made: `mt` groups of 16 tokens a block of `waves` waves, in `passes`
// over the weight, with the hidden dimension cut in `splits`, whose sums lie in the
// workspace; `wide` waves of 64 tokens a block, in `passes`; or the head's block tiles
// (mt and wide 0), from a blocked copy of hidden.
struct LogitsPlan {
  int wide;
  int mt, waves, passes, splits, split_steps;
  int64_t strips;
  int hkb, vt, tb;
  size_t image, parts, total;
};
inline LogitsPlan make_logits_plan(int64_t N, int64_t H, int64_t V) {
  LogitsPlan p{};
  p.image = kHeaderBytes;
  p.total = kHeaderBytes;
  if (N == 0) return p;
  p.strips = ceil_div(V, kLogitStrip);
  // More than 64 tokens: larger tiles, unless the product gives the smaller ones less than
  // 256 blocks, which then share out the hidden dimension too and are faster (H 4096, tiles
  // and then small ones: 1000 ids x 128 tokens 81 and 18 us, 5000 x 256 86 and 31 us). With
  // more blocks it depends on how full the tiles are: 20000 x 128, half of each empty, 92
  // and 83 us, 20000 x 256 99 and 107, 50264 x 200 127 and 222. All of them take tiles.
  const bool large = N > 64 && p.strips * ceil_div(N, 64) >= 256;
  if (large && V % 8 == 0) {
    p.hkb = (int)ceil_div(H, kBK);
    p.vt = (int)ceil_div(V, kTile);
    p.tb = (int)ceil_div(N, kTile);
    p.total = align_up(kHeaderBytes + (size_t)p.tb * (size_t)p.hkb * kBlockBytes);
    return p;
  }
  // The tiles' reads of the weight want aligned rows; of the others, 128 or 256 tokens at
  // once (H 4096, 50257 ids x 200 tokens: 192 us, with 64 at once 263 us).
  if (large && V >= kLogitStrip) {
    p.wide = N <= 128 ? 2 : 4;
    p.passes = (int)ceil_div(N, 64 * p.wide);
    return p;
  }
  p.mt = N <= 16 ? 1 : (N <= 32 ? 2 : 4);
  p.passes = (int)ceil_div(N, 16 * p.mt);
  // Few strips: more waves a strip, as the registers allow, and the hidden dimension
  // cut over blocks, so that the GPU's CUs have a block each and enough loads are in
  // flight.
  const int64_t steps = ceil_div(H, 32), blocks = p.strips * p.passes;
  p.waves = 4;
  p.splits = 1;
  if (blocks < 512) {
    p.waves = p.mt == 4 || steps < 16 ? 4 : (p.mt == 1 && steps >= 32 ? 16 : 8);
    if (blocks < 192) {
      if (p.waves > 8) p.waves = 8;
      const int64_t most = steps / (2 * p.waves), want = ceil_div(384, blocks);
      p.splits = (int)(want < most ? want : (most > 0 ? most : 1));
    }
  }
  p.split_steps = (int)ceil_div(steps, p.splits);
  p.splits = (int)ceil_div(steps, p.split_steps);
  if (p.splits > 1) {
    p.parts = kHeaderBytes;
    p.total = align_up(kHeaderBytes + 4 * (size_t)p.splits * (size_t)N * (size_t)V);
  }
  return p;
}

inline flce_status_t check_logits(int64_t N, int64_t H, int64_t V, float softcap, int out_dtype,
                                  int64_t ld_out) {
  if (N < 0 || N > kMaxLogitRows) return FLCE_ERR_BAD_SHAPE;
  const flce_status_t s = check_shape(N, H, V);
  if (s != FLCE_OK) return s;
  if (ld_out < V || ld_out > ((int64_t)1 << 40)) return FLCE_ERR_BAD_SHAPE;
  if (!std::isfinite(softcap) || (softcap > 0.f && !std::isfinite(1.f / softcap)))
    return FLCE_ERR_BAD_SOFTCAP;
  if (!known_dtype(out_dtype)) return FLCE_ERR_BAD_OPTION;
  return FLCE_OK;
}

// ---- processing of logits ----------------------------------------------------------

constexpr int kProcThreads = 256;
constexpr int kProcStep = 8 * kProcThreads;  // ids a block takes at once, eight a thread

// What a row's history is kept as while a slice of its ids is processed.
enum { HIST_NONE = 0, HIST_SEEN = 1, HIST_COUNT = 2 };

struct ProcPlan {
  int slice;             // ids a block takes, a multiple of kProcStep
  int64_t slices;        // blocks a row
  size_t parts, invalid, total;
};

// Steps of a slice: two, or one where that leaves the GPU less than 1024 blocks (four a
// CU). Four (half the readings of a row's history, but twice the registers) are no
// faster: 512 rows of 152064 bf16 logits with histories of 1000 to 2048 tokens take 89
// us with either.
constexpr int kProcSteps = 2;
inline int proc_steps(int64_t N, int64_t V) {
  return N * ceil_div(V, (int64_t)kProcSteps * kProcStep) < 1024 ? 1 : kProcSteps;
}

// Workspace: header, the softmax state and first largest id of every slice
// [N, slices], the invalid tokens of every row [N].
inline ProcPlan make_proc_plan(int64_t N, int64_t V) {
  ProcPlan p{};
  p.slice = proc_steps(N, V) * kProcStep;
  p.slices = ceil_div(V, p.slice);
  size_t off = kHeaderBytes;
  p.parts = off;
  off = align_up(off + 16 * (size_t)N * (size_t)p.slices);
  p.invalid = off;
  off = align_up(off + 4 * (size_t)N);
  p.total = off;
  return p;
}

inline bool proc_penalised(const flce_process_options_t& o) {
  return o.repetition != nullptr || o.presence != nullptr || o.frequency != nullptr ||
         o.repetition_penalty != 1.0 || o.presence_penalty != 0.0 || o.frequency_penalty != 0.0;
}
inline int proc_history(const flce_process_options_t& o, bool gradient) {
  if (o.tokens == nullptr) return HIST_NONE;
  const bool count = o.presence != nullptr || o.frequency != nullptr ||
                     o.presence_penalty != 0.0 || o.frequency_penalty != 0.0;
  if (!gradient && count) return HIST_COUNT;
  return o.repetition != nullptr || o.repetition_penalty != 1.0 ? HIST_SEEN : HIST_NONE;
}

// Rows of longer histories are counted in 32 bits, of which one is the prompt's; those that
// are longer than a count are refused.
constexpr int64_t kLongHistory = 0x7FFF, kMostHistory = 0x7FFFFFFF;
// Words by which ids of one listed bias wait for each other.
constexpr int kProcTags = 256;
// LDS words of a slice: counts, then in their place sums of the listed biases; tags.
constexpr int proc_count_words(int hist, int slice) {
  return hist == HIST_COUNT ? slice / 2 : (hist == HIST_SEEN ? slice / 32 : 0);
}
constexpr int proc_lds_words(int hist, bool list, int slice) {
  return list ? slice + kProcTags : proc_count_words(hist, slice);
}

// A token's distance from id lo: its place among the n ids from there on if it is below
// n. Any int64 may be a token; those before lo are far past every n.
constexpr uint64_t proc_place(int64_t token, int64_t lo) {
  return (uint64_t)token - (uint64_t)lo;
}
// A slice of n ids whose counts take 32 bits is counted in parts of `part` ids: the ids
// of the one from `from` on, none where the slice ends before it.
constexpr uint32_t proc_part(int n, int from, int part) {
  return (uint32_t)(n <= from ? 0 : (n - from < part ? n - from : part));
}

// Above 0, and in fp32 still so and finite, as its reciprocal there is.
inline bool fp32_divisor(double x) {
  const float f = (float)x;
  return f > 0.f && std::isfinite(f) && std::isfinite(1.f / f);
}
inline flce_status_t check_process(int64_t N, int64_t V, const flce_process_options_t* o) {
  if (N < 0 || N > kMaxN || V < 1 || V > kMaxV) return FLCE_ERR_BAD_SHAPE;
  if (o == nullptr) return FLCE_ERR_NULL_POINTER;
  if (!known_dtype(o->logits_dtype) || !known_dtype(o->out_dtype)) return FLCE_ERR_BAD_OPTION;
  if (!fp32_divisor(o->repetition_penalty) || !std::isfinite(o->presence_penalty) ||
      !std::isfinite(o->frequency_penalty) ||
      !(o->temperature == 0.0 || fp32_divisor(o->temperature)))
    return FLCE_ERR_BAD_OPTION;
  const int64_t most = (int64_t)1 << 40;
  if (o->tokens_size < 0 || o->tokens_size > most || o->tokens_stride < 0 ||
      o->tokens_stride > most || o->bias_stride < 0 || o->bias_stride > most ||
      o->allowed_stride < 0 || o->allowed_stride > most || o->bias_count < 0 ||
      o->bias_count > most)
    return FLCE_ERR_BAD_SHAPE;
  if (o->bias_stride != 0 && o->bias_stride < V) return FLCE_ERR_BAD_SHAPE;
  if (o->allowed_stride != 0 && o->allowed_stride < ceil_div(V, 32)) return FLCE_ERR_BAD_SHAPE;
  // Rows of a padded history lie inside it.
  if (N > 0 && o->tokens_stride > 0 && o->tokens_stride > o->tokens_size / N)
    return FLCE_ERR_BAD_SHAPE;
  if (N > 0 && o->tokens != nullptr && o->offsets == nullptr) return FLCE_ERR_NULL_POINTER;
  if (N > 0 && proc_penalised(*o) && o->tokens_size > 0 && o->tokens == nullptr)
    return FLCE_ERR_NULL_POINTER;
  if (N > 0 && (o->bias_tokens != nullptr || o->bias_values != nullptr ||
                o->bias_offsets != nullptr) &&
      (o->bias_offsets == nullptr ||
       (o->bias_count > 0 && (o->bias_tokens == nullptr || o->bias_values == nullptr))))
    return FLCE_ERR_NULL_POINTER;
  if (!at_multiple(o->tokens, 8) || !at_multiple(o->offsets, 8) ||
      !at_multiple(o->prompt_lengths, 8) || !at_multiple(o->repetition, 4) ||
      !at_multiple(o->presence, 4) || !at_multiple(o->frequency, 4) ||
      !at_multiple(o->temperatures, 4) || !at_multiple(o->bias, 4) ||
      !at_multiple(o->bias_tokens, 8) || !at_multiple(o->bias_values, 4) ||
      !at_multiple(o->bias_offsets, 8) || !at_multiple(o->allowed, 4))
    return FLCE_ERR_MISALIGNED;
  return FLCE_OK;
}

// ---- norm of the gradients, AdamW ----------------------------------------------------

// A launch's grid counts threads in 32 bits: 2^23 blocks of 256 at most here. That
// many blocks take the largest tensor, more than the GPU's memory holds with states.
constexpr int64_t kMaxGrid = (int64_t)1 << 23;
constexpr int64_t kMaxTensorSize = (int64_t)1 << 35;
constexpr int64_t kMaxTensors = (int64_t)1 << 20;

// Values a block of the norm takes: enough for 4096 blocks over all tensors or, in
// small sets, one step of its threads.
constexpr int kNormThreads = 256;
constexpr int64_t kNormStep = 16 * kNormThreads;
constexpr int kNormTensors = 96;       // tensors a launch, whose table is a kernel argument
inline int64_t norm_chunk(int64_t values) {
  return ceil_div(ceil_div(values, 4096), kNormStep) * kNormStep;
}

struct NormPlan {
  int64_t chunk, blocks;
  size_t parts, total;
};
inline flce_status_t make_norm_plan(const int64_t* sizes, int64_t count, NormPlan* p) {
  if (count < 0 || count > kMaxTensors) return FLCE_ERR_BAD_SHAPE;
  if (count > 0 && sizes == nullptr) return FLCE_ERR_NULL_POINTER;
  int64_t values = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] < 0 || sizes[i] > kMaxTensorSize) return FLCE_ERR_BAD_SHAPE;
    values += sizes[i];  // at most 2^55
  }
  p->chunk = values > 0 ? norm_chunk(values) : kNormStep;
  p->blocks = 0;
  for (int64_t i = 0; i < count; ++i) p->blocks += ceil_div(sizes[i], p->chunk);
  p->parts = kHeaderBytes;
  p->total = align_up(kHeaderBytes + 8 * (size_t)p->blocks);
  return FLCE_OK;
}

constexpr int kStateBlock = 256;       // values that share a scale in 8-bit states
constexpr int kAdamThreads = 256;
constexpr int64_t kAdamChunk = 16 * kAdamThreads;  // values a block takes
static_assert(kMaxTensorSize / kAdamChunk <= kMaxGrid, "blocks of a tensor");
constexpr int kAdamTensors = 48;       // tensors a launch, whose table is a kernel argument

inline flce_status_t check_adamw(const flce_adamw_list_t* list, const flce_adamw_options_t* o) {
  if (list == nullptr || o == nullptr) return FLCE_ERR_NULL_POINTER;
  const flce_adamw_list_t& l = *list;
  if (l.count < 0 || l.count > kMaxTensors) return FLCE_ERR_BAD_SHAPE;
  const bool eight = o->state_dtype == FLCE_STATE_8BIT;
  if (l.count > 0 && (l.sizes == nullptr || l.params == nullptr || l.grads == nullptr ||
                      l.exp_avgs == nullptr || l.exp_avg_sqs == nullptr ||
                      l.param_dtypes == nullptr || l.grad_dtypes == nullptr ||
                      (eight && (l.exp_avg_scales == nullptr || l.exp_avg_sq_scales == nullptr))))
    return FLCE_ERR_NULL_POINTER;
  if (!std::isfinite(o->lr) || !std::isfinite((float)o->lr) ||
      !(o->beta1 >= 0.0 && o->beta1 < 1.0) || !(o->beta2 >= 0.0 && o->beta2 < 1.0) ||
      !(o->eps >= 0.0 && std::isfinite((float)o->eps)) ||
      // The quotient's hardware reciprocal takes a denormal for 0.
      (o->eps > 0.0 && (float)o->eps < 0x1p-126f) ||
      !std::isfinite(o->weight_decay) || !std::isfinite((float)(o->lr * o->weight_decay)))
    return FLCE_ERR_BAD_OPTION;
  if (!eight && o->state_dtype != FLCE_STATE_F32) return FLCE_ERR_BAD_OPTION;
  if (o->rounding != FLCE_ROUND_NEAREST && o->rounding != FLCE_ROUND_STOCHASTIC)
    return FLCE_ERR_BAD_OPTION;
  const size_t state = eight ? 1 : 4;
  for (int64_t i = 0; i < l.count; ++i) {
    const int64_t n = l.sizes[i];
    if (n < 0 || n > kMaxTensorSize) return FLCE_ERR_BAD_SHAPE;
    const int p = l.param_dtypes[i], g = l.grad_dtypes[i];
    if (!known_dtype(p) || !known_dtype(g)) return FLCE_ERR_BAD_OPTION;
    const void* master = l.masters != nullptr ? l.masters[i] : nullptr;
    // A copy in fp32 of fp32 weights would be a second set of the same values.
    if (master != nullptr && p != FLCE_GRAD_BF16) return FLCE_ERR_BAD_OPTION;
    if (n == 0) continue;
    if (l.params[i] == nullptr || l.grads[i] == nullptr || l.exp_avgs[i] == nullptr ||
        l.exp_avg_sqs[i] == nullptr)
      return FLCE_ERR_NULL_POINTER;
    if (!at_multiple(l.params[i], dtype_bytes(p)) || !at_multiple(l.grads[i], dtype_bytes(g)) ||
        !at_multiple(master, 4) || !at_multiple(l.exp_avgs[i], state) ||
        !at_multiple(l.exp_avg_sqs[i], state))
      return FLCE_ERR_MISALIGNED;
    if (!eight) continue;
    if (l.exp_avg_scales[i] == nullptr || l.exp_avg_sq_scales[i] == nullptr)
      return FLCE_ERR_NULL_POINTER;
    if (!at_multiple(l.exp_avg_scales[i], 4) || !at_multiple(l.exp_avg_sq_scales[i], 4))
      return FLCE_ERR_MISALIGNED;
  }
  return FLCE_OK;
}

}  // namespace flce
