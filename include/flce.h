/*
 * flce.h -- fused linear cross-entropy + entropy for the LM output head, on
 * AMD Instinct MI355X (gfx950).
 *
 * What the library computes (all from the pages on fusing the LM head with
 * cross-entropy and entropy):
 *
 *   z   = hidden[N,H] x weight[H,V]                       (logits, never stored)
 *   z'  = c * tanh(z / c) if softcap c > 0, else z          (Gemma2 cap)
 *   lse_i     = log sum_j exp(z'_ij)
 *   logprob_i = z'_{i,y_i} - lse_i                          (minus the cross-entropy)
 *   entropy_i = lse_i - sum_j p_ij z'_ij,  p_ij = exp(z'_ij - lse_i)
 *
 * and the gradients of  sum_i gbar_i logprob_i + ebar_i entropy_i  with respect
 * to hidden and weight. The extended entry points (flce_forward_ex,
 * flce_backward_ex) add two per-token outputs with their gradients:
 *
 *   uniform_ce_i = lse_i - (1/V) sum_j z'_ij    (cross-entropy against the uniform
 *                                                distribution: with weight eps,
 *                                                (1-eps)(-logprob) + eps uniform_ce
 *                                                is the label-smoothed cross-entropy)
 *   z_loss_i     = lam * lse_i^2                (z-loss with scale lam)
 *
 * a "sum" reduction, and fp32 gradient outputs. flce_forward_backward
 * returns the outputs and the gradients of one batch in a single call when
 * the upstream gradients are known in advance (the logit gradient formed from
 * logits kept during the forward, no recompute).
 *
 * Sources: verl pull request #462 (memory-efficient linear_cross_entropy),
 * sections "Equivalent compute logic" (the definition above, and that logprobs
 * are the negated cross-entropy) and "API" (hidden is [num_tokens,
 * hidden_size], weight is [hidden_size, vocab_size], labels are integer token
 * ids, a `reduction` argument); Liger-Kernel pull request #551 "[Verl] Add
 * entropy loss to cross_entropy_loss and fused_linear_cross_entropy_loss"
 * (Summary: both outputs without materialising the logits; review thread: the
 * mean divides by the number of non-ignored tokens); Liger-Kernel pull
 * request #435 "Fix LigerCrossEntropyLoss Reduction Behavior for 'None' Mode"
 * (Summary: reduction "none" returns the per-example vector; "Why we pass
 * gradient to output.backward()": a per-element upstream gradient for
 * non-scalar outputs); Liger-Kernel issue #127 "[feat] FusedLinearCrossEntropy
 * support for Gemma2" (proposal: an optional softcap applied after the head
 * matmul; discussion: tanh cap, gradients of hidden and weight by the chain
 * rule).
 *
 * The review thread of Liger-Kernel pull request #551 names a fused z-loss,
 * label smoothing and a sum reduction among the options of such a head,
 * without formulas; the definitions above are the usual ones (the smoothed
 * cross-entropy as torch.nn.functional.cross_entropy defines label_smoothing).
 *
 * Readings where those pages are silent:
 *   - A token whose label equals ignore_index gets every per-token output 0
 *     and no gradient, and is not counted by the mean.
 *   - reduction MEAN reduces each output over the n non-ignored tokens (n = 0
 *     gives 0), SUM sums them; the per-token vectors are written under every
 *     reduction.
 *   - A label that is neither ignore_index nor in [0, V) is treated as ignored
 *     and counted in the workspace status word (see flce_get_status).
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" are HIP device pointers; the caller owns every
 *     buffer, including the workspace. The library allocates no device memory.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream). All
 *     device work is enqueued on it; no call synchronises the device except
 *     flce_get_status and flce_profile_read, which say so.
 *   - Matrices are dense and row-major. bf16 means IEEE bfloat16 bits (uint16).
 *   - Alignment: hidden, weight, grad_hidden, grad_weight and the workspace
 *     must be 16-byte aligned, and H must be a multiple of 8
 *     (FLCE_ERR_MISALIGNED otherwise). V may take any value; when it is not a
 *     multiple of 8 the weight is read from a copy with 16-byte aligned rows
 *     and dW is formed in a buffer of that row stride and copied out (both in
 *     the workspace; flce_workspace_size and flce_fused_workspace_size count
 *     them). N, H and V need no other multiple.
 *   - Argument errors are detected on the host before anything is enqueued;
 *     then nothing is launched and no output is touched. A failed launch
 *     returns FLCE_ERR_HIP. No C++ exception crosses this interface.
 *   - Concurrent calls on different streams need distinct workspaces.
 */
#ifndef FLCE_H
#define FLCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FLCE_OK = 0,
  FLCE_ERR_NULL_POINTER = 1,      /* a required pointer is NULL */
  FLCE_ERR_BAD_SHAPE = 2,         /* N < 0, H < 1, V < 1, or a size beyond the limits below */
  FLCE_ERR_BAD_REDUCTION = 3,     /* reduction not one that the call takes */
  FLCE_ERR_MISALIGNED = 4,        /* see "Alignment" above */
  FLCE_ERR_WORKSPACE_TOO_SMALL = 5,
  FLCE_ERR_BAD_SOFTCAP = 6,       /* softcap is NaN or infinite */
  FLCE_ERR_HIP = 7,               /* a HIP runtime call or kernel launch failed */
  FLCE_ERR_INVALID_LABEL = 8,     /* reported only by flce_get_status */
  FLCE_ERR_BAD_OPTION = 9,        /* z_loss_scale negative or not finite, unknown grad_dtype,
                                   * class_weight under NONE, entropy_per_token not 0 or 1; an
                                   * embedding, policy, preference, process or AdamW option
                                   * outside its range */
  FLCE_ERR_TOO_LARGE = 10         /* flce_forward_noalloc: the shape needs more scratch than
                                   * FLCE_NOALLOC_SCRATCH_BYTES */
} flce_status_t;

enum { FLCE_REDUCTION_NONE = 0, FLCE_REDUCTION_MEAN = 1, FLCE_REDUCTION_SUM = 2 };
enum { FLCE_GRAD_BF16 = 0, FLCE_GRAD_F32 = 1 };

/* Size limits: N <= 2^21, H <= 2^20, V <= 2^22 - 256, and V <= 2^21 with
 * fp32 gradient outputs (FLCE_ERR_BAD_SHAPE beyond). */

/* Workspace bytes needed by the forward (*fwd_bytes) and backward
 * (*bwd_bytes) entry points for this shape and reduction. Host only; either
 * out-pointer may be NULL. The forward size is about 16 * N * ceil(V/256) +
 * 2 * N * H bytes (one partial softmax state per token and 256-wide
 * vocabulary tile, and a re-laid-out copy of hidden). The backward size holds
 * a slice of Vc vocabulary columns of the logit gradient in two bf16 layouts
 * (4 * Np * Vc bytes, Np = 256*ceil(N/256); independent of V): Vc fills
 * 1 GiB while that gives at least 16384 columns, is 16384 up to 4 GiB, and
 * beyond that whatever fits in 4 GiB, down to a floor of 2048 columns. Then
 * re-laid-out copies of hidden and of the weight slice, and, when the slice
 * does not cover the whole vocabulary or dH is K-split, fp32 accumulators of
 * N*H*4 bytes each. */
flce_status_t flce_workspace_size(int64_t N, int64_t H, int64_t V, int reduction,
                                  size_t* fwd_bytes, size_t* bwd_bytes);

/* Forward. The call shape of the API example of verl pull request #462
 * (section "API": hidden [num_tokens, hidden_size], weight [hidden_size,
 * vocab_size], integer labels, a reduction argument, two outputs), with the
 * outputs of its section "Equivalent compute logic" (per-token entropy and the
 * label log-probability, the negated cross-entropy) and the cap of
 * Liger-Kernel issue #127 (proposal: applied after the head matmul).
 *   hidden   device bf16 [N,H]        weight  device bf16 [H,V]
 *   labels   device int64 [N]         ignore_index: label value that marks a skipped token
 *   softcap  c > 0 caps logits as c*tanh(z/c); c <= 0 disables the cap
 *   lse, logprob, entropy   device fp32 [N] outputs (always written).
 *                           Keep lse and entropy for flce_backward.
 *   logprob_mean, entropy_mean  device fp32 [1] outputs; required when
 *                           reduction is MEAN (the means) or SUM (the sums),
 *                           ignored under NONE.
 *   workspace  device scratch of at least the forward size from
 *              flce_workspace_size; its first 256 bytes hold the status word.
 */
flce_status_t flce_forward(const void* hidden, const void* weight, const int64_t* labels,
                           int64_t N, int64_t H, int64_t V, int64_t ignore_index,
                           float softcap, int reduction,
                           float* lse, float* logprob, float* entropy,
                           float* logprob_mean, float* entropy_mean,
                           void* workspace, size_t workspace_bytes, void* stream);

/* Backward: writes grad_hidden = dL/dhidden (device bf16 [N,H]) and
 * grad_weight = dL/dweight (device bf16 [H,V]) for
 *   L = sum_i gbar_i logprob_i + ebar_i entropy_i.
 * Liger-Kernel pull request #435 ("Why we pass gradient to output.backward()")
 * fixes the convention: an unreduced output takes one upstream gradient per
 * element, a reduced one a scalar; the review thread of Liger-Kernel pull
 * request #551 fixes the mean's divisor (the non-ignored tokens) and issue #127
 * (discussion) the cap's chain rule into both gradients.
 * hidden, weight, labels, N, H, V, ignore_index, softcap and reduction must be
 * those of the matching flce_forward; lse and entropy are its outputs.
 *   reduction NONE: grad_logprob, grad_entropy are device fp32 [N]
 *                   (gbar_i = grad_logprob[i]).
 *   reduction MEAN: they are device fp32 [1], the gradients of the two means
 *                   (gbar_i = grad_logprob[0] / n on non-ignored tokens).
 *   reduction SUM:  device fp32 [1], the gradients of the two sums
 *                   (gbar_i = grad_logprob[0] on non-ignored tokens).
 * Either gradient pointer may be NULL, meaning zero. Ignored tokens get zero
 * rows in grad_hidden. The logit gradient is recomputed, not stored by the
 * forward.
 */
flce_status_t flce_backward(const void* hidden, const void* weight, const int64_t* labels,
                            int64_t N, int64_t H, int64_t V, int64_t ignore_index,
                            float softcap, int reduction,
                            const float* lse, const float* entropy,
                            const float* grad_logprob, const float* grad_entropy,
                            void* grad_hidden, void* grad_weight,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Forward without a workspace, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation). Arguments, outputs and errors as flce_forward, minus
 * the workspace: the call runs in a scratch array of FLCE_NOALLOC_SCRATCH_BYTES
 * that the library holds in every device it runs on until the process ends
 * (its address is looked up once per device, on the first call with that
 * device current; `stream` must belong to the current device). Shapes whose
 * forward workspace (flce_workspace_size) exceeds that size are refused with
 * FLCE_ERR_TOO_LARGE before anything is enqueued (about N * (16 ceil(V/256) +
 * 2 H) bytes must fit, e.g. N = 2048 at H = 4096, V = 128256; a vocabulary
 * that is not a multiple of 8 adds 2 H V). The call allocates nothing,
 * enqueues kernels only, and writes every scratch byte it reads before
 * reading it. All calls on one device share that device's array: calls that
 * overlap in time on one device (two streams, two threads) race and give
 * wrong results; serialise them. The invalid-label count of these calls is
 * not reported (flce_get_status needs a workspace); such labels are treated
 * as ignored as in flce_forward. */
#define FLCE_NOALLOC_SCRATCH_BYTES (64u << 20)
flce_status_t flce_forward_noalloc(const void* hidden, const void* weight, const int64_t* labels,
                                   int64_t N, int64_t H, int64_t V, int64_t ignore_index,
                                   float softcap, int reduction,
                                   float* lse, float* logprob, float* entropy,
                                   float* logprob_mean, float* entropy_mean, void* stream);

/* Options of the extended entry points. class_weight was added in version
 * 211 (flce_version), entropy_per_token in version 212; the struct grew from
 * 24 to 32 and then to 40 bytes, so callers built against an older header must
 * be rebuilt. A zero-initialised tail keeps the earlier behaviour. */
typedef struct flce_options {
  int64_t ignore_index;  /* label value that marks a skipped token */
  float softcap;         /* c > 0: z' = c*tanh(z/c); c <= 0: no cap; must be finite */
  int reduction;         /* FLCE_REDUCTION_NONE, _MEAN or _SUM */
  float z_loss_scale;    /* lam >= 0 (finite) of z_loss = lam * lse^2 */
  int grad_dtype;        /* FLCE_GRAD_BF16 or FLCE_GRAD_F32: type of grad_hidden/grad_weight */
  const float* class_weight; /* NULL, or device fp32 [V] (the whole vocabulary; 4-byte
                              * aligned, finite values): target weights of the MEAN and
                              * SUM reductions, see below; FLCE_ERR_BAD_OPTION under NONE */
  int entropy_per_token; /* 0: the entropy follows `reduction` like the other outputs;
                          * 1: under MEAN or SUM the entropy is taken per token while the
                          * other outputs are reduced, so the backward's grad_entropy is
                          * device fp32 [N] (ebar_i = grad_entropy[i], no class weight) and
                          * the other upstream gradients stay [1]; the verl pull request
                          * #462 "Equivalent compute logic" returns entropy per token beside
                          * a reduced logprob. Any other value: FLCE_ERR_BAD_OPTION. The
                          * forward writes the per-token entropy under every reduction
                          * (reduced[1] is still the entropy's reduction). */
} flce_options_t;

/* Target (class) weights. The Liger-Kernel PR #551 review ("[Verl] Add
 * entropy loss to cross_entropy_loss and fused_linear_cross_entropy_loss")
 * lists target weights among the fused options and normalises the weighted
 * case by the weight of the non-ignored tokens instead of their count. With
 * class_weight set, a valid token t carries w_t = class_weight[labels[t]]:
 *   MEAN  reduced[k] = sum_t w_t x_t / sum_t w_t  (0 when the weight sum is 0),
 *         and the scalar upstream gradient g of output k reaches token t as
 *         g * w_t / sum_t w_t;
 *   SUM   reduced[k] = sum_t w_t x_t, gradient g * w_t,
 * for all four outputs x (logprob, entropy, uniform_ce, z_loss). For the
 * cross-entropy this is torch.nn.functional.cross_entropy(weight=...). The
 * per-token vectors stay unweighted. The weight sum is accumulated in
 * float64 in a fixed order. The sharded calls take the same weights (over
 * V_total) in flce_merge_shards and flce_backward_shard; flce_forward_shard
 * ignores them. */

/* Extended forward. As flce_forward, plus
 *   uniform_ce, z_loss  device fp32 [N] outputs, each optional (NULL = not
 *                       written);
 *   reduced             device fp32 [4]: the reductions (MEAN: means over the
 *                       n non-ignored tokens; SUM: sums) of logprob, entropy,
 *                       uniform_ce and z_loss, in that order; required unless
 *                       reduction is NONE, ignored then.
 * The workspace size is the forward size of flce_workspace_size. */
flce_status_t flce_forward_ex(const void* hidden, const void* weight, const int64_t* labels,
                              int64_t N, int64_t H, int64_t V, const flce_options_t* opt,
                              float* lse, float* logprob, float* entropy,
                              float* uniform_ce, float* z_loss, float* reduced,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Extended backward: grad_hidden [N,H] and grad_weight [H,V] (device; bf16
 * or fp32 as opt->grad_dtype says) of
 *   L = sum_i gbar_i logprob_i + ebar_i entropy_i + gu_i uniform_ce_i + gz_i z_loss_i,
 * with the four upstream gradients given as for flce_backward (device fp32,
 * [N] under NONE, [1] under MEAN and SUM; NULL means zero). opt and the
 * tensors must be those of the matching flce_forward_ex. The workspace size is
 * the backward size of flce_workspace_size. */
flce_status_t flce_backward_ex(const void* hidden, const void* weight, const int64_t* labels,
                               int64_t N, int64_t H, int64_t V, const flce_options_t* opt,
                               const float* lse, const float* entropy,
                               const float* grad_logprob, const float* grad_entropy,
                               const float* grad_uniform_ce, const float* grad_z_loss,
                               void* grad_hidden, void* grad_weight,
                               void* workspace, size_t workspace_bytes, void* stream);

/* ---- Vocabulary-sharded head ------------------------------------------------
 * The vocabulary is split into slices [v_begin, v_begin + Vs) of V_total
 * classes, each with its own weight slice weight_shard [H,Vs] (row-major, the
 * columns v_begin .. v_begin+Vs-1 of the full [H,V_total] weight), e.g. one per
 * GPU under tensor parallelism. Labels stay global class ids.
 *
 *   1. flce_forward_shard per slice: the per-token online-softmax state of the
 *      slice, {m, s, u, sum z'} with lse_slice = m + ln s, and the label logit
 *      (0 when the label lies in another slice). 20 bytes per token.
 *   2. Gather the S slices' states into [S,N,4] and label logits into [S,N]
 *      (an all-gather across GPUs) and call flce_merge_shards once: it merges
 *      them in slice order with the same combine as the unsharded forward and
 *      writes the outputs of flce_forward_ex.
 *   3. flce_backward_shard per slice with the merged lse and entropy: the
 *      slice's grad_weight [H,Vs] and its partial grad_hidden [N,H]; the sum
 *      over slices of the partials is grad_hidden (an all-reduce across GPUs;
 *      fp32 partials, opt->grad_dtype = FLCE_GRAD_F32, keep that sum exact to
 *      fp32 rounding).
 * The slice calls need Vs, v_begin within V_total (FLCE_ERR_BAD_SHAPE
 * otherwise); Vs follows the rules of V above; v_begin has no alignment rule.
 */

/* Slice forward. hidden, labels as flce_forward_ex; opt->reduction is ignored.
 *   state        device fp32 [N,4], 16-byte aligned: per token {m, s, u, sum z'}
 *                of the slice (natural-log units; {-1e30, 0, 0, 0} for ignored
 *                tokens)
 *   label_logit  device fp32 [N]: the capped label logit if the label lies in
 *                this slice, else 0
 * Workspace: the forward size of flce_workspace_size(N, H, Vs, ...). */
flce_status_t flce_forward_shard(const void* hidden, const void* weight_shard,
                                 const int64_t* labels, int64_t N, int64_t H, int64_t Vs,
                                 int64_t v_begin, int64_t V_total, const flce_options_t* opt,
                                 float* state, float* label_logit, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Workspace bytes of flce_merge_shards for N tokens (host only). */
flce_status_t flce_merge_workspace_size(int64_t N, size_t* bytes);

/* Merge of S slices: states device fp32 [S,N,4] and label_logits device fp32
 * [S,N] from flce_forward_shard (slice s at offset s*N*4 / s*N; any slice
 * order, merged in array order). Outputs as flce_forward_ex (lse, logprob,
 * entropy required when N > 0; uniform_ce, z_loss optional; reduced [4]
 * required unless reduction is NONE). 1 <= S <= 65536. */
flce_status_t flce_merge_shards(const float* states, const float* label_logits, int64_t S,
                                const int64_t* labels, int64_t N, int64_t V_total,
                                const flce_options_t* opt, float* lse, float* logprob,
                                float* entropy, float* uniform_ce, float* z_loss, float* reduced,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Slice backward: arguments as flce_backward_ex with lse and entropy from
 * flce_merge_shards; writes grad_weight_shard [H,Vs] (the slice's columns of
 * grad_weight) and grad_hidden_partial [N,H], this slice's share of
 * grad_hidden. Workspace: the backward size of flce_workspace_size(N, H, Vs,
 * ...). */
flce_status_t flce_backward_shard(const void* hidden, const void* weight_shard,
                                  const int64_t* labels, int64_t N, int64_t H, int64_t Vs,
                                  int64_t v_begin, int64_t V_total, const flce_options_t* opt,
                                  const float* lse, const float* entropy,
                                  const float* grad_logprob, const float* grad_entropy,
                                  const float* grad_uniform_ce, const float* grad_z_loss,
                                  void* grad_hidden_partial, void* grad_weight_shard,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* ---- Fused forward + backward (gradient in the forward) ----------------------
 * When the upstream gradients are known before the forward runs (a terminal
 * loss such as the mean cross-entropy, or per-token weights fixed in
 * advance), the logit gradient can be formed from logits kept during the
 * forward instead of recomputing them in the backward: this is how the fused
 * linear cross-entropy of Liger-Kernel pull request #551 (item 1 of its
 * description) produces the loss and its input gradient in one pass. Here the
 * tokens are taken in chunks; per chunk the capped logits of the whole
 * vocabulary are kept as z' - m in bf16 (m: the maximum over 128 vocabulary
 * rows, so the rounding error is relative to the distance from the maximum),
 * and the gradient is formed from them once the chunk's logsumexp is known.
 * Compared with flce_forward_ex + flce_backward_ex this saves the backward's
 * logit GEMM (2*N*H*V flops) and costs workspace and HBM traffic:
 *   chunk images  4 * 256*ceil(Nc/256) * 256*ceil(V/256) bytes,
 *   the weight re-laid out, 2 * H * 256*ceil(V/256) bytes,
 *   with more than one chunk and bf16 gradients, an fp32 dW accumulator of
 *   4 * H * V bytes (fp32 gradients accumulate in grad_weight itself).
 * The results agree with flce_forward_ex followed by flce_backward_ex to the
 * rounding of the kept logits (bf16 of z' - m), not bit for bit.
 *
 * chunk_tokens: tokens per chunk Nc (rounded up to 256); 0 picks the largest
 * multiple of 256 whose chunk images fit in 1 GiB (the budget of the
 * backward's logit-gradient images; at least 256 tokens), e.g. 2048 tokens at
 * V = 128256. A larger chunk saves passes over the fp32 dW accumulator at the
 * price of memory; chunk_tokens >= N keeps every logit of the call (4 bytes
 * each) in one chunk. V <= 2^21.
 * Workspace bytes for this shape, options and chunk_tokens (host only): */
flce_status_t flce_fused_workspace_size(int64_t N, int64_t H, int64_t V, const flce_options_t* opt,
                                        int64_t chunk_tokens, size_t* bytes);

/* The outputs of flce_forward_ex (lse, logprob, entropy required when N > 0;
 * uniform_ce, z_loss optional; reduced [4] required unless reduction is NONE)
 * and the gradients of flce_backward_ex (grad_hidden [N,H], grad_weight [H,V],
 * bf16 or fp32 as opt->grad_dtype says) for the upstream gradients given here
 * as for flce_backward_ex ([N] under NONE, [1] under MEAN and SUM, NULL =
 * zero). Under MEAN the scalar gradients are divided by the number of valid
 * tokens counted by this call. Errors as flce_backward_ex; FLCE_ERR_BAD_SHAPE
 * also for V > 2^21 or chunk_tokens < 0. */
flce_status_t flce_forward_backward(const void* hidden, const void* weight, const int64_t* labels,
                                    int64_t N, int64_t H, int64_t V, const flce_options_t* opt,
                                    int64_t chunk_tokens, const float* grad_logprob,
                                    const float* grad_entropy, const float* grad_uniform_ce,
                                    const float* grad_z_loss, float* lse, float* logprob,
                                    float* entropy, float* uniform_ce, float* z_loss,
                                    float* reduced, void* grad_hidden, void* grad_weight,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* ---- Embedding lookup and its gradient ----------------------------------------
 * The input end of the vocabulary matrix: for token ids x_i
 *   hidden_i = scale * E[x_i],     dE[v] = scale * sum_{i : x_i = v} grad_hidden_i,
 * where E[v] is row v of a table [V,H] (FLCE_EMBED_VH) or column v of a weight
 * [H,V] (FLCE_EMBED_HV: the head's own weight, so that a model with tied
 * embeddings keeps one matrix; Gemma2-style models scale by sqrt(H)).
 * A token equal to ignore_index, or outside [0, V_total), gives a zero row and
 * takes part in no gradient; the latter are counted in the workspace's status
 * word (flce_get_status). A vocabulary slice [v_begin, v_begin + Vs) of V_total
 * ids gives zero rows for the ids of other slices, so that the sum of the
 * slices' outputs is the whole lookup (an all-reduce across GPUs), and the
 * slice's own gradient; unsharded calls pass Vs = V_total, v_begin = 0.
 * Every product is formed and every sum accumulated in fp32, in an order that
 * depends on the inputs only (no atomics), and rounded once to the output type. */
enum { FLCE_EMBED_VH = 0, FLCE_EMBED_HV = 1 };

typedef struct flce_embedding_options {
  int64_t ignore_index;  /* token id that marks a skipped position */
  double scale;          /* finite; used as fp32 */
  int layout;            /* FLCE_EMBED_VH or FLCE_EMBED_HV */
  int hidden_dtype;      /* FLCE_GRAD_BF16 or FLCE_GRAD_F32: type of the backward's grad_hidden
                          * (the forward reads and writes bf16 whatever it says) */
  int grad_dtype;        /* FLCE_GRAD_BF16 or FLCE_GRAD_F32: type of grad_weight */
  int accumulate;        /* 0: grad_weight is written whole (zero for unused ids);
                          * 1: the gradient is added to what grad_weight holds, e.g. the head's
                          * grad_weight of a tied matrix (ids without a token are not written) */
} flce_embedding_options_t;

/* Workspace bytes of the two calls for Vs ids (host only; either out-pointer
 * may be NULL). */
flce_status_t flce_embedding_workspace_size(int64_t N, int64_t H, int64_t Vs,
                                            const flce_embedding_options_t* opt, size_t* fwd_bytes,
                                            size_t* bwd_bytes);

/* hidden device bf16 [N,H] from weight device bf16 ([Vs,H] or [H,Vs]) and
 * tokens device int64 [N]. H must be a multiple of 8; Vs may take any value.
 * weight, hidden and workspace 16-byte aligned. */
flce_status_t flce_embedding_forward(const void* weight, const int64_t* tokens, int64_t N,
                                     int64_t H, int64_t Vs, int64_t v_begin, int64_t V_total,
                                     const flce_embedding_options_t* opt, void* hidden,
                                     void* workspace, size_t workspace_bytes, void* stream);

/* grad_weight device ([Vs,H] or [H,Vs], type grad_dtype) from grad_hidden
 * device [N,H] (type hidden_dtype). grad_hidden, grad_weight and workspace
 * 16-byte aligned. */
flce_status_t flce_embedding_backward(const void* grad_hidden, const int64_t* tokens, int64_t N,
                                      int64_t H, int64_t Vs, int64_t v_begin, int64_t V_total,
                                      const flce_embedding_options_t* opt, void* grad_weight,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* ---- Losses on the head's per-token outputs -------------------------------------
 * The losses that an RL or preference fine-tuning step forms between the head's
 * forward (per-token logprob and entropy) and its backward (per-token upstream
 * gradients). All take the packed batch the head takes: N tokens, labels with
 * ignore_index (and ids outside [0, V)) marking tokens without a loss, and B
 * sequences given by cu_seqlens, device int64 [B+1]: sequence s is the tokens
 * [cu_seqlens[s], cu_seqlens[s+1]), which must not decrease and must lie in
 * [0, N]. Tokens before the first and behind the last sequence take no part
 * (gradient 0). What the per-token arrays hold at tokens that take no part is
 * never used (it may be NaN or infinite).
 * Every per-token term is computed, and every sum accumulated, in float64 in a
 * fixed order; outputs are rounded once to fp32.
 * A sequence whose offsets decrease or leave [0, N] makes the reduced loss, the
 * statistics and the gradient of every token with a valid label NaN, and
 * (preference) its pair's outputs; the results of the other sequences are then unspecified. The status
 * word counts such sequences or, when there are none, the labels of sequences
 * that are neither ignore_index nor in [0, V). */
enum { FLCE_REDUCTION_SEQUENCE_MEAN = 3 };  /* flce_policy_loss_* only */
enum { FLCE_KL_K1 = 0, FLCE_KL_K2 = 1, FLCE_KL_K3 = 2 };
enum { FLCE_RATIO_TOKEN = 0, FLCE_RATIO_SEQUENCE = 1 };

/* Clipped policy loss with a KL term. With d = logprob - old_logprob (under
 * FLCE_RATIO_SEQUENCE its mean over the sequence's valid tokens), r = exp(d) and
 * the advantage A, a valid token's loss is
 *   policy = 0 where A = 0, else
 *   policy = -min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A), and where A < 0
 *            and dual_clip > 0 at most -dual_clip A,
 *   loss   = policy + kl_coef kl - entropy_coef entropy,
 *   kl(x)  = x (K1), x^2 / 2 (K2), exp(-x) + x - 1 (K3),  x = logprob - ref_logprob.
 * A ratio exactly on a bound is not clipped. The gradient of a clipped policy
 * term is zero. MEAN averages over the batch's valid tokens, SUM sums,
 * SEQUENCE_MEAN averages within each sequence and then over the sequences that
 * have a valid token. No valid token gives 0. */
typedef struct flce_policy_options {
  int64_t ignore_index;
  double clip_low;      /* in [0, 1] */
  double clip_high;     /* >= 0 */
  double dual_clip;     /* 0: off, else > 1 */
  double kl_coef;       /* needs ref_logprob unless 0 */
  double entropy_coef;  /* needs entropy unless 0 */
  int kl_estimator;     /* FLCE_KL_* */
  int level;            /* FLCE_RATIO_*; SEQUENCE needs cu_seqlens and one advantage a sequence */
  int reduction;        /* FLCE_REDUCTION_MEAN, _SUM or _SEQUENCE_MEAN */
  int advantages_per_sequence; /* 0: advantages [N], 1: advantages [B] */
} flce_policy_options_t;

/* Workspace bytes of the two policy-loss calls that take one (host only). */
flce_status_t flce_policy_workspace_size(int64_t N, int64_t B, size_t* bytes);

/* logprob, old_logprob (and where given entropy, ref_logprob): device fp32 [N];
 * advantages device fp32 [N] or [B]; labels device int64 [N]; cu_seqlens device
 * int64 [B+1], or NULL with B = 1: one sequence of all tokens.
 *   loss       device fp32 [1], or NULL
 *   stats      device fp32 [8]: loss, policy, kl, entropy, share of clipped
 *              tokens, -d (the k1 estimate of KL(old || new)), each reduced like
 *              the loss; then the number of valid tokens and of sequences that
 *              have one
 *   seq_state  device float64 [B+1, 2]: what flce_policy_loss_backward needs */
flce_status_t flce_policy_loss_forward(const float* logprob, const float* entropy,
                                       const float* old_logprob, const float* ref_logprob,
                                       const float* advantages, const int64_t* labels,
                                       const int64_t* cu_seqlens, int64_t N, int64_t B, int64_t V,
                                       const flce_policy_options_t* opt, float* loss,
                                       float* stats, double* seq_state, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* grad_logprob, and unless NULL grad_entropy (device fp32 [N]), of
 * grad_loss[0] * loss (device fp32 [1]; NULL means 1), from the inputs of the
 * matching forward and its seq_state. */
flce_status_t flce_policy_loss_backward(const float* logprob, const float* old_logprob,
                                        const float* ref_logprob, const float* advantages,
                                        const int64_t* labels, const int64_t* cu_seqlens,
                                        int64_t N, int64_t B, int64_t V,
                                        const flce_policy_options_t* opt, const double* seq_state,
                                        const float* grad_loss, float* grad_logprob,
                                        float* grad_entropy, void* stream);

/* Both in one call, for an upstream gradient known in advance (one launch for
 * small batches). The results are those of the
 * two calls above. */
flce_status_t flce_policy_loss_forward_backward(
    const float* logprob, const float* entropy, const float* old_logprob, const float* ref_logprob,
    const float* advantages, const int64_t* labels, const int64_t* cu_seqlens, int64_t N, int64_t B,
    int64_t V, const flce_policy_options_t* opt, const float* grad_loss, float* loss,
    float* stats, float* grad_logprob, float* grad_entropy, void* workspace, size_t workspace_bytes,
    void* stream);

/* Preference loss over P pairs of sequences: sequence i < P is the chosen and
 * sequence P + i the rejected answer of pair i (2 P sequences). With R_s the sum
 * over the valid tokens of sequence s of logprob - ref_logprob (ref_logprob NULL:
 * of logprob), divided by their number under length_normalize (an empty sequence
 * has R = 0), and x = beta (R_chosen - R_rejected) - margin, a pair's loss is
 *   SIGMOID  -(1 - eps) log sigmoid(x) - eps log sigmoid(-x),  eps = label_smoothing
 *   HINGE    max(0, 1 - x)   (no gradient at x = 1)
 *   IPO      (R_chosen - R_rejected - 1 / (2 beta))^2
 * Every pair counts in the mean. */
enum { FLCE_PREFERENCE_SIGMOID = 0, FLCE_PREFERENCE_HINGE = 1, FLCE_PREFERENCE_IPO = 2 };

typedef struct flce_preference_options {
  int64_t ignore_index;
  double beta;             /* > 0 */
  double label_smoothing;  /* in [0, 0.5]; SIGMOID only, else 0 */
  double margin;           /* finite; SIGMOID and HINGE only, else 0 */
  int kind;                /* FLCE_PREFERENCE_* */
  int length_normalize;    /* 0 or 1 */
  int reduction;           /* FLCE_REDUCTION_NONE, _MEAN or _SUM over the pairs */
} flce_preference_options_t;

/* Workspace bytes of the two preference-loss calls that take one (host only). */
flce_status_t flce_preference_workspace_size(int64_t N, int64_t P, size_t* bytes);

/* logprob, ref_logprob (may be NULL): device fp32 [N]; labels device int64 [N];
 * cu_seqlens device int64 [2P+1].
 *   pair_loss  device fp32 [P], written under every reduction
 *   loss       device fp32 [1]; required unless reduction is NONE, ignored then
 *   chosen_reward, rejected_reward  device fp32 [P]: beta R of the two sides
 *   seq_state  device float64 [2P+1]: what flce_preference_loss_backward needs */
flce_status_t flce_preference_loss_forward(const float* logprob, const float* ref_logprob,
                                           const int64_t* labels, const int64_t* cu_seqlens,
                                           int64_t N, int64_t P, int64_t V,
                                           const flce_preference_options_t* opt, float* loss,
                                           float* pair_loss, float* chosen_reward,
                                           float* rejected_reward, double* seq_state,
                                           void* workspace, size_t workspace_bytes, void* stream);

/* grad_logprob device fp32 [N] for the upstream gradient grad_loss: device fp32
 * [P] under NONE (NULL: ones), [1] otherwise (NULL: 1). */
flce_status_t flce_preference_loss_backward(const int64_t* labels, const int64_t* cu_seqlens,
                                            int64_t N, int64_t P, int64_t V,
                                            const flce_preference_options_t* opt,
                                            const double* seq_state, const float* grad_loss,
                                            float* grad_logprob, void* stream);

/* Both in one call. The results are those of the
 * two calls above. */
flce_status_t flce_preference_loss_forward_backward(
    const float* logprob, const float* ref_logprob, const int64_t* labels,
    const int64_t* cu_seqlens, int64_t N, int64_t P, int64_t V,
    const flce_preference_options_t* opt, const float* grad_loss, float* loss, float* pair_loss,
    float* chosen_reward, float* rejected_reward, float* grad_logprob, void* workspace,
    size_t workspace_bytes, void* stream);

/* ---- Logits to sample from --------------------------------------------------------
 * The head's logits for a few rows, e.g. the last positions of the sequences that
 * are being generated:
 *   z_iv = cap(sum_h hidden[i,h] weight[h,v] + bias[v]),
 *   cap(z) = c * tanh(z / c) if softcap c > 0, else z.
 * The products are summed in fp32 in a fixed order and rounded once to the
 * output's type. For many tokens there is flce_forward, which never writes the
 * logits: N <= 1024 here. */

/* Workspace bytes (host only). */
flce_status_t flce_logits_workspace_size(int64_t N, int64_t H, int64_t V, size_t* bytes);

/* hidden device bf16 [N,H], weight device bf16 [H,V], both 16-byte aligned (H a
 * multiple of 8, V any size); bias device fp32 [V] or NULL; out device [N,V] of
 * out_dtype (FLCE_GRAD_BF16 or FLCE_GRAD_F32), row i from element i * ld_out on
 * (ld_out >= V), aligned to its elements. softcap finite, as its reciprocal in fp32 if it
 * is above 0. The call has no status to read. */
flce_status_t flce_logits(const void* hidden, const void* weight, const float* bias, int64_t N,
                          int64_t H, int64_t V, float softcap, int out_dtype, void* out,
                          int64_t ld_out, void* workspace, size_t workspace_bytes, void* stream);

/* ---- Penalties, biases and masks on logits ------------------------------------------
 * What a sampler does to a row of logits before it draws a token. Row i has a
 * history of tokens, the first prompt_lengths[i] of which are its prompt and the
 * others generated. With n(v) the occurrences of id v among the generated ones,
 * a logit x of id v becomes, in this order,
 *   x > 0 ? x / r : x * r          if v is anywhere in the history (repetition r)
 *   x - frequency * n(v), then x - presence if n(v) > 0
 *   x + bias[v] + the sum of the row's listed biases of v (in the list's order)
 *   x / temperature                (not if the temperature is 0: such a row is for
 *                                   its largest value)
 *   -inf                           if the row's mask does not allow v, whatever x is
 * in fp32, where the divisions are products with the fp32 reciprocal, and is
 * rounded once to the output's type. Each row also gets, of the logits as they are
 * returned,
 *   lse      logsumexp (-inf if nothing is allowed), so that out[t] - lse is the
 *            log-probability with which token t is drawn (the policy loss's
 *            old_logprob);
 *   entropy  lse - sum p x (0 if nothing is allowed, NaN if lse is not finite
 *            otherwise);
 *   greedy   the first id of the largest value (the first NaN, if there is one; -1
 *            if nothing is allowed). */
typedef struct flce_process_options {
  int64_t ignore_index;    /* token id of a history or of listed biases to pass over */
  /* History: tokens device int64. Packed (tokens_stride 0): row i is tokens
   * [offsets[i], offsets[i+1]) of the tokens_size ones (offsets [N+1], within
   * [0, tokens_size] and not decreasing). Padded (tokens_stride > 0, N * tokens_stride
   * <= tokens_size): row i is the first offsets[i] tokens (in [0, tokens_stride]) from
   * i * tokens_stride on (offsets [N]). Both NULL: no history. A row has at most 2^31 - 1
   * tokens; the offsets of a longer one are bad. */
  const int64_t* tokens;
  int64_t tokens_size, tokens_stride;
  const int64_t* offsets;
  const int64_t* prompt_lengths;  /* [N], cut to the history; NULL: 0 */
  /* Device fp32 [N] in the ranges of the values of all rows below (not checked), or NULL
   * for those. */
  const float* repetition;
  const float* presence;
  const float* frequency;
  const float* temperatures;
  double repetition_penalty;      /* > 0, 1: off; finite in fp32, as its reciprocal there */
  double presence_penalty;        /* 0: off */
  double frequency_penalty;       /* 0: off */
  double temperature;             /* 0, or like repetition_penalty; 1: off */
  const float* bias;              /* device fp32 [V] (bias_stride 0) or [N, bias_stride], or NULL */
  int64_t bias_stride;
  /* Listed biases: row i's are the pairs [bias_offsets[i], bias_offsets[i+1]) of the
   * bias_count ones, or NULL. */
  const int64_t* bias_tokens;
  const float* bias_values;
  int64_t bias_count;
  const int64_t* bias_offsets;    /* [N+1], within [0, bias_count] and not decreasing */
  const int32_t* allowed;         /* device bits: id v of a row is allowed if bit v % 32 of
                                   * word v / 32 is set; one row for all (allowed_stride 0) or
                                   * rows of allowed_stride words; NULL: all allowed */
  int64_t allowed_stride;
  int logits_dtype, out_dtype;    /* FLCE_GRAD_BF16 or FLCE_GRAD_F32 */
} flce_process_options_t;

/* Workspace bytes of the two calls (host only). */
flce_status_t flce_process_workspace_size(int64_t N, int64_t V, size_t* bytes);

/* logits device [N,V] of logits_dtype, row i from element i * ld on (ld >= V); out
 * likewise of out_dtype and ld_out (it may be logits itself, of the same type and
 * ld, and shares no memory with it otherwise); lse and entropy device fp32 [N], greedy
 * device int64 [N], each or NULL. All aligned to their elements. Tokens of a history (if
 * there is a penalty) or of listed biases that are neither ignore_index nor in [0, V) are
 * passed over and counted in the status word. A row whose offsets are bad (see above)
 * counts there as one, and its outputs are NaN and -1. */
flce_status_t flce_process_logits(const void* logits, int64_t ld, int64_t N, int64_t V,
                                  const flce_process_options_t* opt, void* out, int64_t ld_out,
                                  float* lse, float* entropy, int64_t* greedy, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Upstream gradients of a forward's outputs, each NULL for zero: of the returned logits
 * (type out_dtype, rows of ld_grad_out), of lse and of entropy (device fp32 [N]). The
 * latter two need what the forward returned: out (rows of ld_out), lse and, for
 * grad_entropy, entropy. */
typedef struct flce_process_grads {
  const void* grad_out;
  int64_t ld_grad_out;
  const float* grad_lse;
  const float* grad_entropy;
  const void* out;
  int64_t ld_out;
  const float* lse;
  const float* entropy;
} flce_process_grads_t;

/* grad_logits device [N,V] (type logits_dtype, rows of ld_grad) = what a logit is
 * multiplied by (r where x <= 0 and 1 / r where x > 0 for seen ids, then
 * 1 / temperature; 0 where the mask does not allow it) times
 *   grad_out + p (grad_lse - grad_entropy (x' - lse + entropy)),  p = exp(x' - lse)
 * with x' the returned logit (no second term where p is 0); NaN in rows of bad
 * offsets. logits and opt are those that went into the forward, whose output must not
 * have been written over them. grad_logits may be grad_out itself, of the same type
 * and ld. Listed and dense biases play no part and are not looked at. */
flce_status_t flce_process_logits_backward(const flce_process_grads_t* grads, const void* logits,
                                           int64_t ld, int64_t N, int64_t V,
                                           const flce_process_options_t* opt, void* grad_logits,
                                           int64_t ld_grad, void* workspace,
                                           size_t workspace_bytes, void* stream);

/* ---- Norm of the gradients and AdamW --------------------------------------------------
 * The update that ends a training step, over many tensors in a few launches, with
 * the step's count, the clip factor and (optionally) the learning rate on the
 * device, so that a captured step stays right when it is replayed. The arrays of
 * pointers and sizes are host memory, read before the call returns. */

/* Workspace bytes of flce_grad_norm (host only): sizes[i] values in tensor i. */
flce_status_t flce_grad_norm_workspace_size(const int64_t* sizes, int64_t count, size_t* bytes);

/* norm (device fp32 [1]) = sqrt(sum of squares) over all values of the count tensors
 * (device, type dtypes[i], aligned to their elements), summed in float64 in a fixed
 * order. scale (device fp32 [1], or NULL) = min(1, max_norm / norm) of the float64 norm, 1
 * if max_norm is 0, and NaN if a value is not finite. (Of finite values norm alone can
 * be above fp32's range, and then is infinite.) */
flce_status_t flce_grad_norm(const void* const* grads, const int64_t* sizes, const int* dtypes,
                             int64_t count, double max_norm, float* norm, float* scale,
                             void* workspace, size_t workspace_bytes, void* stream);

enum { FLCE_STATE_F32 = 0, FLCE_STATE_8BIT = 1 };
enum { FLCE_ROUND_NEAREST = 0, FLCE_ROUND_STOCHASTIC = 1 };

/* The tensors of an update: host arrays of `count` entries. Tensor i has sizes[i]
 * values, its pointers are device pointers aligned to their elements, to memory of its
 * own; sizes of 0 are passed over. With FLCE_STATE_8BIT the states are e4m3 codes (OCP:
 * the largest is 448) in blocks of 256 values from the tensor's start on, and
 * exp_avg_scales and exp_avg_sq_scales (fp32, one a block) what a code is multiplied by;
 * exp_avg_sqs then holds the root of the second moment. */
typedef struct flce_adamw_list {
  int64_t count;
  const int64_t* sizes;
  void* const* params;           /* of param_dtypes; written */
  const void* const* grads;      /* of grad_dtypes */
  void* const* masters;          /* fp32 copies that the update is made on (a parameter then is
                                  * its copy rounded to the nearest); NULL, or NULL entries, for
                                  * none; bf16 parameters only */
  void* const* exp_avgs;         /* fp32 or codes */
  void* const* exp_avg_sqs;
  void* const* exp_avg_scales;   /* 8-bit states only */
  void* const* exp_avg_sq_scales;
  const int* param_dtypes;       /* FLCE_GRAD_BF16 or FLCE_GRAD_F32 */
  const int* grad_dtypes;
} flce_adamw_list_t;

typedef struct flce_adamw_options {
  double lr;               /* finite */
  double beta1, beta2;     /* in [0, 1) */
  double eps;              /* 0 or at least 2^-126 (with 0, a value whose gradients were all 0
                            * becomes 0 / 0) */
  double weight_decay;     /* finite */
  int state_dtype;         /* FLCE_STATE_* */
  int rounding;            /* FLCE_ROUND_*: of bf16 weights without a master copy, and of codes */
  uint64_t seed;           /* of stochastic rounding */
} flce_adamw_options_t;

/* Workspace bytes of flce_adamw_step (host only). */
size_t flce_adamw_workspace_size(void);

/* With t = step[0] + 1 (step device int64 [1], then set to t), s = grad_scale[0]
 * (device fp32 [1]; NULL: 1) and lr = lr_device[0] (device fp32 [1]; NULL: opt->lr),
 * for every value in fp32:
 *   g = s grad,  m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,
 *   p = (1 - lr weight_decay) p - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps).
 * If s is not finite (an overflow in the backward), nothing is changed, step among
 * it. Without a grad_scale, a gradient that is not finite makes its weight NaN and its
 * states NaN or infinite; in 8 bits all states of its block are NaN then: a NaN or an
 * infinity (the square of a gradient above 2^64 is one) makes the block's scale infinite
 * and every code 0 or NaN. In 8-bit states a block's scale is otherwise its largest
 * magnitude a times 1 / 448 and its codes are those of the values times 448 (1 / a) (all
 * 0 if a is below 2^-100), in fp32; a second moment above 0 has a code above 0.
 * Stochastic rounding goes up with the probability of the part cut off, by 16 bits
 * of a hash of the seed, t, the tensor's index and the value's: lists of a step that are
 * updated by calls of their own take different seeds, or they draw the same bits. */
flce_status_t flce_adamw_step(const flce_adamw_list_t* list, const flce_adamw_options_t* opt,
                              const float* lr_device, const float* grad_scale, int64_t* step,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Reads the status word that the last call with this workspace left, after
 * synchronising `stream`. *invalid_labels (may be NULL) receives the number of
 * labels (embedding, processing of logits: tokens) that were neither ignore_index nor in
 * [0, V), or of bad sequence offsets (losses, processing of logits); returns
 * FLCE_ERR_INVALID_LABEL if that number is not 0, else FLCE_OK. */
flce_status_t flce_get_status(const void* workspace, int64_t* invalid_labels, void* stream);

/* Static English text for a status code. */
const char* flce_status_string(flce_status_t status);

/* Library version, major*10000 + minor*100 + patch. It changes with the layout of
 * an existing structure or the meaning of an existing call. Entry points added
 * beside these, such as the embedding and the losses after version 212, leave it:
 * a program that loads the library at run time looks for their symbols. */
int flce_version(void);

/* Measurement hooks. When enabled, every kernel the library launches is
 * bracketed by a pair of hipEvents recorded on the launch stream; the host
 * side keeps one table per kernel kind. Host state, not thread-safe; meant for
 * benchmarks. */
flce_status_t flce_profile_enable(int enable);
flce_status_t flce_profile_reset(void);
/* Number of kernel kinds in the table. */
int flce_profile_kinds(void);
/* Synchronises the recorded events, then returns the name, the number of
 * launches and the summed duration (ms) of kernel kind `kind`. */
flce_status_t flce_profile_read(int kind, const char** name, int64_t* launches, double* total_ms);

/* Measurement hook, for context in benchmarks: the bf16 MFMA rate (TFLOP/s,
 * in *tflops) that this device sustains in the GEMM kernels' wave tile: one
 * 512-thread block per CU (two waves per SIMD), each wave running `steps`
 * (4 <= steps <= 2^24, rounded down to a multiple of 4) 16-wide K steps of
 * 4 x 2 v_mfma_f32_32x32x16_bf16, with the GEMM kernels' data movement added
 * by `mode`:
 *   0  operands held in registers, pseudo-random bf16 in [-2, 2);
 *   1  the same with zero operands;
 *   2  mode 0 with each step's six operand fragments read from LDS
 *      (ds_read_b128);
 *   3  mode 2 plus the global -> LDS DMA of a 256 x 256 block tile (32 KiB per
 *      block per 32-deep K block) from a 2 MiB window that stays in L2.
 * The published dense peak assumes a clock that the matrix cores hold on
 * zero operands but not under the power they draw on varying data; modes 2
 * and 3 show what the LDS and L2 traffic of the tile costs on top.
 * workspace: device, 16-byte aligned, at least 256 * 512 * 4 bytes (results)
 * plus 2 MiB for mode 3 (the DMA window, filled here). Synchronises `stream`.
 * FLCE_ERR_BAD_OPTION for another mode. */
flce_status_t flce_probe_mfma_rate(int mode, int64_t steps, double* tflops, void* workspace,
                                   size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FLCE_H */
