"""``linear_cross_entropy``: the head as a torch autograd function, in the
call shape of the API example of verl pull request #462 (section "API"):
``linear_cross_entropy(hidden, weight, labels, reduction="mean")`` returns two
outputs, the label log-probability and the entropy. Following that page's
"Equivalent compute logic", the first output is the log-probability of the
label (minus the cross-entropy), not the cross-entropy itself.

``embedding``, ``policy_loss`` and ``preference_loss`` are the operators
beside the head in the same manner: the tied (or separate) embedding lookup,
and the losses of RL and preference tuning on the head's per-token outputs.

Marshalling only: the forward calls flce_forward through ``flce.forward``
and keeps the per-token lse and entropy; the backward hands the upstream
gradients of the two outputs to flce_backward through ``flce.backward``.

Under graph capture: torch adds a leaf's gradient on the stream on which the
leaf's accumulating node was made, and that node lives as long as any graph of
the leaf. A stream made for the work joins a capture through events, so a result
of a warm-up on a side stream may still be bound. The default stream cannot join
one: a captured backward over a leaf that an eager graph made there still holds
would reach out of the capture, which ends the process. While such a result of
this module on the same leaf lives (drop it first), ``embedding``,
``policy_loss`` and ``preference_loss`` refuse the call, and the backward of
``linear_cross_entropy`` raises. Seen are leaves among the arguments and leaves
that an argument is a cast, view or multiple of; not seen are leaves further
back in the graph, and results that other operators made on a leaf first.
"""
from __future__ import annotations

import torch

from torch.autograd.function import once_differentiable

from . import flce

__all__ = ["LinearCrossEntropy", "linear_cross_entropy", "Embedding", "embedding",
           "PolicyLoss", "policy_loss", "PreferenceLoss", "preference_loss"]


def _accumulator(node):
    """The accumulating node of a leaf on a GPU: the node itself, or the one behind it
    where up to eight operations of one input each (casts, views, scalings) lie
    between; else None."""
    for _ in range(9):
        if node.name() == "torch::autograd::AccumulateGrad":
            return node if node.variable.is_cuda else None
        behind = [n for n, _ in node.next_functions if n is not None]
        if len(behind) != 1:
            break
        node = behind[0]
    return None


def _accumulators(tensors):
    """The accumulating nodes of the leaves that the tensors are or are cast from."""
    if not torch.is_grad_enabled():
        return []
    nodes = [_accumulator(torch.autograd.graph.get_gradient_edge(t).node) for t in tensors
             if isinstance(t, torch.Tensor) and t.is_cuda and t.requires_grad]
    return [node for node in nodes if node is not None]


_DEFAULT_STREAM = 0  # raw handle


def _refuse_captured(nodes):
    """Under capture: raises if an accumulating node among the nodes belongs to a
    live graph that this module made on the default stream."""
    for node in nodes:
        if (node.metadata.get("flce_stream") == _DEFAULT_STREAM
                and torch._C._cuda_getCurrentRawStream(node.variable.device.index)
                != _DEFAULT_STREAM):
            raise RuntimeError(
                "an eager result of this leaf is still alive on the default stream: a backward "
                "over it cannot be captured; drop the result first, make it on a side stream, "
                "or use torch.no_grad() for the forward alone")


def _refuse_captured_leaves(*tensors):
    if getattr(tensors[0], "is_cuda", False) and torch.cuda.is_current_stream_capturing():
        _refuse_captured(_accumulators(tensors))


def _note_leaves(*tensors):
    """Notes the stream of a new graph on its leaves' accumulating nodes (kept
    alive by the graph, and with them the note)."""
    for node in _accumulators(tensors):
        node.metadata.setdefault("flce_stream", torch._C._cuda_getCurrentRawStream(
            node.variable.device.index))


def _reached(node):
    """Whether the running backward pass goes on to the accumulating node."""
    try:
        return torch._C._will_engine_execute_node(node)
    except RuntimeError:  # of torch.autograd.grad, which asks for this leaf
        return True


class LinearCrossEntropy(torch.autograd.Function):
    """(logprob, entropy) of the fused head; see ``linear_cross_entropy``."""

    @staticmethod
    def forward(ctx, hidden, weight, labels, reduction="mean", ignore_index=-100, softcap=0.0,
                class_weight=None, entropy_reduction=None):
        out = flce.forward(hidden, weight, labels, ignore_index=ignore_index, softcap=softcap,
                           reduction=reduction, class_weight=class_weight)
        ctx.save_for_backward(hidden, weight, labels, out["lse"], out["entropy"])
        ctx.class_weight = class_weight
        ctx.reduction = reduction
        ctx.ignore_index = ignore_index
        ctx.softcap = softcap
        ctx.entropy_tokens = reduction == "none" or entropy_reduction == "none"
        ctx.entropy_reduction = entropy_reduction
        lp = out["logprob"] if reduction == "none" else out[f"logprob_{reduction}"].reshape(())
        ent = out["entropy"] if ctx.entropy_tokens else out[f"entropy_{reduction}"].reshape(())
        return lp, ent

    @staticmethod
    def backward(ctx, grad_logprob, grad_entropy):
        if torch.cuda.is_current_stream_capturing():
            # Of hidden and weight; a captured forward alone is always allowed.
            leaves = [_accumulator(node) for node, _ in ctx.next_functions[:2] if node is not None]
            _refuse_captured([node for node in leaves if node is not None and _reached(node)])
        hidden, weight, labels, lse, entropy = ctx.saved_tensors
        n = hidden.shape[0]

        def prep(g, size):
            return None if g is None else g.float().reshape(size).contiguous()

        gh, gw = flce.backward(hidden, weight, labels, lse, entropy,
                               prep(grad_logprob, n if ctx.reduction == "none" else 1),
                               prep(grad_entropy, n if ctx.entropy_tokens else 1),
                               ignore_index=ctx.ignore_index, softcap=ctx.softcap,
                               reduction=ctx.reduction, class_weight=ctx.class_weight,
                               entropy_reduction=ctx.entropy_reduction)
        return gh, gw, None, None, None, None, None, None


def linear_cross_entropy(hidden, weight, labels, reduction="mean", ignore_index=-100,
                         softcap=0.0, class_weight=None, entropy_reduction=None):
    """(logprob, entropy) for hidden bf16 [N,H], weight bf16 [H,V], labels
    int64 [N]: per token ([N] fp32) under reduction "none", else the mean over
    the non-ignored tokens ("mean") or their sum ("sum"), 0-d fp32 tensors.
    ``entropy_reduction="none"`` returns the entropy per token ([N], 0 at
    ignored tokens) beside the reduced logprob, the output shapes of the verl
    pull request #462 "Equivalent compute logic"; None reduces both alike.
    class_weight (fp32 [V], "mean" / "sum" only) weights token t by
    class_weight[labels[t]] in the reductions; the mean then divides by the
    weight sum of the non-ignored tokens. Differentiable with respect to
    hidden and weight (gradients in bf16)."""
    out = LinearCrossEntropy.apply(hidden, weight, labels, reduction, ignore_index, softcap,
                                   class_weight, entropy_reduction)
    _note_leaves(hidden, weight)
    return out


class Embedding(torch.autograd.Function):
    """The scaled lookup; see ``embedding``."""

    @staticmethod
    def forward(ctx, weight, tokens, layout, scale, ignore_index):
        hidden = flce.embedding(weight, tokens, layout=layout, scale=scale,
                                ignore_index=ignore_index)["hidden"]
        ctx.save_for_backward(tokens)
        ctx.vocab_size = weight.shape[1 if layout == "hv" else 0]
        ctx.layout, ctx.scale, ctx.ignore_index = layout, scale, ignore_index
        return hidden

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_hidden):
        tokens, = ctx.saved_tensors
        grad_hidden = grad_hidden.contiguous()
        if grad_hidden.data_ptr() % 16 != 0:  # a view into another tensor's gradient
            grad_hidden = grad_hidden.clone()
        gw = flce.embedding_backward(grad_hidden, tokens, ctx.vocab_size, layout=ctx.layout,
                                     scale=ctx.scale, ignore_index=ctx.ignore_index)
        return gw, None, None, None, None


def embedding(weight, tokens, layout="hv", scale=1.0, ignore_index=-100):
    """hidden bf16 [N,H] = scale * E[tokens] for tokens int64 [N] and weight
    bf16: the head's [H,V] (layout "hv", tied embeddings) or a table [V,H]
    ("vh"). Zero rows at ignore_index and at ids outside the vocabulary.
    Differentiable with respect to weight (gradient in bf16)."""
    _refuse_captured_leaves(weight)
    hidden = Embedding.apply(weight, tokens, layout, scale, ignore_index)
    _note_leaves(weight)
    return hidden


class PolicyLoss(torch.autograd.Function):
    """(loss, stats) of the clipped policy loss; see ``policy_loss``."""

    @staticmethod
    def forward(ctx, logprob, entropy, labels, old_logprob, advantages, ref_logprob, cu_seqlens,
                options):
        out = flce.policy_loss(logprob, labels, old_logprob, advantages, entropy=entropy,
                               ref_logprob=ref_logprob, cu_seqlens=cu_seqlens, **options)
        ctx.save_for_backward(logprob, labels, old_logprob, advantages, ref_logprob, cu_seqlens,
                              out["seq_state"])
        ctx.options = options
        ctx.mark_non_differentiable(out["stats"])
        ctx.set_materialize_grads(False)
        return out["loss"].reshape(()), out["stats"]

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss, _grad_stats):
        if grad_loss is None:
            return (None,) * 8
        logprob, labels, old_logprob, advantages, ref_logprob, cu_seqlens, state = \
            ctx.saved_tensors
        glp, gent = flce.policy_loss_backward(
            logprob, labels, old_logprob, advantages, state,
            grad_loss=grad_loss.reshape(1), ref_logprob=ref_logprob,
            cu_seqlens=cu_seqlens, want_entropy=ctx.needs_input_grad[1], **ctx.options)
        return glp, gent, None, None, None, None, None, None


def policy_loss(logprob, labels, old_logprob, advantages, entropy=None, ref_logprob=None,
                cu_seqlens=None, **options):
    """(loss, stats): the clipped policy loss of ``flce.policy_loss`` (same
    arguments and options) as a 0-d fp32 tensor, and its statistics (fp32 [8],
    not differentiable). Differentiable with respect to logprob and entropy,
    e.g. the outputs of ``linear_cross_entropy(..., reduction="none")``;
    old_logprob, ref_logprob and advantages are constants."""
    flce._policy_options(**options)  # refuses what the backward could not take
    _refuse_captured_leaves(logprob, entropy)
    out = PolicyLoss.apply(logprob, entropy, labels, old_logprob, advantages, ref_logprob,
                           cu_seqlens, options)
    _note_leaves(logprob, entropy)
    return out


class PreferenceLoss(torch.autograd.Function):
    """(loss, chosen_reward, rejected_reward); see ``preference_loss``."""

    @staticmethod
    def forward(ctx, logprob, labels, cu_seqlens, ref_logprob, options):
        out = flce.preference_loss(logprob, labels, cu_seqlens, ref_logprob=ref_logprob,
                                   **options)
        ctx.save_for_backward(labels, cu_seqlens, out["seq_state"])
        ctx.options = options
        ctx.mark_non_differentiable(out["chosen_reward"], out["rejected_reward"])
        ctx.set_materialize_grads(False)
        loss = out["loss"]
        if options.get("reduction", "mean") != "none":
            loss = loss.reshape(())
        return loss, out["chosen_reward"], out["rejected_reward"]

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss, _grad_chosen, _grad_rejected):
        if grad_loss is None:
            return (None,) * 5
        labels, cu_seqlens, state = ctx.saved_tensors
        glp = flce.preference_loss_backward(
            labels, cu_seqlens, state, grad_loss=grad_loss.reshape(-1).contiguous(), **ctx.options)
        return glp, None, None, None, None


def preference_loss(logprob, labels, cu_seqlens, ref_logprob=None, **options):
    """(loss, chosen_reward, rejected_reward): the preference loss of
    ``flce.preference_loss`` (same arguments and options), 0-d or [P] under
    reduction "none", and the rewards [P] of the two sides (not
    differentiable). Differentiable with respect to logprob; ref_logprob is a
    constant."""
    flce._preference_options(**options)  # refuses what the backward could not take
    _refuse_captured_leaves(logprob)
    out = PreferenceLoss.apply(logprob, labels, cu_seqlens, ref_logprob, options)
    _note_leaves(logprob)
    return out
