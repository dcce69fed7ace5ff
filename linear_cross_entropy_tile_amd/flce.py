"""ctypes binding for libflce.so (declared in include/flce.h).

Two layers, both argument marshalling only:

* ``flce_workspace_size``, ``flce_forward``, ``flce_backward``,
  ``flce_forward_ex``, ``flce_backward_ex``, ``flce_get_status``, ... : one
  Python function per C entry point, same name, same arguments (device
  pointers and streams as integers, the options as ``FlceOptions``). A non-OK
  status raises ``FlceError``.
* ``forward`` / ``backward`` / ``forward_backward`` (the fused call, for
  upstream gradients known before the forward), the embedding
  (``embedding``, ``embedding_backward``), the losses between the head's
  forward and its backward (``policy_loss``, ``preference_loss``, each with
  ``_backward`` and ``_forward_backward``), what sampling needs (``logits``,
  ``process_logits``, ``process_logits_backward``) and the update
  (``grad_norm``, ``adamw_state``, ``adamw_step``): take torch CUDA tensors, check
  dtypes and layouts, allocate outputs and the workspace with torch (so
  torch's caching allocator owns all memory), and call the C entry points on
  torch's current stream. No arithmetic of the operators happens here.

The library is loaded on first use. There is no fallback: if libflce.so is
missing or the device is not a GPU, calls raise.
"""
from __future__ import annotations

import array
import ctypes
import functools
import os

__all__ = [
    "FlceError", "lib", "LIB_PATH",
    "FLCE_REDUCTION_NONE", "FLCE_REDUCTION_MEAN", "FLCE_REDUCTION_SUM",
    "FLCE_GRAD_BF16", "FLCE_GRAD_F32", "FlceOptions",
    "flce_workspace_size", "flce_forward", "flce_backward", "flce_forward_ex",
    "flce_backward_ex", "flce_fused_workspace_size", "flce_forward_backward", "flce_get_status",
    "flce_forward_noalloc", "FLCE_NOALLOC_SCRATCH_BYTES",
    "flce_status_string", "flce_version", "flce_profile_enable", "flce_profile_reset",
    "flce_profile_kinds", "flce_profile_read", "profile_table", "flce_probe_mfma_rate",
    "forward", "backward", "forward_backward", "workspace_bytes", "check_shapes",
    "FLCE_REDUCTION_SEQUENCE_MEAN", "FLCE_EMBED_VH", "FLCE_EMBED_HV",
    "FlceEmbeddingOptions", "FlcePolicyOptions", "FlcePreferenceOptions",
    "flce_embedding_workspace_size", "flce_embedding_forward", "flce_embedding_backward",
    "flce_policy_workspace_size", "flce_policy_loss_forward", "flce_policy_loss_backward",
    "flce_policy_loss_forward_backward", "flce_preference_workspace_size",
    "flce_preference_loss_forward", "flce_preference_loss_backward",
    "flce_preference_loss_forward_backward", "embedding", "embedding_backward", "policy_loss",
    "policy_loss_backward", "policy_loss_forward_backward", "preference_loss",
    "preference_loss_backward", "preference_loss_forward_backward",
    "FLCE_STATE_F32", "FLCE_STATE_8BIT", "FLCE_ROUND_NEAREST", "FLCE_ROUND_STOCHASTIC",
    "FlceProcessOptions", "FlceProcessGrads", "FlceAdamwList", "FlceAdamwOptions",
    "flce_logits_workspace_size", "flce_logits", "flce_process_workspace_size", "flce_process_logits",
    "flce_process_logits_backward", "flce_grad_norm_workspace_size", "flce_grad_norm",
    "flce_adamw_workspace_size", "flce_adamw_step", "logits", "process_logits",
    "process_logits_backward", "grad_norm", "adamw_state", "adamw_step",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libflce.so")

FLCE_REDUCTION_NONE = 0
FLCE_REDUCTION_MEAN = 1
FLCE_REDUCTION_SUM = 2
_REDUCTIONS = {"none": FLCE_REDUCTION_NONE, "mean": FLCE_REDUCTION_MEAN,
               "sum": FLCE_REDUCTION_SUM}
FLCE_GRAD_BF16 = 0
FLCE_GRAD_F32 = 1
_GRAD_DTYPES = {"bf16": FLCE_GRAD_BF16, "f32": FLCE_GRAD_F32}
FLCE_REDUCTION_SEQUENCE_MEAN = 3
_POLICY_REDUCTIONS = {"mean": FLCE_REDUCTION_MEAN, "sum": FLCE_REDUCTION_SUM,
                      "sequence_mean": FLCE_REDUCTION_SEQUENCE_MEAN}
FLCE_EMBED_VH = 0
FLCE_EMBED_HV = 1
_EMBED_LAYOUTS = {"vh": FLCE_EMBED_VH, "hv": FLCE_EMBED_HV}
_KL_ESTIMATORS = {"k1": 0, "k2": 1, "k3": 2}
_RATIO_LEVELS = {"token": 0, "sequence": 1}
_PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}
MAX_VOCAB = (1 << 22) - 256
FLCE_STATE_F32 = 0
FLCE_STATE_8BIT = 1
_STATE_DTYPES = {"f32": FLCE_STATE_F32, "8bit": FLCE_STATE_8BIT}
FLCE_ROUND_NEAREST = 0
FLCE_ROUND_STOCHASTIC = 1
_ROUNDINGS = {"nearest": FLCE_ROUND_NEAREST, "stochastic": FLCE_ROUND_STOCHASTIC}

STATUS_NAMES = {
    0: "FLCE_OK", 1: "FLCE_ERR_NULL_POINTER", 2: "FLCE_ERR_BAD_SHAPE",
    3: "FLCE_ERR_BAD_REDUCTION", 4: "FLCE_ERR_MISALIGNED",
    5: "FLCE_ERR_WORKSPACE_TOO_SMALL", 6: "FLCE_ERR_BAD_SOFTCAP", 7: "FLCE_ERR_HIP",
    8: "FLCE_ERR_INVALID_LABEL", 9: "FLCE_ERR_BAD_OPTION", 10: "FLCE_ERR_TOO_LARGE",
}
FLCE_NOALLOC_SCRATCH_BYTES = 64 << 20


class FlceOptions(ctypes.Structure):
    """flce_options_t."""
    _fields_ = [("ignore_index", ctypes.c_int64), ("softcap", ctypes.c_float),
                ("reduction", ctypes.c_int), ("z_loss_scale", ctypes.c_float),
                ("grad_dtype", ctypes.c_int), ("class_weight", ctypes.c_void_p),
                ("entropy_per_token", ctypes.c_int)]


class FlceEmbeddingOptions(ctypes.Structure):
    """flce_embedding_options_t."""
    _fields_ = [("ignore_index", ctypes.c_int64), ("scale", ctypes.c_double),
                ("layout", ctypes.c_int), ("hidden_dtype", ctypes.c_int),
                ("grad_dtype", ctypes.c_int), ("accumulate", ctypes.c_int)]


class FlcePolicyOptions(ctypes.Structure):
    """flce_policy_options_t."""
    _fields_ = [("ignore_index", ctypes.c_int64), ("clip_low", ctypes.c_double),
                ("clip_high", ctypes.c_double), ("dual_clip", ctypes.c_double),
                ("kl_coef", ctypes.c_double), ("entropy_coef", ctypes.c_double),
                ("kl_estimator", ctypes.c_int), ("level", ctypes.c_int),
                ("reduction", ctypes.c_int), ("advantages_per_sequence", ctypes.c_int)]


class FlcePreferenceOptions(ctypes.Structure):
    """flce_preference_options_t."""
    _fields_ = [("ignore_index", ctypes.c_int64), ("beta", ctypes.c_double),
                ("label_smoothing", ctypes.c_double), ("margin", ctypes.c_double),
                ("kind", ctypes.c_int), ("length_normalize", ctypes.c_int),
                ("reduction", ctypes.c_int)]



class FlceProcessOptions(ctypes.Structure):
    """flce_process_options_t."""
    _fields_ = [("ignore_index", ctypes.c_int64), ("tokens", ctypes.c_void_p),
                ("tokens_size", ctypes.c_int64), ("tokens_stride", ctypes.c_int64),
                ("offsets", ctypes.c_void_p), ("prompt_lengths", ctypes.c_void_p),
                ("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("temperatures", ctypes.c_void_p),
                ("repetition_penalty", ctypes.c_double), ("presence_penalty", ctypes.c_double),
                ("frequency_penalty", ctypes.c_double), ("temperature", ctypes.c_double),
                ("bias", ctypes.c_void_p), ("bias_stride", ctypes.c_int64),
                ("bias_tokens", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("bias_count", ctypes.c_int64), ("bias_offsets", ctypes.c_void_p),
                ("allowed", ctypes.c_void_p), ("allowed_stride", ctypes.c_int64),
                ("logits_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int)]


class FlceProcessGrads(ctypes.Structure):
    """flce_process_grads_t."""
    _fields_ = [("grad_out", ctypes.c_void_p), ("ld_grad_out", ctypes.c_int64),
                ("grad_lse", ctypes.c_void_p), ("grad_entropy", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64), ("lse", ctypes.c_void_p),
                ("entropy", ctypes.c_void_p)]


class FlceAdamwList(ctypes.Structure):
    """flce_adamw_list_t."""
    _fields_ = [("count", ctypes.c_int64)] + [(name, ctypes.c_void_p) for name in (
        "sizes", "params", "grads", "masters", "exp_avgs", "exp_avg_sqs", "exp_avg_scales",
        "exp_avg_sq_scales", "param_dtypes", "grad_dtypes")]


class FlceAdamwOptions(ctypes.Structure):
    """flce_adamw_options_t."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("state_dtype", ctypes.c_int), ("rounding", ctypes.c_int),
                ("seed", ctypes.c_uint64)]


# Every exported symbol with its (restype, argtypes).
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SIG = {
    "flce_workspace_size": (ctypes.c_int, [_I64, _I64, _I64, ctypes.c_int,
                                           ctypes.POINTER(ctypes.c_size_t),
                                           ctypes.POINTER(ctypes.c_size_t)]),
    "flce_forward": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_float,
                                    ctypes.c_int, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "flce_backward": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_float,
                                     ctypes.c_int, _P, _P, _P, _P, _P, _P, _P,
                                     ctypes.c_size_t, _P]),
    "flce_forward_noalloc": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_float,
                                            ctypes.c_int, _P, _P, _P, _P, _P, _P]),
    "flce_forward_ex": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, ctypes.POINTER(FlceOptions),
                                       _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "flce_backward_ex": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, ctypes.POINTER(FlceOptions),
                                        _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "flce_fused_workspace_size": (ctypes.c_int, [_I64, _I64, _I64, ctypes.POINTER(FlceOptions),
                                                 _I64, ctypes.POINTER(ctypes.c_size_t)]),
    "flce_forward_backward": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64,
                                             ctypes.POINTER(FlceOptions), _I64, _P, _P, _P, _P,
                                             _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t,
                                             _P]),
    "flce_forward_shard": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _I64, _I64,
                                          ctypes.POINTER(FlceOptions), _P, _P, _P,
                                          ctypes.c_size_t, _P]),
    "flce_merge_workspace_size": (ctypes.c_int, [_I64, ctypes.POINTER(ctypes.c_size_t)]),
    "flce_merge_shards": (ctypes.c_int, [_P, _P, _I64, _P, _I64, _I64, ctypes.POINTER(FlceOptions),
                                         _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "flce_backward_shard": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _I64, _I64,
                                           ctypes.POINTER(FlceOptions), _P, _P, _P, _P, _P, _P,
                                           _P, _P, _P, ctypes.c_size_t, _P]),
    "flce_embedding_workspace_size": (ctypes.c_int, [_I64, _I64, _I64,
                                                     ctypes.POINTER(FlceEmbeddingOptions),
                                                     ctypes.POINTER(ctypes.c_size_t),
                                                     ctypes.POINTER(ctypes.c_size_t)]),
    "flce_embedding_forward": (ctypes.c_int, [_P, _P, _I64, _I64, _I64, _I64, _I64,
                                              ctypes.POINTER(FlceEmbeddingOptions), _P, _P,
                                              ctypes.c_size_t, _P]),
    "flce_embedding_backward": (ctypes.c_int, [_P, _P, _I64, _I64, _I64, _I64, _I64,
                                               ctypes.POINTER(FlceEmbeddingOptions), _P, _P,
                                               ctypes.c_size_t, _P]),
    "flce_policy_workspace_size": (ctypes.c_int, [_I64, _I64, ctypes.POINTER(ctypes.c_size_t)]),
    "flce_policy_loss_forward": (ctypes.c_int, [_P] * 7 + [_I64] * 3
                                 + [ctypes.POINTER(FlcePolicyOptions), _P, _P, _P, _P,
                                    ctypes.c_size_t, _P]),
    "flce_policy_loss_backward": (ctypes.c_int, [_P] * 6 + [_I64] * 3
                                  + [ctypes.POINTER(FlcePolicyOptions), _P, _P, _P, _P, _P]),
    "flce_policy_loss_forward_backward": (ctypes.c_int, [_P] * 7 + [_I64] * 3
                                          + [ctypes.POINTER(FlcePolicyOptions), _P, _P, _P, _P, _P,
                                             _P, ctypes.c_size_t, _P]),
    "flce_preference_workspace_size": (ctypes.c_int, [_I64, _I64,
                                                      ctypes.POINTER(ctypes.c_size_t)]),
    "flce_preference_loss_forward": (ctypes.c_int, [_P] * 4 + [_I64] * 3
                                     + [ctypes.POINTER(FlcePreferenceOptions), _P, _P, _P, _P, _P,
                                        _P, ctypes.c_size_t, _P]),
    "flce_preference_loss_backward": (ctypes.c_int, [_P] * 2 + [_I64] * 3
                                      + [ctypes.POINTER(FlcePreferenceOptions), _P, _P, _P, _P]),
    "flce_preference_loss_forward_backward": (ctypes.c_int, [_P] * 4 + [_I64] * 3
                                              + [ctypes.POINTER(FlcePreferenceOptions), _P, _P, _P,
                                                 _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "flce_logits_workspace_size": (ctypes.c_int, [_I64, _I64, _I64,
                                                  ctypes.POINTER(ctypes.c_size_t)]),
    "flce_logits": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, ctypes.c_float, ctypes.c_int, _P,
                                   _I64, _P, ctypes.c_size_t, _P]),
    "flce_process_workspace_size": (ctypes.c_int, [_I64, _I64, ctypes.POINTER(ctypes.c_size_t)]),
    "flce_process_logits": (ctypes.c_int, [_P, _I64, _I64, _I64,
                                           ctypes.POINTER(FlceProcessOptions), _P, _I64, _P, _P,
                                           _P, _P, ctypes.c_size_t, _P]),
    "flce_process_logits_backward": (ctypes.c_int, [ctypes.POINTER(FlceProcessGrads), _P, _I64,
                                                    _I64, _I64,
                                                    ctypes.POINTER(FlceProcessOptions), _P, _I64,
                                                    _P, ctypes.c_size_t, _P]),
    "flce_grad_norm_workspace_size": (ctypes.c_int, [_P, _I64, ctypes.POINTER(ctypes.c_size_t)]),
    "flce_grad_norm": (ctypes.c_int, [_P, _P, _P, _I64, ctypes.c_double, _P, _P, _P,
                                      ctypes.c_size_t, _P]),
    "flce_adamw_workspace_size": (ctypes.c_size_t, []),
    "flce_adamw_step": (ctypes.c_int, [ctypes.POINTER(FlceAdamwList),
                                       ctypes.POINTER(FlceAdamwOptions), _P, _P, _P, _P,
                                       ctypes.c_size_t, _P]),
    "flce_get_status": (ctypes.c_int, [_P, ctypes.POINTER(_I64), _P]),
    "flce_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "flce_version": (ctypes.c_int, []),
    "flce_profile_enable": (ctypes.c_int, [ctypes.c_int]),
    "flce_profile_reset": (ctypes.c_int, []),
    "flce_profile_kinds": (ctypes.c_int, []),
    "flce_profile_read": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_char_p),
                                         ctypes.POINTER(_I64), ctypes.POINTER(ctypes.c_double)]),
    "flce_probe_mfma_rate": (ctypes.c_int, [ctypes.c_int, _I64, ctypes.POINTER(ctypes.c_double),
                                            _P, ctypes.c_size_t, _P]),
}


class FlceError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = STATUS_NAMES.get(status, str(status))
        try:
            text = lib().flce_status_string(status).decode()
        except Exception:  # pragma: no cover - library itself unavailable
            text = ""
        super().__init__(f"{where}: {name} ({text})")


_LIB = None


def lib():
    """The loaded libflce.so (loads it on first call)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "or python -m linear_cross_entropy_tile_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIG.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def _check(status: int, where: str) -> None:
    if status != 0:
        raise FlceError(status, where)


# ---------------------------------------------------------------- C entry points

def flce_workspace_size(N: int, H: int, V: int, reduction: int):
    f = ctypes.c_size_t(0)
    b = ctypes.c_size_t(0)
    _check(lib().flce_workspace_size(N, H, V, reduction, ctypes.byref(f), ctypes.byref(b)),
           "flce_workspace_size")
    return f.value, b.value


def flce_forward(hidden, weight, labels, N, H, V, ignore_index, softcap, reduction,
                 lse, logprob, entropy, logprob_mean, entropy_mean, workspace,
                 workspace_bytes, stream):
    _check(lib().flce_forward(hidden, weight, labels, N, H, V, ignore_index, softcap, reduction,
                              lse, logprob, entropy, logprob_mean, entropy_mean, workspace,
                              workspace_bytes, stream), "flce_forward")


def flce_forward_noalloc(hidden, weight, labels, N, H, V, ignore_index, softcap, reduction,
                         lse, logprob, entropy, logprob_mean, entropy_mean, stream):
    _check(lib().flce_forward_noalloc(hidden, weight, labels, N, H, V, ignore_index, softcap,
                                      reduction, lse, logprob, entropy, logprob_mean,
                                      entropy_mean, stream), "flce_forward_noalloc")


def flce_backward(hidden, weight, labels, N, H, V, ignore_index, softcap, reduction,
                  lse, entropy, grad_logprob, grad_entropy, grad_hidden, grad_weight,
                  workspace, workspace_bytes, stream):
    _check(lib().flce_backward(hidden, weight, labels, N, H, V, ignore_index, softcap,
                               reduction, lse, entropy, grad_logprob, grad_entropy,
                               grad_hidden, grad_weight, workspace, workspace_bytes, stream),
           "flce_backward")


def flce_forward_ex(hidden, weight, labels, N, H, V, opt, lse, logprob, entropy, uniform_ce,
                    z_loss, reduced, workspace, workspace_bytes, stream):
    _check(lib().flce_forward_ex(hidden, weight, labels, N, H, V, ctypes.byref(opt), lse,
                                 logprob, entropy, uniform_ce, z_loss, reduced, workspace,
                                 workspace_bytes, stream), "flce_forward_ex")


def flce_backward_ex(hidden, weight, labels, N, H, V, opt, lse, entropy, grad_logprob,
                     grad_entropy, grad_uniform_ce, grad_z_loss, grad_hidden, grad_weight,
                     workspace, workspace_bytes, stream):
    _check(lib().flce_backward_ex(hidden, weight, labels, N, H, V, ctypes.byref(opt), lse,
                                  entropy, grad_logprob, grad_entropy, grad_uniform_ce,
                                  grad_z_loss, grad_hidden, grad_weight, workspace,
                                  workspace_bytes, stream), "flce_backward_ex")


def flce_fused_workspace_size(N: int, H: int, V: int, opt, chunk_tokens: int = 0) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().flce_fused_workspace_size(N, H, V, ctypes.byref(opt), chunk_tokens,
                                           ctypes.byref(b)), "flce_fused_workspace_size")
    return b.value


def flce_forward_backward(hidden, weight, labels, N, H, V, opt, chunk_tokens, grad_logprob,
                          grad_entropy, grad_uniform_ce, grad_z_loss, lse, logprob, entropy,
                          uniform_ce, z_loss, reduced, grad_hidden, grad_weight, workspace,
                          workspace_bytes, stream):
    _check(lib().flce_forward_backward(hidden, weight, labels, N, H, V, ctypes.byref(opt),
                                       chunk_tokens, grad_logprob, grad_entropy, grad_uniform_ce,
                                       grad_z_loss, lse, logprob, entropy, uniform_ce, z_loss,
                                       reduced, grad_hidden, grad_weight, workspace,
                                       workspace_bytes, stream), "flce_forward_backward")


def flce_forward_shard(hidden, weight_shard, labels, N, H, Vs, v_begin, V_total, opt, state,
                       label_logit, workspace, workspace_bytes, stream):
    _check(lib().flce_forward_shard(hidden, weight_shard, labels, N, H, Vs, v_begin, V_total,
                                    ctypes.byref(opt), state, label_logit, workspace,
                                    workspace_bytes, stream), "flce_forward_shard")


def flce_merge_workspace_size(N: int) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().flce_merge_workspace_size(N, ctypes.byref(b)), "flce_merge_workspace_size")
    return b.value


def flce_merge_shards(states, label_logits, S, labels, N, V_total, opt, lse, logprob, entropy,
                      uniform_ce, z_loss, reduced, workspace, workspace_bytes, stream):
    _check(lib().flce_merge_shards(states, label_logits, S, labels, N, V_total, ctypes.byref(opt),
                                   lse, logprob, entropy, uniform_ce, z_loss, reduced, workspace,
                                   workspace_bytes, stream), "flce_merge_shards")


def flce_backward_shard(hidden, weight_shard, labels, N, H, Vs, v_begin, V_total, opt, lse,
                        entropy, grad_logprob, grad_entropy, grad_uniform_ce, grad_z_loss,
                        grad_hidden_partial, grad_weight_shard, workspace, workspace_bytes,
                        stream):
    _check(lib().flce_backward_shard(hidden, weight_shard, labels, N, H, Vs, v_begin, V_total,
                                     ctypes.byref(opt), lse, entropy, grad_logprob, grad_entropy,
                                     grad_uniform_ce, grad_z_loss, grad_hidden_partial,
                                     grad_weight_shard, workspace, workspace_bytes, stream),
           "flce_backward_shard")


def flce_embedding_workspace_size(N: int, H: int, Vs: int, opt):
    f = ctypes.c_size_t(0)
    b = ctypes.c_size_t(0)
    _check(lib().flce_embedding_workspace_size(N, H, Vs, ctypes.byref(opt), ctypes.byref(f),
                                               ctypes.byref(b)), "flce_embedding_workspace_size")
    return f.value, b.value


def flce_embedding_forward(weight, tokens, N, H, Vs, v_begin, V_total, opt, hidden, workspace,
                           workspace_bytes, stream):
    _check(lib().flce_embedding_forward(weight, tokens, N, H, Vs, v_begin, V_total,
                                        ctypes.byref(opt), hidden, workspace, workspace_bytes,
                                        stream), "flce_embedding_forward")


def flce_embedding_backward(grad_hidden, tokens, N, H, Vs, v_begin, V_total, opt, grad_weight,
                            workspace, workspace_bytes, stream):
    _check(lib().flce_embedding_backward(grad_hidden, tokens, N, H, Vs, v_begin, V_total,
                                         ctypes.byref(opt), grad_weight, workspace,
                                         workspace_bytes, stream), "flce_embedding_backward")


def flce_policy_workspace_size(N: int, B: int) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().flce_policy_workspace_size(N, B, ctypes.byref(b)), "flce_policy_workspace_size")
    return b.value


def flce_policy_loss_forward(logprob, entropy, old_logprob, ref_logprob, advantages, labels,
                             cu_seqlens, N, B, V, opt, loss, stats, seq_state, workspace,
                             workspace_bytes, stream):
    _check(lib().flce_policy_loss_forward(logprob, entropy, old_logprob, ref_logprob, advantages,
                                          labels, cu_seqlens, N, B, V, ctypes.byref(opt), loss,
                                          stats, seq_state, workspace, workspace_bytes, stream),
           "flce_policy_loss_forward")


def flce_policy_loss_backward(logprob, old_logprob, ref_logprob, advantages, labels, cu_seqlens,
                              N, B, V, opt, seq_state, grad_loss, grad_logprob, grad_entropy,
                              stream):
    _check(lib().flce_policy_loss_backward(logprob, old_logprob, ref_logprob, advantages, labels,
                                           cu_seqlens, N, B, V, ctypes.byref(opt), seq_state,
                                           grad_loss, grad_logprob, grad_entropy, stream),
           "flce_policy_loss_backward")


def flce_policy_loss_forward_backward(logprob, entropy, old_logprob, ref_logprob, advantages,
                                      labels, cu_seqlens, N, B, V, opt, grad_loss, loss,
                                      stats, grad_logprob, grad_entropy, workspace,
                                      workspace_bytes, stream):
    _check(lib().flce_policy_loss_forward_backward(logprob, entropy, old_logprob, ref_logprob,
                                                   advantages, labels, cu_seqlens, N, B, V,
                                                   ctypes.byref(opt), grad_loss, loss, stats,
                                                   grad_logprob, grad_entropy, workspace,
                                                   workspace_bytes, stream),
           "flce_policy_loss_forward_backward")


def flce_preference_workspace_size(N: int, P: int) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().flce_preference_workspace_size(N, P, ctypes.byref(b)),
           "flce_preference_workspace_size")
    return b.value


def flce_preference_loss_forward(logprob, ref_logprob, labels, cu_seqlens, N, P, V, opt, loss,
                                 pair_loss, chosen_reward, rejected_reward, seq_state, workspace,
                                 workspace_bytes, stream):
    _check(lib().flce_preference_loss_forward(logprob, ref_logprob, labels, cu_seqlens, N, P, V,
                                              ctypes.byref(opt), loss, pair_loss, chosen_reward,
                                              rejected_reward, seq_state, workspace,
                                              workspace_bytes, stream),
           "flce_preference_loss_forward")


def flce_preference_loss_backward(labels, cu_seqlens, N, P, V, opt, seq_state, grad_loss,
                                  grad_logprob, stream):
    _check(lib().flce_preference_loss_backward(labels, cu_seqlens, N, P, V, ctypes.byref(opt),
                                               seq_state, grad_loss, grad_logprob, stream),
           "flce_preference_loss_backward")


def flce_preference_loss_forward_backward(logprob, ref_logprob, labels, cu_seqlens, N, P, V, opt,
                                          grad_loss, loss, pair_loss, chosen_reward,
                                          rejected_reward, grad_logprob, workspace,
                                          workspace_bytes, stream):
    _check(lib().flce_preference_loss_forward_backward(logprob, ref_logprob, labels, cu_seqlens,
                                                       N, P, V, ctypes.byref(opt), grad_loss,
                                                       loss, pair_loss, chosen_reward,
                                                       rejected_reward, grad_logprob, workspace,
                                                       workspace_bytes, stream),
           "flce_preference_loss_forward_backward")


def flce_logits_workspace_size(N: int, H: int, V: int) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().flce_logits_workspace_size(N, H, V, ctypes.byref(b)),
           "flce_logits_workspace_size")
    return b.value


def flce_logits(hidden, weight, bias, N, H, V, softcap, out_dtype, out, ld_out, workspace,
                workspace_bytes, stream):
    _check(lib().flce_logits(hidden, weight, bias, N, H, V, softcap, out_dtype, out, ld_out,
                             workspace, workspace_bytes, stream), "flce_logits")


def flce_process_workspace_size(N: int, V: int) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().flce_process_workspace_size(N, V, ctypes.byref(b)),
           "flce_process_workspace_size")
    return b.value


def flce_process_logits(logits, ld, N, V, opt, out, ld_out, lse, entropy, greedy, workspace,
                        workspace_bytes, stream):
    _check(lib().flce_process_logits(logits, ld, N, V, ctypes.byref(opt), out, ld_out, lse,
                                     entropy, greedy, workspace, workspace_bytes, stream),
           "flce_process_logits")


def flce_process_logits_backward(grads, logits, ld, N, V, opt, grad_logits, ld_grad, workspace,
                                 workspace_bytes, stream):
    _check(lib().flce_process_logits_backward(ctypes.byref(grads), logits, ld, N, V,
                                              ctypes.byref(opt), grad_logits, ld_grad, workspace,
                                              workspace_bytes, stream),
           "flce_process_logits_backward")


def flce_grad_norm_workspace_size(sizes, count: int) -> int:
    """sizes: a ctypes array of int64, or its address."""
    b = ctypes.c_size_t(0)
    _check(lib().flce_grad_norm_workspace_size(sizes, count, ctypes.byref(b)),
           "flce_grad_norm_workspace_size")
    return b.value


def flce_grad_norm(grads, sizes, dtypes, count, max_norm, norm, scale, workspace, workspace_bytes,
                   stream):
    _check(lib().flce_grad_norm(grads, sizes, dtypes, count, max_norm, norm, scale, workspace,
                                workspace_bytes, stream), "flce_grad_norm")


def flce_adamw_workspace_size() -> int:
    return lib().flce_adamw_workspace_size()


def flce_adamw_step(tensors, opt, lr_device, grad_scale, step, workspace, workspace_bytes,
                    stream):
    _check(lib().flce_adamw_step(ctypes.byref(tensors), ctypes.byref(opt), lr_device, grad_scale,
                                 step, workspace, workspace_bytes, stream), "flce_adamw_step")


def flce_get_status(workspace, stream) -> int:
    """Number of invalid labels (or tokens) the last call on this workspace saw (syncs)."""
    n = _I64(0)
    st = lib().flce_get_status(workspace, ctypes.byref(n), stream)
    if st not in (0, 8):
        _check(st, "flce_get_status")
    return n.value


def flce_status_string(status: int) -> str:
    return lib().flce_status_string(status).decode()


def flce_version() -> int:
    return lib().flce_version()


def flce_profile_enable(enable: bool) -> None:
    _check(lib().flce_profile_enable(1 if enable else 0), "flce_profile_enable")


def flce_profile_reset() -> None:
    _check(lib().flce_profile_reset(), "flce_profile_reset")


def flce_profile_kinds() -> int:
    return lib().flce_profile_kinds()


def flce_profile_read(kind: int):
    name = ctypes.c_char_p()
    n = _I64(0)
    ms = ctypes.c_double(0.0)
    _check(lib().flce_profile_read(kind, ctypes.byref(name), ctypes.byref(n), ctypes.byref(ms)),
           "flce_profile_read")
    return name.value.decode(), n.value, ms.value


PROBE_REGISTERS, PROBE_ZEROS, PROBE_LDS, PROBE_LDS_DMA = 0, 1, 2, 3


def flce_probe_mfma_rate(mode, steps: int, workspace, workspace_bytes, stream) -> float:
    """Sustained bf16 MFMA TFLOP/s of the GEMM wave tile (synchronises the
    stream). mode: PROBE_REGISTERS (or False), PROBE_ZEROS (or True),
    PROBE_LDS, PROBE_LDS_DMA; see include/flce.h."""
    t = ctypes.c_double(0.0)
    _check(lib().flce_probe_mfma_rate(int(mode), steps, ctypes.byref(t), workspace,
                                      workspace_bytes, stream), "flce_probe_mfma_rate")
    return t.value


def profile_table() -> dict:
    """{kernel kind: (launches, total ms)} for kinds launched at least once."""
    out = {}
    for k in range(flce_profile_kinds()):
        name, n, ms = flce_profile_read(k)
        if n:
            out[name] = (n, ms)
    return out


# ---------------------------------------------------------------- torch marshalling

def _torch():
    import torch
    return torch


def _stream():
    return _torch().cuda.current_stream().cuda_stream


def _require(t, dtype, ndim, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor")


def check_shapes(hidden, weight, labels, *per_token) -> None:
    """Raises ValueError unless hidden [N,H], weight [H,V], labels [N] and
    each (name, tensor) pair of ``per_token`` ([N] each; None skipped) agree
    in size: the kernels read them by those extents."""
    N, H = hidden.shape
    if weight.dim() != 2 or weight.shape[0] != H or labels.shape[0] != N:
        raise ValueError("shape mismatch among hidden [N,H], weight [H,V], labels [N]")
    for name, t in per_token:
        if t is not None and (t.dim() != 1 or t.shape[0] != N):
            raise ValueError(f"{name} must have N = {N} elements")


def _entropy_per_token(reduction: str, entropy_reduction) -> int:
    if entropy_reduction is None or entropy_reduction == reduction:
        return 0
    if entropy_reduction != "none":
        raise ValueError("entropy_reduction must be None, 'none' or the reduction itself")
    return 1


def workspace_bytes(N: int, H: int, V: int, reduction: str = "none"):
    return flce_workspace_size(N, H, V, _REDUCTIONS[reduction])


_OUT_NAMES = ("logprob", "entropy", "uniform_ce", "z_loss")


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _check_class_weight(cw, V):
    if cw is not None:
        _require(cw, _torch().float32, 1, "class_weight")
        if cw.shape[0] != V:
            raise ValueError("class_weight must have one weight per class (V)")


def forward(hidden, weight, labels, ignore_index: int = -100, softcap: float = 0.0,
            reduction: str = "none", z_loss_scale: float = 0.0, aux: bool = False,
            class_weight=None, workspace=None) -> dict:
    """lse, logprob, entropy [N] (fp32); with ``aux`` also uniform_ce and
    z_loss [N]; under "mean" / "sum" the reductions as ``<name>_mean`` /
    ``<name>_sum`` (fp32 [1]).

    hidden: bf16 [N,H]; weight: bf16 [H,V]; labels: int64 [N];
    class_weight: optional fp32 [V] target weights of the "mean" / "sum"
    reductions. Without aux, z-loss, "sum" and class weights this calls
    flce_forward, else flce_forward_ex.
    """
    torch = _torch()
    _require(hidden, torch.bfloat16, 2, "hidden")
    _require(weight, torch.bfloat16, 2, "weight")
    _require(labels, torch.int64, 1, "labels")
    check_shapes(hidden, weight, labels)
    N, H = hidden.shape
    V = weight.shape[1]
    red = _REDUCTIONS[reduction]
    fbytes, _ = flce_workspace_size(N, H, V, red)
    if workspace is None or workspace.numel() < fbytes:
        workspace = torch.empty(max(fbytes, 256), dtype=torch.uint8, device=hidden.device)
    dev = hidden.device
    f32 = dict(dtype=torch.float32, device=dev)
    lse = torch.empty(N, **f32)
    lp = torch.empty(N, **f32)
    ent = torch.empty(N, **f32)
    out = {"lse": lse, "logprob": lp, "entropy": ent, "workspace": workspace}
    _check_class_weight(class_weight, V)
    extended = aux or z_loss_scale != 0.0 or red == FLCE_REDUCTION_SUM or class_weight is not None
    if not extended:
        lpm = entm = None
        if red == FLCE_REDUCTION_MEAN:
            lpm = torch.empty(1, **f32)
            entm = torch.empty(1, **f32)
            out["logprob_mean"] = lpm
            out["entropy_mean"] = entm
        flce_forward(hidden.data_ptr(), weight.data_ptr(), labels.data_ptr(), N, H, V,
                     int(ignore_index), float(softcap), red, lse.data_ptr(), lp.data_ptr(),
                     ent.data_ptr(), _ptr(lpm), _ptr(entm), workspace.data_ptr(),
                     workspace.numel(), _stream())
        return out
    uce = torch.empty(N, **f32) if aux else None
    zl = torch.empty(N, **f32) if aux else None
    reduced = torch.empty(4, **f32) if red != FLCE_REDUCTION_NONE else None
    opt = FlceOptions(int(ignore_index), float(softcap), red, float(z_loss_scale), FLCE_GRAD_BF16,
                      _ptr(class_weight))
    flce_forward_ex(hidden.data_ptr(), weight.data_ptr(), labels.data_ptr(), N, H, V, opt,
                    lse.data_ptr(), lp.data_ptr(), ent.data_ptr(), _ptr(uce), _ptr(zl),
                    _ptr(reduced), workspace.data_ptr(), workspace.numel(), _stream())
    if aux:
        out["uniform_ce"] = uce
        out["z_loss"] = zl
    if reduced is not None:
        for k, name in enumerate(_OUT_NAMES):
            out[f"{name}_{reduction}"] = reduced[k:k + 1]
    return out


def _check_grads(grads, N, red, reduction, ept):
    torch = _torch()
    for g, name in grads:
        if g is not None:
            _require(g, torch.float32, 1, name)
            want = N if (red == FLCE_REDUCTION_NONE or (ept and name == "grad_entropy")) else 1
            if g.shape[0] != want:
                raise ValueError(f"{name} must have {want} element(s) under '{reduction}'")


def backward(hidden, weight, labels, lse, entropy, grad_logprob=None, grad_entropy=None,
             ignore_index: int = -100, softcap: float = 0.0, reduction: str = "none",
             grad_uniform_ce=None, grad_z_loss=None, z_loss_scale: float = 0.0,
             grad_dtype: str = "bf16", class_weight=None, entropy_reduction=None,
             workspace=None):
    """(grad_hidden [N,H], grad_weight [H,V]), bf16 or fp32 (``grad_dtype``).

    Upstream gradients: fp32 [N] under "none", fp32 [1] under "mean" and
    "sum", or None for zero; with ``entropy_reduction="none"`` under "mean" /
    "sum" the entropy's gradient is per token [N] (the entropy taken
    unreduced beside the reduced logprob; options field entropy_per_token).
    class_weight as for ``forward``. Without the auxiliary gradients, z-loss,
    "sum", class weights, a per-token entropy and fp32 outputs this calls
    flce_backward, else flce_backward_ex.
    """
    torch = _torch()
    _require(hidden, torch.bfloat16, 2, "hidden")
    _require(weight, torch.bfloat16, 2, "weight")
    _require(labels, torch.int64, 1, "labels")
    _require(lse, torch.float32, 1, "lse")
    _require(entropy, torch.float32, 1, "entropy")
    check_shapes(hidden, weight, labels, ("lse", lse), ("entropy", entropy))
    N, H = hidden.shape
    V = weight.shape[1]
    red = _REDUCTIONS[reduction]
    gdt = _GRAD_DTYPES[grad_dtype]
    ept = _entropy_per_token(reduction, entropy_reduction)
    grads = ((grad_logprob, "grad_logprob"), (grad_entropy, "grad_entropy"),
             (grad_uniform_ce, "grad_uniform_ce"), (grad_z_loss, "grad_z_loss"))
    _check_grads(grads, N, red, reduction, ept)
    _, bbytes = flce_workspace_size(N, H, V, red)
    if workspace is None or workspace.numel() < bbytes:
        workspace = torch.empty(max(bbytes, 256), dtype=torch.uint8, device=hidden.device)
    odt = torch.float32 if gdt == FLCE_GRAD_F32 else torch.bfloat16
    gh = torch.empty((N, H), dtype=odt, device=hidden.device)
    gw = torch.empty((H, V), dtype=odt, device=hidden.device)
    _check_class_weight(class_weight, V)
    extended = (grad_uniform_ce is not None or grad_z_loss is not None or z_loss_scale != 0.0
                or red == FLCE_REDUCTION_SUM or gdt != FLCE_GRAD_BF16 or class_weight is not None
                or ept)
    if not extended:
        flce_backward(hidden.data_ptr(), weight.data_ptr(), labels.data_ptr(), N, H, V,
                      int(ignore_index), float(softcap), red, lse.data_ptr(), entropy.data_ptr(),
                      _ptr(grad_logprob), _ptr(grad_entropy), gh.data_ptr(), gw.data_ptr(),
                      workspace.data_ptr(), workspace.numel(), _stream())
        return gh, gw
    opt = FlceOptions(int(ignore_index), float(softcap), red, float(z_loss_scale), gdt,
                      _ptr(class_weight), ept)
    flce_backward_ex(hidden.data_ptr(), weight.data_ptr(), labels.data_ptr(), N, H, V, opt,
                     lse.data_ptr(), entropy.data_ptr(), _ptr(grad_logprob), _ptr(grad_entropy),
                     _ptr(grad_uniform_ce), _ptr(grad_z_loss), gh.data_ptr(), gw.data_ptr(),
                     workspace.data_ptr(), workspace.numel(), _stream())
    return gh, gw


def forward_backward(hidden, weight, labels, grad_logprob=None, grad_entropy=None,
                     ignore_index: int = -100, softcap: float = 0.0, reduction: str = "none",
                     grad_uniform_ce=None, grad_z_loss=None, z_loss_scale: float = 0.0,
                     grad_dtype: str = "bf16", aux: bool = False, chunk_tokens: int = 0,
                     class_weight=None, entropy_reduction=None, workspace=None) -> dict:
    """The fused forward + backward (flce_forward_backward): the outputs of
    ``forward`` and, under "grad_hidden" / "grad_weight", the gradients of
    ``backward`` for upstream gradients known before the call (fp32 [N] under
    "none", [1] under "mean" and "sum", None for zero; entropy_reduction as
    for ``backward``).
    """
    torch = _torch()
    _require(hidden, torch.bfloat16, 2, "hidden")
    _require(weight, torch.bfloat16, 2, "weight")
    _require(labels, torch.int64, 1, "labels")
    check_shapes(hidden, weight, labels)
    N, H = hidden.shape
    V = weight.shape[1]
    red = _REDUCTIONS[reduction]
    gdt = _GRAD_DTYPES[grad_dtype]
    ept = _entropy_per_token(reduction, entropy_reduction)
    grads = ((grad_logprob, "grad_logprob"), (grad_entropy, "grad_entropy"),
             (grad_uniform_ce, "grad_uniform_ce"), (grad_z_loss, "grad_z_loss"))
    _check_grads(grads, N, red, reduction, ept)
    _check_class_weight(class_weight, V)
    opt = FlceOptions(int(ignore_index), float(softcap), red, float(z_loss_scale), gdt,
                      _ptr(class_weight), ept)
    nbytes = flce_fused_workspace_size(N, H, V, opt, int(chunk_tokens))
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=hidden.device)
    dev = hidden.device
    f32 = dict(dtype=torch.float32, device=dev)
    odt = torch.float32 if gdt == FLCE_GRAD_F32 else torch.bfloat16
    out = {"lse": torch.empty(N, **f32), "logprob": torch.empty(N, **f32),
           "entropy": torch.empty(N, **f32), "workspace": workspace,
           "grad_hidden": torch.empty((N, H), dtype=odt, device=dev),
           "grad_weight": torch.empty((H, V), dtype=odt, device=dev)}
    uce = torch.empty(N, **f32) if aux else None
    zl = torch.empty(N, **f32) if aux else None
    reduced = torch.empty(4, **f32) if red != FLCE_REDUCTION_NONE else None
    flce_forward_backward(hidden.data_ptr(), weight.data_ptr(), labels.data_ptr(), N, H, V, opt,
                          int(chunk_tokens), _ptr(grad_logprob), _ptr(grad_entropy),
                          _ptr(grad_uniform_ce), _ptr(grad_z_loss), out["lse"].data_ptr(),
                          out["logprob"].data_ptr(), out["entropy"].data_ptr(), _ptr(uce),
                          _ptr(zl), _ptr(reduced), out["grad_hidden"].data_ptr(),
                          out["grad_weight"].data_ptr(), workspace.data_ptr(), workspace.numel(),
                          _stream())
    if aux:
        out["uniform_ce"] = uce
        out["z_loss"] = zl
    if reduced is not None:
        for k, name in enumerate(_OUT_NAMES):
            out[f"{name}_{reduction}"] = reduced[k:k + 1]
    return out


# ---- beside the head: embedding, policy loss, preference loss

def _call(dev, name, *args) -> None:
    """The C entry point ``name``(*args, stream) on torch's current stream of
    ``dev``, with that device current (ctypes passes an options structure by
    reference)."""
    torch = _torch()
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    f = getattr(_LIB or lib(), name)
    if torch.cuda.current_device() == dev.index:
        status = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = f(*args, stream)
    if status != 0:
        raise FlceError(status, name)


def _check_devices(dev, *named) -> None:
    for name, t in named:
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")


# Sizes depend on nothing but their arguments.
_policy_bytes = functools.lru_cache(maxsize=256)(flce_policy_workspace_size)
_preference_bytes = functools.lru_cache(maxsize=256)(flce_preference_workspace_size)


def _choice(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}, got {value!r}")
    return table[value]


def _workspace(workspace, nbytes, dev):
    """``workspace`` when it is large enough, else a new one."""
    torch = _torch()
    if workspace is not None:
        _require(workspace, torch.uint8, 1, "workspace")
        _check_devices(dev, ("workspace", workspace))
        if workspace.numel() >= nbytes:
            return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)


@functools.lru_cache(maxsize=256)
def _embedding_bytes(N, H, V, layout):
    return flce_embedding_workspace_size(N, H, V, FlceEmbeddingOptions(0, 1.0, layout, 0, 0, 0))


def _require_grad_dtype(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name} must be a bf16 or fp32 tensor")
    _require(t, t.dtype, 2, name)
    return FLCE_GRAD_F32 if t.dtype == torch.float32 else FLCE_GRAD_BF16


def embedding(weight, tokens, layout: str = "hv", scale: float = 1.0, ignore_index: int = -100,
              v_begin: int = 0, v_total=None, workspace=None) -> dict:
    """{"hidden": bf16 [N,H], "workspace"}: hidden_i = scale * E[tokens_i].

    weight: bf16, the head's [H,V] under layout "hv" (tied embeddings) or a
    table [V,H] under "vh"; tokens: int64 [N]. Tokens equal to ignore_index or
    outside the vocabulary give zero rows; the latter are counted
    (flce_get_status on the workspace). With a vocabulary slice [v_begin,
    v_begin + V) of v_total ids, tokens of other slices give zero rows.
    """
    torch = _torch()
    _require(weight, torch.bfloat16, 2, "weight")
    _require(tokens, torch.int64, 1, "tokens")
    dev = weight.device
    _check_devices(dev, ("tokens", tokens))
    lay = _choice(_EMBED_LAYOUTS, layout, "layout")
    H, V = weight.shape if lay == FLCE_EMBED_HV else (weight.shape[1], weight.shape[0])
    N = tokens.shape[0]
    opt = FlceEmbeddingOptions(int(ignore_index), float(scale), lay, FLCE_GRAD_BF16,
                               FLCE_GRAD_BF16, 0)
    nbytes, _ = _embedding_bytes(N, H, V, lay)
    workspace = _workspace(workspace, nbytes, dev)
    hidden = torch.empty((N, H), dtype=torch.bfloat16, device=dev)
    _call(dev, "flce_embedding_forward", weight.data_ptr(), tokens.data_ptr(), N, H, V,
          int(v_begin), V if v_total is None else int(v_total), opt, hidden.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return {"hidden": hidden, "workspace": workspace}


def embedding_backward(grad_hidden, tokens, vocab_size: int, layout: str = "hv",
                       scale: float = 1.0, ignore_index: int = -100, v_begin: int = 0,
                       v_total=None, grad_dtype: str = "bf16", grad_weight=None, workspace=None):
    """grad_weight [H,V] ("hv") or [V,H] ("vh"), V = vocab_size (the slice's ids).

    grad_hidden: bf16 or fp32 [N,H]; tokens and the options as for
    ``embedding``. Without grad_weight a new tensor of ``grad_dtype`` is
    returned, zero for ids that do not occur. With grad_weight (bf16 or fp32,
    e.g. the head's gradient of a tied weight, from ``backward``) the gradient
    is added to it in place and it is returned.
    """
    torch = _torch()
    hdt = _require_grad_dtype(grad_hidden, "grad_hidden")
    _require(tokens, torch.int64, 1, "tokens")
    N, H = grad_hidden.shape
    if tokens.shape[0] != N:
        raise ValueError(f"tokens must have N = {N} elements")
    dev = grad_hidden.device
    _check_devices(dev, ("tokens", tokens), ("grad_weight", grad_weight))
    lay = _choice(_EMBED_LAYOUTS, layout, "layout")
    gdt = _choice(_GRAD_DTYPES, grad_dtype, "grad_dtype")
    V = int(vocab_size)
    shape = (H, V) if lay == FLCE_EMBED_HV else (V, H)
    accumulate = grad_weight is not None
    if accumulate:
        gdt = _require_grad_dtype(grad_weight, "grad_weight")
        if tuple(grad_weight.shape) != shape:
            raise ValueError(f"grad_weight must be {list(shape)}")
    opt = FlceEmbeddingOptions(int(ignore_index), float(scale), lay, hdt, gdt,
                               1 if accumulate else 0)
    _, nbytes = _embedding_bytes(N, H, V, lay)
    workspace = _workspace(workspace, nbytes, dev)
    if not accumulate:
        grad_weight = torch.empty(shape, device=dev, dtype=torch.float32 if gdt == FLCE_GRAD_F32
                                  else torch.bfloat16)
    _call(dev, "flce_embedding_backward", grad_hidden.data_ptr(), tokens.data_ptr(), N, H, V,
          int(v_begin), V if v_total is None else int(v_total), opt, grad_weight.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return grad_weight


def _check_vector(t, dtype, size, index, name) -> None:
    """``t`` must be a contiguous 1-d tensor of ``size`` elements on device
    ``index`` (these calls are made once a step on small batches, where the
    checks count)."""
    try:
        if (t.dtype is dtype and t.is_cuda and t.dim() == 1 and t.numel() == size
                and t.is_contiguous() and t.get_device() == index):
            return
    except AttributeError:
        pass
    _require(t, dtype, 1, name)
    if t.numel() != size:
        raise ValueError(f"{name} must have {size} element(s)")
    raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _sequences(labels, cu_seqlens):
    """(device, N, number of sequences) after checking both tensors."""
    torch = _torch()
    _require(labels, torch.int64, 1, "labels")
    dev = labels.device
    if cu_seqlens is None:
        return dev, labels.numel(), 1
    _require(cu_seqlens, torch.int64, 1, "cu_seqlens")
    _check_devices(dev, ("cu_seqlens", cu_seqlens))
    if cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must have one element more than there are sequences")
    return dev, labels.numel(), cu_seqlens.numel() - 1


def _policy_options(clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, kl_estimator="k3",
                    entropy_coef=0.0, level="token", reduction="mean", ignore_index=-100,
                    vocab_size=None, advantages_per_sequence=False):
    return (FlcePolicyOptions(int(ignore_index), float(clip_low), float(clip_high),
                              float(dual_clip), float(kl_coef), float(entropy_coef),
                              _choice(_KL_ESTIMATORS, kl_estimator, "kl_estimator"),
                              _choice(_RATIO_LEVELS, level, "level"),
                              _choice(_POLICY_REDUCTIONS, reduction, "reduction"),
                              1 if advantages_per_sequence else 0),
            MAX_VOCAB if vocab_size is None else int(vocab_size))


def _policy_check(opt, logprob, labels, old_logprob, advantages, entropy, ref_logprob, cu_seqlens,
                  grad_loss):
    """(device, N, B) of a policy call, after checking its tensors."""
    dev, N, B = _sequences(labels, cu_seqlens)
    f32, index = _torch().float32, dev.index
    if opt.kl_coef != 0.0 and ref_logprob is None:
        raise ValueError("kl_coef needs ref_logprob")
    if opt.level == 1 and (cu_seqlens is None or not opt.advantages_per_sequence):
        raise ValueError("level 'sequence' needs cu_seqlens and advantages_per_sequence")
    _check_vector(logprob, f32, N, index, "logprob")
    _check_vector(old_logprob, f32, N, index, "old_logprob")
    _check_vector(advantages, f32, B if opt.advantages_per_sequence else N, index, "advantages")
    if ref_logprob is not None:
        _check_vector(ref_logprob, f32, N, index, "ref_logprob")
    if entropy is not None:
        _check_vector(entropy, f32, N, index, "entropy")
    if grad_loss is not None:
        _check_vector(grad_loss, f32, 1, index, "grad_loss")
    return dev, N, B


def policy_loss(logprob, labels, old_logprob, advantages, entropy=None, ref_logprob=None,
                cu_seqlens=None, workspace=None, **options) -> dict:
    """The clipped policy loss with a KL term (flce_policy_loss_forward), from
    the head's per-token logprob (and entropy).

    logprob, old_logprob, ref_logprob, entropy: fp32 [N]; labels: int64 [N];
    cu_seqlens: int64 [B+1] sequence offsets, None for one sequence of all
    tokens; advantages: fp32 [N], or [B] with advantages_per_sequence.

    Options: clip_low = clip_high = 0.2, dual_clip = 0 (off), kl_coef = 0 (needs
    ref_logprob otherwise), kl_estimator = "k1" | "k2" | "k3" (default),
    entropy_coef = 0 (needs entropy otherwise), level = "token" (default) or
    "sequence" ratios, reduction = "mean" over the valid tokens (default),
    "sum" or "sequence_mean" (the mean over sequences of their token means),
    ignore_index = -100 and vocab_size (None: the library's limit; labels
    outside [0, vocab_size) mark tokens without a loss, as ignore_index does),
    advantages_per_sequence = False.

    Returns loss (fp32 [1]), stats (fp32 [8]: loss, policy term, kl, entropy,
    share of clipped tokens, estimate of KL(old || new), valid tokens,
    sequences with a valid token), seq_state (for ``policy_loss_backward``) and
    workspace.
    """
    torch = _torch()
    opt, V = _policy_options(**options)
    dev, N, B = _policy_check(opt, logprob, labels, old_logprob, advantages, entropy, ref_logprob,
                              cu_seqlens, None)
    if opt.entropy_coef != 0.0 and entropy is None:
        raise ValueError("entropy_coef needs entropy")
    workspace = _workspace(workspace, _policy_bytes(N, B), dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    stats = torch.empty(8, dtype=torch.float32, device=dev)
    state = torch.empty((B + 1, 2), dtype=torch.float64, device=dev)
    _call(dev, "flce_policy_loss_forward", logprob.data_ptr(), _ptr(entropy),
          old_logprob.data_ptr(), _ptr(ref_logprob), advantages.data_ptr(), labels.data_ptr(),
          _ptr(cu_seqlens), N, B, V, opt, loss.data_ptr(), stats.data_ptr(), state.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return {"loss": loss, "stats": stats, "seq_state": state, "workspace": workspace}


def policy_loss_backward(logprob, labels, old_logprob, advantages, seq_state, grad_loss=None,
                         ref_logprob=None, cu_seqlens=None, want_entropy: bool = True,
                         **options):
    """(grad_logprob, grad_entropy), fp32 [N] each (grad_entropy None unless
    want_entropy), of grad_loss (fp32 [1], None for 1) times the loss; inputs,
    options and seq_state of the matching ``policy_loss``."""
    torch = _torch()
    opt, V = _policy_options(**options)
    dev, N, B = _policy_check(opt, logprob, labels, old_logprob, advantages, None, ref_logprob,
                              cu_seqlens, grad_loss)
    _require(seq_state, torch.float64, 2, "seq_state")
    if tuple(seq_state.shape) != (B + 1, 2):
        raise ValueError(f"seq_state must be [{B + 1}, 2]")
    _check_devices(dev, ("seq_state", seq_state))
    glp = torch.empty(N, dtype=torch.float32, device=dev)
    gent = torch.empty(N, dtype=torch.float32, device=dev) if want_entropy else None
    _call(dev, "flce_policy_loss_backward", logprob.data_ptr(), old_logprob.data_ptr(),
          _ptr(ref_logprob), advantages.data_ptr(), labels.data_ptr(), _ptr(cu_seqlens), N, B, V,
          opt, seq_state.data_ptr(), _ptr(grad_loss), glp.data_ptr(), _ptr(gent))
    return glp, gent


def policy_loss_forward_backward(logprob, labels, old_logprob, advantages, grad_loss=None,
                                 entropy=None, ref_logprob=None, cu_seqlens=None, workspace=None,
                                 **options) -> dict:
    """``policy_loss`` (same inputs and options) and its gradients in one call,
    for an upstream gradient known before it (grad_loss fp32 [1], None for 1):
    loss, stats, workspace, grad_logprob (fp32 [N]) and, with entropy,
    grad_entropy (fp32 [N]), ready for the head's ``backward`` under reduction
    "none"."""
    torch = _torch()
    opt, V = _policy_options(**options)
    dev, N, B = _policy_check(opt, logprob, labels, old_logprob, advantages, entropy, ref_logprob,
                              cu_seqlens, grad_loss)
    if opt.entropy_coef != 0.0 and entropy is None:
        raise ValueError("entropy_coef needs entropy")
    workspace = _workspace(workspace, _policy_bytes(N, B), dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    stats = torch.empty(8, dtype=torch.float32, device=dev)
    glp = torch.empty(N, dtype=torch.float32, device=dev)
    out = {"loss": loss, "stats": stats, "workspace": workspace, "grad_logprob": glp}
    gent = None
    if entropy is not None:
        gent = out["grad_entropy"] = torch.empty(N, dtype=torch.float32, device=dev)
    _call(dev, "flce_policy_loss_forward_backward", logprob.data_ptr(), _ptr(entropy),
          old_logprob.data_ptr(), _ptr(ref_logprob), advantages.data_ptr(), labels.data_ptr(),
          _ptr(cu_seqlens), N, B, V, opt, _ptr(grad_loss), loss.data_ptr(), stats.data_ptr(),
          glp.data_ptr(), _ptr(gent), workspace.data_ptr(), workspace.numel())
    return out


def _preference_options(kind="sigmoid", beta=0.1, label_smoothing=0.0, margin=0.0,
                        length_normalize=False, reduction="mean", ignore_index=-100,
                        vocab_size=None):
    return (FlcePreferenceOptions(int(ignore_index), float(beta), float(label_smoothing),
                                  float(margin), _choice(_PREFERENCE_KINDS, kind, "kind"),
                                  1 if length_normalize else 0,
                                  _choice(_REDUCTIONS, reduction, "reduction")),
            MAX_VOCAB if vocab_size is None else int(vocab_size))


def _preference_check(opt, labels, cu_seqlens, grad_loss, arrays):
    """(device, N, P) of a preference call, after checking its tensors (arrays:
    (name, fp32 [N] tensor or None))."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    dev, N, B = _sequences(labels, cu_seqlens)
    if B % 2 != 0:
        raise ValueError("cu_seqlens must hold an even number of sequences: the chosen ones, "
                         "then the rejected ones")
    P = B // 2
    f32, index = _torch().float32, dev.index
    for name, t in arrays:
        if t is not None:
            _check_vector(t, f32, N, index, name)
    if grad_loss is not None:
        _check_vector(grad_loss, f32, P if opt.reduction == FLCE_REDUCTION_NONE else 1, index,
                      "grad_loss")
    return dev, N, P


def _pair_outputs(P, dev, reduction):
    """The outputs of a preference call: (loss pointer, dict)."""
    torch = _torch()
    pair, chosen, rejected = (torch.empty(P, dtype=torch.float32, device=dev) for _ in range(3))
    loss = (None if reduction == FLCE_REDUCTION_NONE
            else torch.empty(1, dtype=torch.float32, device=dev))
    return _ptr(loss), {"loss": pair if loss is None else loss, "pair_loss": pair,
                        "chosen_reward": chosen, "rejected_reward": rejected}


def preference_loss(logprob, labels, cu_seqlens, ref_logprob=None, workspace=None,
                    **options) -> dict:
    """The preference loss over P pairs (flce_preference_loss_forward), from
    the head's per-token logprob.

    logprob, ref_logprob (None: no reference): fp32 [N]; labels: int64 [N];
    cu_seqlens: int64 [2P+1] offsets of the P chosen and then the P rejected
    sequences; pair i is the sequences i and P + i.

    Options: kind = "sigmoid" (default), "hinge" or "ipo", beta = 0.1,
    label_smoothing = 0 (sigmoid only), margin = 0 (not for ipo),
    length_normalize = False, reduction = "mean" over the pairs (default),
    "sum" or "none", ignore_index = -100 and vocab_size as for ``policy_loss``.

    Returns loss (fp32 [1], or [P] under "none"), pair_loss [P], chosen_reward
    [P], rejected_reward [P], seq_state (for ``preference_loss_backward``) and
    workspace.
    """
    torch = _torch()
    opt, V = _preference_options(**options)
    _require(logprob, torch.float32, 1, "logprob")
    dev, N, P = _preference_check(opt, labels, cu_seqlens, None,
                                  (("logprob", logprob), ("ref_logprob", ref_logprob)))
    workspace = _workspace(workspace, _preference_bytes(N, P), dev)
    loss, out = _pair_outputs(P, dev, opt.reduction)
    state = torch.empty(2 * P + 1, dtype=torch.float64, device=dev)
    _call(dev, "flce_preference_loss_forward", logprob.data_ptr(), _ptr(ref_logprob),
          labels.data_ptr(), cu_seqlens.data_ptr(), N, P, V, opt, loss,
          out["pair_loss"].data_ptr(), out["chosen_reward"].data_ptr(),
          out["rejected_reward"].data_ptr(), state.data_ptr(), workspace.data_ptr(),
          workspace.numel())
    out.update(seq_state=state, workspace=workspace)
    return out


def preference_loss_backward(labels, cu_seqlens, seq_state, grad_loss=None, **options):
    """grad_logprob (fp32 [N]) of grad_loss (fp32 [1], or [P] under reduction
    "none"; None for ones) times the loss; inputs, options and seq_state of the
    matching ``preference_loss``."""
    torch = _torch()
    opt, V = _preference_options(**options)
    dev, N, P = _preference_check(opt, labels, cu_seqlens, grad_loss, ())
    _require(seq_state, torch.float64, 1, "seq_state")
    if seq_state.shape[0] != 2 * P + 1:
        raise ValueError(f"seq_state must have {2 * P + 1} elements")
    _check_devices(dev, ("seq_state", seq_state))
    glp = torch.empty(N, dtype=torch.float32, device=dev)
    _call(dev, "flce_preference_loss_backward", labels.data_ptr(), cu_seqlens.data_ptr(), N, P, V,
          opt, seq_state.data_ptr(), _ptr(grad_loss), glp.data_ptr())
    return glp


def preference_loss_forward_backward(logprob, labels, cu_seqlens, grad_loss=None,
                                     ref_logprob=None, workspace=None, **options) -> dict:
    """``preference_loss`` (same inputs and options) and its gradient in one
    call, for an upstream gradient known before it (grad_loss as for
    ``preference_loss_backward``): loss, pair_loss, chosen_reward,
    rejected_reward, grad_logprob (fp32 [N]) and workspace."""
    torch = _torch()
    opt, V = _preference_options(**options)
    _require(logprob, torch.float32, 1, "logprob")
    dev, N, P = _preference_check(opt, labels, cu_seqlens, grad_loss,
                                  (("logprob", logprob), ("ref_logprob", ref_logprob)))
    workspace = _workspace(workspace, _preference_bytes(N, P), dev)
    loss, out = _pair_outputs(P, dev, opt.reduction)
    glp = torch.empty(N, dtype=torch.float32, device=dev)
    _call(dev, "flce_preference_loss_forward_backward", logprob.data_ptr(), _ptr(ref_logprob),
          labels.data_ptr(), cu_seqlens.data_ptr(), N, P, V, opt, _ptr(grad_loss), loss,
          out["pair_loss"].data_ptr(), out["chosen_reward"].data_ptr(),
          out["rejected_reward"].data_ptr(), glp.data_ptr(), workspace.data_ptr(),
          workspace.numel())
    out.update(grad_logprob=glp, workspace=workspace)
    return out


# ---- the two ends of a training step: logits to sample from, the update

def _rows(t, dtypes, name):
    """(N, V, row stride) of a 2-d tensor whose rows are dense; they may lie
    apart, as in a slice of a wider tensor."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-d tensor with dense rows")
    N, V = t.shape
    if N <= 1:
        return N, V, V
    if t.stride(0) < V:
        raise ValueError(f"the rows of {name} must not overlap")
    return N, V, t.stride(0)


def _torch_dtype(code):
    torch = _torch()
    return torch.float32 if code == FLCE_GRAD_F32 else torch.bfloat16


def _written(tensors) -> None:
    """Tells autograd that a call has written to these tensors: a graph that saved
    one of them refuses its backward."""
    torch = _torch()
    torch.autograd.graph.increment_version([t for t in tensors if not t.is_inference()])


def _out_rows(out, N, V, dtype, dev, name="out"):
    """(out or a new [N,V] tensor, row stride)."""
    torch = _torch()
    if out is None:
        return torch.empty((N, V), dtype=dtype, device=dev), V
    n, v, ld = _rows(out, (dtype,), name)
    if (n, v) != (N, V):
        raise ValueError(f"{name} must be [{N}, {V}]")
    _check_devices(dev, (name, out))
    return out, ld


def logits(hidden, weight, bias=None, softcap: float = 0.0, out_dtype: str = "f32", out=None,
           workspace=None) -> dict:
    """{"logits": [N,V], "workspace"}: the head's logits of a few rows (at most
    1024), e.g. the last positions of the sequences that are being generated.

    hidden: bf16 [N,H]; weight: bf16 [H,V]; bias: fp32 [V] or None; softcap: 0
    or less for none. The result is fp32 or (out_dtype "bf16") bf16; with out
    (of that type, rows may lie apart) it is written there.
    """
    torch = _torch()
    _require(hidden, torch.bfloat16, 2, "hidden")
    _require(weight, torch.bfloat16, 2, "weight")
    N, H = hidden.shape
    if weight.shape[0] != H:
        raise ValueError("shape mismatch between hidden [N,H] and weight [H,V]")
    V = weight.shape[1]
    dev = hidden.device
    _check_devices(dev, ("weight", weight))
    if bias is not None:
        _check_vector(bias, torch.float32, V, dev.index, "bias")
    odt = _choice(_GRAD_DTYPES, out_dtype, "out_dtype")
    given = out is not None
    out, ld = _out_rows(out, N, V, _torch_dtype(odt), dev)
    workspace = _workspace(workspace, _logits_bytes(N, H, V), dev)
    _call(dev, "flce_logits", hidden.data_ptr(), weight.data_ptr(), _ptr(bias), N, H, V,
          float(softcap), odt, out.data_ptr(), ld, workspace.data_ptr(), workspace.numel())
    if given:
        _written([out])
    return {"logits": out, "workspace": workspace}


_logits_bytes = functools.lru_cache(maxsize=256)(flce_logits_workspace_size)
_process_bytes = functools.lru_cache(maxsize=256)(flce_process_workspace_size)


def _process_options(x, out_dtype, tokens=None, cu_seqlens=None, lengths=None,
                     prompt_lengths=None, repetition_penalty=1.0, presence_penalty=0.0,
                     frequency_penalty=0.0, temperature=1.0, bias=None, bias_tokens=None,
                     bias_values=None, bias_cu_seqlens=None, allowed=None, ignore_index=-100):
    """(N, V, row stride, FlceProcessOptions) for logits x, after checking the
    tensors."""
    torch = _torch()
    f32, i64 = torch.float32, torch.int64
    N, V, ld = _rows(x, (torch.bfloat16, f32), "logits")
    dev = x.device
    index = dev.index
    o = FlceProcessOptions()
    o.ignore_index = int(ignore_index)
    if tokens is None:
        if cu_seqlens is not None or lengths is not None or prompt_lengths is not None:
            raise ValueError("cu_seqlens, lengths and prompt_lengths need tokens")
    else:
        padded = isinstance(tokens, torch.Tensor) and tokens.dim() == 2
        _require(tokens, i64, 2 if padded else 1, "tokens")
        _check_devices(dev, ("tokens", tokens))
        if padded:
            if lengths is None or cu_seqlens is not None:
                raise ValueError("tokens [N, L] need lengths [N] (and no cu_seqlens)")
            if tokens.shape[0] != N:
                raise ValueError(f"tokens must have {N} rows")
            _check_vector(lengths, i64, N, index, "lengths")
            offsets = lengths
        else:
            if cu_seqlens is None or lengths is not None:
                raise ValueError("packed tokens need cu_seqlens [N+1] (and no lengths)")
            _check_vector(cu_seqlens, i64, N + 1, index, "cu_seqlens")
            offsets = cu_seqlens
        if prompt_lengths is not None:
            _check_vector(prompt_lengths, i64, N, index, "prompt_lengths")
            o.prompt_lengths = prompt_lengths.data_ptr()
        # Rows of no tokens have no address, nor do their lengths say anything.
        if not padded or tokens.shape[1] > 0:
            o.tokens = tokens.data_ptr() or offsets.data_ptr()
            o.tokens_size = tokens.numel()
            o.tokens_stride = tokens.shape[1] if padded else 0
            o.offsets = offsets.data_ptr()
    for value, array, scalar in ((repetition_penalty, "repetition", "repetition_penalty"),
                                 (presence_penalty, "presence", "presence_penalty"),
                                 (frequency_penalty, "frequency", "frequency_penalty"),
                                 (temperature, "temperatures", "temperature")):
        one = 1.0 if scalar in ("repetition_penalty", "temperature") else 0.0
        if isinstance(value, torch.Tensor):
            _check_vector(value, f32, N, index, scalar)
            setattr(o, array, value.data_ptr())
            setattr(o, scalar, one)
        else:
            setattr(o, scalar, float(value))
    if bias is not None:
        if isinstance(bias, torch.Tensor) and bias.dim() == 2:
            n, v, stride = _rows(bias, (f32,), "bias")
            if (n, v) != (N, V):
                raise ValueError(f"bias must be [{V}] or [{N}, {V}]")
            _check_devices(dev, ("bias", bias))
            o.bias_stride = stride
        else:
            _check_vector(bias, f32, V, index, "bias")
        o.bias = bias.data_ptr()
    listed = (bias_tokens, bias_values, bias_cu_seqlens)
    if any(t is not None for t in listed):
        if any(t is None for t in listed):
            raise ValueError("listed biases are bias_tokens, bias_values and bias_cu_seqlens")
        _require(bias_tokens, i64, 1, "bias_tokens")
        _check_devices(dev, ("bias_tokens", bias_tokens))
        _check_vector(bias_values, f32, bias_tokens.numel(), index, "bias_values")
        _check_vector(bias_cu_seqlens, i64, N + 1, index, "bias_cu_seqlens")
        o.bias_tokens, o.bias_values = bias_tokens.data_ptr(), bias_values.data_ptr()
        o.bias_count, o.bias_offsets = bias_tokens.numel(), bias_cu_seqlens.data_ptr()
    if allowed is not None:
        words = -(-V // 32)
        if isinstance(allowed, torch.Tensor) and allowed.dim() == 2:
            n, w, stride = _rows(allowed, (torch.int32,), "allowed")
            if n != N or w < words:
                raise ValueError(f"allowed must be [{words}] or [{N}, {words}]")
            _check_devices(dev, ("allowed", allowed))
            o.allowed_stride = stride
        else:
            _require(allowed, torch.int32, 1, "allowed")
            if allowed.numel() < words:
                raise ValueError(f"allowed must be [{words}] or [{N}, {words}]")
            _check_devices(dev, ("allowed", allowed))
        o.allowed = allowed.data_ptr()
    o.logits_dtype = FLCE_GRAD_F32 if x.dtype == f32 else FLCE_GRAD_BF16
    o.out_dtype = o.logits_dtype if out_dtype is None else _choice(_GRAD_DTYPES, out_dtype,
                                                                   "out_dtype")
    return N, V, ld, o


def process_logits(logits, out_dtype=None, out=None, workspace=None, **options) -> dict:
    """Penalties, biases, temperature and mask on logits (flce_process_logits):
    {"logits": [N,V], "lse": fp32 [N], "entropy": fp32 [N], "greedy": int64 [N],
    "workspace"}.

    logits: bf16 or fp32 [N,V] (rows may lie apart), e.g. of ``logits``. The
    result has their type or out_dtype ("f32" | "bf16"); out may be logits
    itself, and shares no memory with it otherwise. In row i a logit x of id v becomes
      x / repetition if x > 0, else x * repetition   (v anywhere in the history)
      x - frequency * n - (presence if n)            (n: v's count past the prompt)
      x + bias[v] + the row's listed biases of v
      x / temperature                                (0: unscaled)
      -inf                                           (v not allowed)
    in this order; lse, entropy and greedy (the first largest id, -1 if nothing
    is allowed) are those of the returned row, so that logits[i, t] - lse[i] is
    the log-probability with which token t is drawn.

    Options: the rows' histories as tokens (int64, packed) with cu_seqlens
    (int64 [N+1]), or as tokens [N, L] with lengths (int64 [N], not looked at if
    L is 0), at most 2**31 - 1 tokens a row; prompt_lengths
    (int64 [N], None for 0); repetition_penalty = 1, presence_penalty = 0,
    frequency_penalty = 0 and temperature = 1, numbers or fp32 [N]; bias (fp32
    [V] or [N,V]); bias_tokens (int64 [K]), bias_values (fp32 [K]) and
    bias_cu_seqlens (int64 [N+1]), a list of biases a row, of which those of one
    id add up; allowed (int32 [V/32 rounded up], or [N, ...]: id v is allowed if
    bit v % 32 of word v // 32 is set); ignore_index = -100. Tokens that are
    neither ignore_index nor an id are passed over and counted
    (flce_get_status on the workspace), in histories if there is a penalty. A
    row whose offsets are bad counts as one, and its outputs are NaN and -1.
    """
    torch = _torch()
    N, V, ld, opt = _process_options(logits, out_dtype, **options)
    dev = logits.device
    given = out is not None
    out, ld_out = _out_rows(out, N, V, _torch_dtype(opt.out_dtype), dev)
    workspace = _workspace(workspace, _process_bytes(N, V), dev)
    stats = torch.empty((2, N), dtype=torch.float32, device=dev)
    greedy = torch.empty(N, dtype=torch.int64, device=dev)
    lse, entropy = stats[0], stats[1]
    _call(dev, "flce_process_logits", logits.data_ptr(), ld, N, V, opt, out.data_ptr(), ld_out,
          lse.data_ptr(), entropy.data_ptr(), greedy.data_ptr(), workspace.data_ptr(),
          workspace.numel())
    if given:
        _written([out])
    return {"logits": out, "lse": lse, "entropy": entropy, "greedy": greedy,
            "workspace": workspace}


def process_logits_backward(grad_out, logits, processed=None, lse=None, entropy=None,
                            grad_lse=None, grad_entropy=None, out_dtype=None, out=None,
                            workspace=None, **options):
    """Gradient [N,V] (type of logits) of ``process_logits`` with respect to the
    logits, for the upstream gradients grad_out [N,V] of the returned logits
    (None for zero) and grad_lse and grad_entropy (fp32 [N], None for zero) of
    lse and entropy; the latter two need processed, lse and entropy, the
    "logits", "lse" and "entropy" that the call returned. logits and options are
    those of the call (logits as they were before it); without grad_out and
    processed, out_dtype too. out may be grad_out itself, if the types agree."""
    torch = _torch()
    f32, both = torch.float32, (torch.bfloat16, torch.float32)
    g = FlceProcessGrads()
    for t in (grad_out, processed):
        if isinstance(t, torch.Tensor) and t.dtype in both:
            out_dtype = "f32" if t.dtype == f32 else "bf16"
    N, V, ld, opt = _process_options(logits, out_dtype, **options)
    dev = logits.device
    for t, name, pointer, stride in ((grad_out, "grad_out", "grad_out", "ld_grad_out"),
                                     (processed, "processed", "out", "ld_out")):
        if t is not None:
            n, v, rows = _rows(t, (_torch_dtype(opt.out_dtype),), name)
            if (n, v) != (N, V):
                raise ValueError(f"{name} must be [{N}, {V}]")
            _check_devices(dev, (name, t))
            setattr(g, pointer, t.data_ptr())
            setattr(g, stride, rows)
    for t, name in ((lse, "lse"), (entropy, "entropy"), (grad_lse, "grad_lse"),
                    (grad_entropy, "grad_entropy")):
        if t is not None:
            _check_vector(t, f32, N, dev.index, name)
            setattr(g, name, t.data_ptr())
    if (grad_lse is not None or grad_entropy is not None) and (processed is None or lse is None):
        raise ValueError("grad_lse and grad_entropy need processed and lse")
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs entropy")
    given = out is not None
    out, ld_grad = _out_rows(out, N, V, logits.dtype, dev)
    workspace = _workspace(workspace, _process_bytes(N, V), dev)
    _call(dev, "flce_process_logits_backward", g, logits.data_ptr(), ld, N, V, opt,
          out.data_ptr(), ld_grad, workspace.data_ptr(), workspace.numel())
    if given:
        _written([out])
    return out


def _tensors(ts, dtypes, name, like=None, sizes=None):
    """Checks a list of dense tensors of one device, of the types ``dtypes`` (a
    set): (device, sizes, their types)."""
    torch = _torch()
    if not isinstance(ts, (list, tuple)):
        raise ValueError(f"{name} must be a list of tensors")
    if sizes is not None and len(ts) != len(sizes):
        raise ValueError(f"{name} must have {len(sizes)} tensors, got {len(ts)}")
    if len(ts) == 0:
        return like, [], set()
    T = torch.Tensor
    try:  # lists are long and steps short: no loop of Python's own where all is well
        numel = list(map(T.numel, ts))
        kinds = {t.dtype for t in ts}
        dev = like if like is not None else ts[0].device
        if (kinds <= dtypes and all(map(T.is_contiguous, ts)) and dev.type == "cuda"
                and set(map(T.get_device, ts)) == {dev.index}
                and (sizes is None or numel == sizes)):
            return dev, numel, kinds
    except (TypeError, AttributeError):
        pass
    dev = like
    for i, t in enumerate(ts):
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
            raise ValueError(f"{name}[{i}] must be a CUDA (HIP) tensor")
        if t.dtype not in dtypes:
            raise ValueError(f"{name}[{i}] must be {' or '.join(sorted(map(str, dtypes)))}, "
                             f"got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous")
        if dev is None:
            dev = t.device
        if t.device != dev:
            raise ValueError(f"{name}[{i}] must be on {dev}, got {t.device}")
        if sizes is not None and t.numel() != sizes[i]:
            raise ValueError(f"{name}[{i}] must have {sizes[i]} elements, got {t.numel()}")
    raise ValueError(f"{name}: not a list of dense tensors")


def _addresses(ts):
    return array.array("Q", map(_torch().Tensor.data_ptr, ts))


def _dtype_codes(ts, kinds):
    """FLCE_GRAD_* of each tensor; kinds: their types."""
    f32 = _torch().float32
    if len(kinds) <= 1:
        return array.array("i", [FLCE_GRAD_F32 if f32 in kinds else FLCE_GRAD_BF16]) * len(ts)
    return array.array("i", [FLCE_GRAD_F32 if t.dtype is f32 else FLCE_GRAD_BF16 for t in ts])


def grad_norm(grads, max_norm: float = 0.0, workspace=None) -> dict:
    """{"norm": fp32 [1], "scale": fp32 [1], "workspace"}: the 2-norm over all
    values of a list of dense bf16 or fp32 tensors (summed in float64), and the
    factor min(1, max_norm / norm) that clips it (1 without max_norm, NaN if a
    value is not finite), for ``adamw_step``'s grad_scale. Both stay on the
    device."""
    torch = _torch()
    dev, sizes, kinds = _tensors(grads, {torch.bfloat16, torch.float32}, "grads")
    if dev is None:
        raise ValueError("grads must have a tensor")
    n = len(sizes)
    pointers, csizes = _addresses(grads), array.array("q", sizes)
    dtypes = _dtype_codes(grads, kinds)
    psizes = csizes.buffer_info()[0]
    workspace = _workspace(workspace, flce_grad_norm_workspace_size(psizes, n), dev)
    both = torch.empty(2, dtype=torch.float32, device=dev)
    norm, scale = both[:1], both[1:]
    _call(dev, "flce_grad_norm", pointers.buffer_info()[0], psizes, dtypes.buffer_info()[0], n,
          float(max_norm), norm.data_ptr(), scale.data_ptr(), workspace.data_ptr(),
          workspace.numel())
    return {"norm": norm, "scale": scale, "workspace": workspace}


STATE_BLOCK = 256


def adamw_state(params, state: str = "f32", master: bool = False) -> dict:
    """The state of ``adamw_step`` for a list of dense bf16 or fp32 tensors:
    step (int64 [1], 0) and, one tensor a parameter each, exp_avg and exp_avg_sq
    of its shape (fp32, or under "8bit" torch.float8_e4m3fn codes, exp_avg_sq's
    of the second moment's root), exp_avg_scale and exp_avg_sq_scale ("8bit":
    fp32, one factor for each 256 values; None otherwise), all 0, and with
    ``master`` master, an fp32 copy of each bf16 parameter (None for fp32 ones;
    without it the whole list is None)."""
    torch = _torch()
    kind = _choice(_STATE_DTYPES, state, "state")
    dev, sizes, _ = _tensors(params, {torch.bfloat16, torch.float32}, "params")
    if dev is None:
        raise ValueError("params must have a tensor")
    dtype = torch.float32 if kind == FLCE_STATE_F32 else torch.float8_e4m3fn

    def zeros():
        return [torch.zeros(p.shape, dtype=dtype, device=dev) for p in params]

    def scales():
        return ([torch.zeros(-(-n // STATE_BLOCK), dtype=torch.float32, device=dev)
                 for n in sizes] if kind == FLCE_STATE_8BIT else None)

    return {"step": torch.zeros(1, dtype=torch.int64, device=dev),
            "exp_avg": zeros(), "exp_avg_sq": zeros(),
            "exp_avg_scale": scales(), "exp_avg_sq_scale": scales(),
            "master": [p.detach().float() if p.dtype == torch.bfloat16 else None
                       for p in params] if master else None}


def adamw_step(params, grads, state, lr=1e-3, beta1: float = 0.9, beta2: float = 0.999,
               eps: float = 1e-8, weight_decay: float = 0.01, grad_scale=None,
               rounding: str = "nearest", seed: int = 0, workspace=None) -> None:
    """One AdamW step over a list of tensors, in place (flce_adamw_step).

    params and grads: dense bf16 or fp32 tensors of the same sizes, the types in
    any mixture; state: of ``adamw_state``, updated in place, its step raised by
    one; no two tensors of params and state share memory. lr: a number, or fp32
    [1] on the device (a captured step then follows it). eps: 0 or at least
    2**-126. grad_scale: fp32 [1] that the gradients are multiplied by, e.g.
    ``grad_norm``'s scale; if it is not finite, nothing is changed (without one, a
    gradient that is not finite makes its weight NaN and loses its states, in 8
    bits those of its block of 256). Under rounding "stochastic" bf16 parameters
    without a master copy and 8-bit states are rounded up with the probability of
    the part cut off, by a hash of seed, the step, the tensor's place in the list
    and the value's in the tensor (lists updated one by one take different seeds).
    """
    torch = _torch()
    f32 = torch.float32
    both = {torch.bfloat16, f32}
    dev, sizes, pkinds = _tensors(params, both, "params")
    if dev is None:
        raise ValueError("params must have a tensor")
    gkinds = _tensors(grads, both, "grads", dev, sizes)[2]
    m, v = state["exp_avg"], state["exp_avg_sq"]
    ms, vs, master = state["exp_avg_scale"], state["exp_avg_sq_scale"], state["master"]
    eight = ms is not None
    sdt = {torch.float8_e4m3fn if eight else f32}
    _tensors(m, sdt, "state exp_avg", dev, sizes)
    _tensors(v, sdt, "state exp_avg_sq", dev, sizes)
    lists = [array.array("q", sizes), _addresses(params), _addresses(grads), None, _addresses(m),
             _addresses(v), None, None, _dtype_codes(params, pkinds), _dtype_codes(grads, gkinds)]
    if eight:
        blocks = [-(-n // STATE_BLOCK) for n in sizes]
        _tensors(ms, {f32}, "state exp_avg_scale", dev, blocks)
        _tensors(vs, {f32}, "state exp_avg_sq_scale", dev, blocks)
        lists[6:8] = _addresses(ms), _addresses(vs)
    if master is not None:
        if len(master) != len(sizes):
            raise ValueError(f"state master must have {len(sizes)} entries")
        own = [(t, n) for t, n in zip(master, sizes) if t is not None]
        _tensors([t for t, _ in own], {f32}, "state master", dev, [n for _, n in own])
        if f32 in pkinds and any(t is not None and p.dtype == f32
                                 for t, p in zip(master, params)):
            raise ValueError("state master: fp32 parameters have no copy")
        lists[3] = array.array("Q", [0 if t is None else t.data_ptr() for t in master])
    # Two of the written tensors at one address would be updated at once. (No values, no
    # address.)
    written = array.array("Q")
    for a in (lists[1], *lists[3:8]):
        if a is not None:
            written += a
    if len(set(written)) < len(written) - max(0, written.count(0) - 1):
        raise ValueError("params and state: the same tensor twice")
    step = state["step"]
    _check_vector(step, torch.int64, 1, dev.index, "state step")
    lr_device = None
    if isinstance(lr, torch.Tensor):
        _check_vector(lr, f32, 1, dev.index, "lr")
        lr_device, lr = lr, 0.0
    if grad_scale is not None:
        _check_vector(grad_scale, f32, 1, dev.index, "grad_scale")
    opt = FlceAdamwOptions(float(lr), float(beta1), float(beta2), float(eps),
                           float(weight_decay), FLCE_STATE_8BIT if eight else FLCE_STATE_F32,
                           _choice(_ROUNDINGS, rounding, "rounding"), int(seed) & (1 << 64) - 1)
    table = FlceAdamwList(len(sizes), *[None if a is None else a.buffer_info()[0] for a in lists])
    workspace = _workspace(workspace, _ADAMW_BYTES, dev)
    _call(dev, "flce_adamw_step", table, opt, _ptr(lr_device), _ptr(grad_scale),
          step.data_ptr(), workspace.data_ptr(), workspace.numel())
    _written(params if master is None else [*params, *(t for t in master if t is not None)])


_ADAMW_BYTES = 512  # flce_adamw_workspace_size()
