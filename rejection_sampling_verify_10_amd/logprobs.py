"""Log probabilities of given tokens, with the rows' entropy and likeliest tokens, and their gradient.

The binding of ``spec_token_logprobs`` and ``spec_token_logprobs_grad`` (``include/spec_verify.h`` states what every
argument means).  After a verification:

    tokens, accept_len = verify_chain(logits, ...)                       # [B, K+1], -1 behind the emitted ones
    r = token_logprobs(logits, tokens, temperature, top_n=5)             # rows behind the emitted tokens are not read

Training a draft model on M tokens a position (ids [.., M]) and their gradients g = d loss / d log probability:

    r = token_logprobs(logits, ids)
    dlogits = token_logprobs_grad(logits, ids, r.stats, g)

or, with logits that require a gradient, through autograd: r.logprobs and r.entropy carry the graph.

    loss = -(weights * token_logprobs(logits, ids).logprobs).sum()
    loss.backward()

(A backward pass that is captured wants no eager graph of the same leaves alive, as any of PyTorch's.)
"""

from __future__ import annotations

from typing import Dict, NamedTuple, Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import SPEC_TOPK_MAX, lib
from .kvq import _CODES, _call, _scratch, _tensor


class TokenLogprobs(NamedTuple):
    logprobs: torch.Tensor                      # of the tokens' shape, float32
    entropy: torch.Tensor                       # [..], one a row, float32
    stats: torch.Tensor                         # [.., 3] float32, for token_logprobs_grad
    top_tokens: Optional[torch.Tensor]          # [.., top_n] int32, None without
    top_logprobs: Optional[torch.Tensor]        # [.., top_n] float32


def _logit_rows(t: torch.Tensor, name: str) -> Tuple[int, int, Tuple[int, ...]]:
    """(rows, elements between rows, leading shape) of logits [.., V] whose leading dimensions lie evenly in memory."""
    if t.dtype not in _CODES:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} must be [.., V]")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    rows, step = 1, t.shape[-1]
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if rows == 1:
            step = stride
        elif stride != rows * step:
            raise ValueError(f"the rows of {name} must lie at one distance from each other")
        rows *= size
    if rows > 1 and step < t.shape[-1]:
        raise ValueError(f"the rows of {name} must not overlap")
    if 0 in t.shape:
        raise ValueError(f"{name} must have at least one row")
    return rows, step, tuple(t.shape[:-1])


class _Sizes(NamedTuple):
    rows: int
    step: int                                   # elements between the logits' rows
    M: int                                      # tokens a row
    lead: Tuple[int, ...]
    workspace: int


_sizes: Dict[tuple, _Sizes] = {}                # of the calls made so far, by their shapes


def _call_sizes(logits: torch.Tensor, tokens: Optional[torch.Tensor], top_n: int) -> _Sizes:
    """What a call's shapes say, checked: tokens are of the logits' leading shape, or have a dimension of M more."""
    if logits.dtype not in _CODES:
        raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    if not logits.is_cuda:
        raise ValueError("logits must be a GPU tensor")
    key = (logits.shape, logits.stride(), logits.dtype, None if tokens is None else tokens.shape, top_n)
    s = _sizes.get(key)
    if s is None:
        rows, step, lead = _logit_rows(logits, "logits")
        if not 0 <= top_n <= SPEC_TOPK_MAX:
            raise ValueError(f"top_n must lie in [0, {SPEC_TOPK_MAX}]")
        M = 0
        if tokens is not None:
            M = 1 if tokens.dim() == len(lead) else tokens.shape[-1] if tokens.dim() else 0
            if not 1 <= M <= SPEC_TOPK_MAX:
                raise ValueError(f"tokens must have between 1 and {SPEC_TOPK_MAX} a row")
            if tuple(tokens.shape) not in (lead, lead + (M,)):
                raise ValueError(f"tokens must have shape {lead} or {lead + (M,)}, got {tuple(tokens.shape)}")
        s = _Sizes(rows, step, M, lead, token_logprobs_workspace_bytes(rows, logits.shape[-1], top_n, logits.dtype))
        if len(_sizes) >= 4096:
            _sizes.clear()
        _sizes[key] = s
    return s


def token_logprobs_workspace_bytes(rows: int, V: int, top_n: int = 0, dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of :func:`token_logprobs`'s workspace (:func:`new_workspace` makes one)."""
    return int(lib().spec_token_logprobs_workspace_bytes(rows, V, top_n, _CODES[dtype]))


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor], temperature: float = 1.0, top_n: int = 0, *,
                   workspace: Optional[torch.Tensor] = None) -> TokenLogprobs:
    """Log probabilities of ``tokens`` under softmax(logits / temperature) (``spec_token_logprobs``).

    logits [.., V] bf16 or f32 (rows at any one distance from each other); tokens int32 of the leading shape, or with
    M <= 64 a row in a last dimension, or None (every row's entropy and tops alone; logprobs is then empty).  Negative
    tokens are none, and rows without a token are not read: their log probabilities and entropy are 0, their tops -1
    and -inf.  ``workspace`` (:func:`new_workspace`; zero-filled once, calls leave it zero) avoids one a call.

    Where the logits require a gradient, logprobs and entropy pass one on (once: it has none itself); the rest does not.
    """
    if logits.requires_grad and torch.is_grad_enabled():
        return TokenLogprobs(*_Logprobs.apply(logits, tokens, temperature, top_n, workspace))
    return _forward(logits, tokens, temperature, top_n, workspace)


def _forward(logits, tokens, temperature, top_n, workspace) -> TokenLogprobs:
    top_n = int(top_n)
    rows, step, M, lead, need = _call_sizes(logits, tokens, top_n)
    V, dev = logits.shape[-1], logits.device
    f32, new = torch.float32, logits.new_empty
    tp = None if tokens is None else _tensor(tokens, "tokens", torch.int32, tokens.shape, dev)
    lp = new(lead + (0,) if tokens is None else tokens.shape, dtype=f32)
    entropy, stats = new(lead, dtype=f32), new(lead + (3,), dtype=f32)
    top = top_lp = top_ptr = top_lp_ptr = None
    if top_n:
        top, top_lp = new(lead + (top_n,), dtype=torch.int32), new(lead + (top_n,), dtype=f32)
        top_ptr, top_lp_ptr = top.data_ptr(), top_lp.data_ptr()
    wp = None
    if need:
        if workspace is None:
            workspace = torch.zeros(need + 256, dtype=torch.uint8, device=dev)
        wp, workspace = _scratch(need, dev, workspace)
    _call(lib().spec_token_logprobs, "spec_token_logprobs", dev, logits.data_ptr(), _CODES[logits.dtype], step, rows, V,
          tp, M, temperature, top_n, lp.data_ptr() if M else None, entropy.data_ptr(), stats.data_ptr(), top_ptr, top_lp_ptr,
          wp, need)
    return TokenLogprobs(lp, entropy, stats, top, top_lp)


class _Logprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature, top_n, workspace):
        r = _forward(logits, tokens, temperature, top_n, workspace)
        ctx.save_for_backward(logits, tokens, r.stats)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(*(t for t in r[2:] if t is not None))
        return tuple(r)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_lp, g_entropy, *_):
        logits, tokens, stats = ctx.saved_tensors
        if tokens is None:                      # every row's entropy alone: any token, without a gradient of its own
            tokens = torch.zeros(logits.shape[:-1], dtype=torch.int32, device=logits.device)
            g_lp = None
        if g_lp is None and g_entropy is None:
            return None, None, None, None, None
        g_lp = torch.zeros_like(tokens, dtype=torch.float32) if g_lp is None else g_lp.contiguous()
        g_entropy = None if g_entropy is None else g_entropy.contiguous()
        return token_logprobs_grad(logits, tokens, stats, g_lp, g_entropy, ctx.temperature), None, None, None, None


def token_logprobs_grad(logits: torch.Tensor, tokens: torch.Tensor, stats: torch.Tensor, grad_logprobs: torch.Tensor,
                        grad_entropy: Optional[torch.Tensor] = None, temperature: float = 1.0, *,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient for the logits (``spec_token_logprobs_grad``), of their shape and type.

    logits, tokens, temperature: as :func:`token_logprobs` had them, stats: as it gave them; grad_logprobs of the
    tokens' shape and grad_entropy of the leading one, float32.  ``out``: a tensor to write to, of any row distance;
    the logits themselves may be given, anything else must not overlap them.
    """
    rows, step, M, lead, _ = _call_sizes(logits, tokens, 0)
    dev = logits.device
    tp = _tensor(tokens, "tokens", torch.int32, tokens.shape, dev)
    out_step = logits.shape[-1]
    if out is None:
        out = logits.new_empty(logits.shape)
    elif out.dtype != logits.dtype or out.shape != logits.shape or out.device != dev:
        raise ValueError("out must have the logits' shape, type and device")
    else:
        out_step = _logit_rows(out, "out")[1]
        if not out.is_inference():
            torch.autograd.graph.increment_version(out)     # a graph that has kept it, as the logits' may, is told
    _call(lib().spec_token_logprobs_grad, "spec_token_logprobs_grad", dev, logits.data_ptr(), _CODES[logits.dtype], step,
          rows, logits.shape[-1], tp, M, _tensor(stats, "stats", torch.float32, lead + (3,), dev),
          _tensor(grad_logprobs, "grad_logprobs", torch.float32, tokens.shape, dev),
          None if grad_entropy is None else _tensor(grad_entropy, "grad_entropy", torch.float32, lead, dev),
          temperature, out.data_ptr(), out_step)
    return out
