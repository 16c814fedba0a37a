"""Attention with modified scores: capped by a tanh, biased by distance, masked
by causality, a window, documents or a prefix, with grouped heads.

``mask_plan`` turns the mask into a plan on the device (one interval of keys per
query); ``mod_fwd`` and ``mod_bwd`` are the forward and backward pass over it,
``mod_attention`` their differentiable form.  Argument marshalling only: see
include/fa.h for the definitions, layouts and limits.
"""
from __future__ import annotations

from dataclasses import dataclass
from functools import lru_cache
from typing import Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _check, _need, _need_shape, _need_workspace, _on, _same_device, _scale, _stream_ptr, lib

__all__ = ["MaskPlan", "mask_plan", "mod_fwd", "mod_bwd", "mod_bwd_workspace_size", "mod_attention"]

_INT_MAX = 2**31 - 1


@dataclass(frozen=True)
class MaskPlan:
    """Which keys each query sees, for batches of B entries of N tokens: made by
    mask_plan, read by mod_fwd and mod_bwd of every layer and head."""
    data: torch.Tensor
    B: int
    N: int


def _window(window: int) -> int:
    w = int(window)
    if w != window or not 0 <= w <= _INT_MAX:
        raise ValueError(f"window must be an integer in [0, {_INT_MAX}] (0: no window), got {window}")
    return w


def _softcap(softcap: Optional[float]) -> float:
    c = 0.0 if softcap is None else float(softcap)
    if not 0.0 <= c < float("inf"):
        raise ValueError(f"softcap must be finite and >= 0 (0: no cap), got {softcap}")
    return c


def _slopes(slopes, H: int):
    if slopes is not None:
        _need_shape(slopes, "slopes", torch.float32, (H,))
        if slopes.requires_grad:
            raise ValueError("slopes are constants of the attention: they get no gradient (detach them)")


def mask_plan(B: int, N: int, causal: bool = False, window: int = 0, doc_ids: Optional[torch.Tensor] = None,
              prefix: Optional[torch.Tensor] = None, device=None) -> MaskPlan:
    """The plan of a mask over N tokens in each of B batch entries.

    doc_ids int32 [B, N]: a query sees the run of equal ids around it; negative
    ids are padding.  causal: only keys at or before the query.  prefix int32
    [B], with causal: the first prefix[b] tokens see each other in both
    directions and are seen by all later ones.  window > 0: only keys closer
    than that.  device: where to make it (that of the tensors given, else the
    current CUDA device)."""
    B, N, window = int(B), int(N), _window(window)
    if doc_ids is not None:
        _need_shape(doc_ids, "doc_ids", torch.int32, (B, N))
    if prefix is not None:
        _need_shape(prefix, "prefix", torch.int32, (B,))
    L = lib()
    need = L.fa_mask_plan_size(B, N)
    if need == 0:
        raise ValueError(f"no mask plan for B = {B}, N = {N}")
    if device is None:
        like = doc_ids if doc_ids is not None else prefix
        device = like.device if like is not None else torch.device("cuda", torch.cuda.current_device())
    data = torch.empty(need, dtype=torch.uint8, device=device)
    _same_device(data, doc_ids, prefix)
    with _on(data):
        st = L.fa_mask_plan(data.data_ptr(), need, None if doc_ids is None else doc_ids.data_ptr(),
                            None if prefix is None else prefix.data_ptr(), B, N, window, int(bool(causal)),
                            _stream_ptr(data))
    _check(st, "fa_mask_plan")
    return MaskPlan(data, B, N)


@lru_cache(maxsize=256)
def _plan_size(B: int, N: int) -> int:
    return int(lib().fa_mask_plan_size(B, N))


def _need_plan(plan, B: int, N: int):
    """`plan` must be mask_plan's for this B and N: the kernels index its bytes from
    the sizes of q."""
    if not isinstance(plan, MaskPlan):
        raise TypeError("plan must come from mask_plan")
    if (plan.B, plan.N) != (B, N):
        raise ValueError(f"the plan is for B = {plan.B}, N = {plan.N}, not for B = {B}, N = {N}")
    need = _plan_size(B, N)
    t = plan.data
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.uint8 and t.dim() == 1 and t.is_contiguous()
            and t.shape[0] >= need):
        raise ValueError(f"the plan's data must be the bytes that mask_plan wrote: contiguous uint8 of {need} or more")


def _sizes(q, k, v, plan):
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 4)
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, N, Hkv, d) or Hkv < 1 or H % Hkv != 0:
        raise ValueError(f"k must be [{B}, {N}, Hkv, {d}] with Hkv dividing {H}, got {tuple(k.shape)}")
    _need_shape(v, "v", torch.bfloat16, k.shape)
    _need_plan(plan, B, N)
    return B, N, H, Hkv, d


def mod_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, plan: MaskPlan, softcap: float = 0.0,
            slopes: Optional[torch.Tensor] = None, scale: Optional[float] = None, low: bool = False, out=None,
            lse=None, out_low=None):
    """O, LSE of q [B, N, H, d] with k, v [B, N, Hkv, d] under the plan's mask.

    softcap > 0 caps the scores, slopes (fp32 [H]) lowers them with distance.
    low=True (or an out_low buffer): also returns the part of O that its bf16
    rounding loses, for mod_bwd."""
    B, N, H, Hkv, d = _sizes(q, k, v, plan)
    softcap = _softcap(softcap)
    _slopes(slopes, H)
    if out is not None:
        _need_shape(out, "out", torch.bfloat16, q.shape)
    if lse is not None:
        _need_shape(lse, "lse", torch.float32, (B, H, N))
    if out_low is not None:
        _need_shape(out_low, "out_low", torch.bfloat16, q.shape)
    _same_device(q, k, v, plan.data, slopes, out, lse, out_low)
    o = torch.empty_like(q) if out is None else out
    l = q.new_empty((B, H, N), dtype=torch.float32) if lse is None else lse
    ol = out_low if out_low is not None else (torch.empty_like(q) if low else None)
    with _on(q):
        st = lib().fa_mod_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              None if ol is None else ol.data_ptr(), l.data_ptr(), plan.data.data_ptr(),
                              None if slopes is None else slopes.data_ptr(), B, N, H, Hkv, d, _scale(scale, d), softcap,
                              _stream_ptr(q))
    _check(st, "fa_mod_fwd")
    return (o, l) if ol is None else (o, l, ol)


def mod_bwd_workspace_size(B: int, N: int, H: int, Hkv: int, d: int) -> int:
    return int(lib().fa_mod_bwd_workspace_size(B, N, H, Hkv, d))


def mod_bwd(q, k, v, o, lse, do, plan: MaskPlan, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
            scale: Optional[float] = None, o_low: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, dq=None, dk=None, dv=None, deterministic: bool = False):
    """dQ [B, N, H, d], dK and dV [B, N, Hkv, d] (summed over each group of heads);
    o, lse (and o_low) from mod_fwd with the same plan, softcap, slopes and scale.

    deterministic=True: dQ too is bitwise reproducible (dK and dV always are)."""
    B, N, H, Hkv, d = _sizes(q, k, v, plan)
    softcap = _softcap(softcap)
    _slopes(slopes, H)
    _need_shape(o, "o", torch.bfloat16, q.shape)
    _need_shape(do, "do", torch.bfloat16, q.shape)
    if o_low is not None:
        _need_shape(o_low, "o_low", torch.bfloat16, q.shape)
    _need_shape(lse, "lse", torch.float32, (B, H, N))
    if dq is not None:
        _need_shape(dq, "dq", torch.bfloat16, q.shape)
    if dk is not None:
        _need_shape(dk, "dk", torch.bfloat16, k.shape)
    if dv is not None:
        _need_shape(dv, "dv", torch.bfloat16, k.shape)
    L = lib()
    need = L.fa_mod_bwd_workspace_size(B, N, H, Hkv, d)
    if workspace is not None:
        _need_workspace(workspace, need)
    _same_device(q, k, v, o, lse, do, plan.data, o_low, slopes, workspace, dq, dk, dv)
    ws = q.new_empty(max(need, 256), dtype=torch.uint8) if workspace is None else workspace
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(k) if dv is None else dv
    with _on(q):
        fn = L.fa_mod_bwd_deterministic if deterministic else L.fa_mod_bwd
        st = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), None if o_low is None else o_low.data_ptr(),
                lse.data_ptr(), do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), plan.data.data_ptr(),
                None if slopes is None else slopes.data_ptr(), ws.data_ptr(), ws.nbytes, B, N, H, Hkv, d,
                _scale(scale, d), softcap, _stream_ptr(q))
    _check(st, "fa_mod_bwd_deterministic" if deterministic else "fa_mod_bwd")
    return dq, dk, dv


class _ModAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, plan, softcap, slopes, scale, deterministic):
        o, lse, o_low = mod_fwd(q, k, v, plan, softcap=softcap, slopes=slopes, scale=scale, low=True)
        ctx.save_for_backward(q, k, v, o, lse, o_low, plan.data, *(() if slopes is None else (slopes,)))
        ctx.sizes, ctx.softcap, ctx.scale, ctx.deterministic = (plan.B, plan.N), softcap, scale, deterministic
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, o_low, data, *slopes = ctx.saved_tensors
        g = mod_bwd(q, k, v, o, lse, do.contiguous(), MaskPlan(data, *ctx.sizes), softcap=ctx.softcap,
                    slopes=slopes[0] if slopes else None, scale=ctx.scale, o_low=o_low,
                    deterministic=ctx.deterministic)
        return (*g, None, None, None, None, None)


def _differentiated(*ts) -> bool:
    """Some derivative is asked for: a gradient, or a tangent of forward mode (which
    the Function lacks and refuses)."""
    ts = [t for t in ts if isinstance(t, torch.Tensor)]
    return (torch.is_grad_enabled() and any(t.requires_grad for t in ts)) or \
        any(forward_ad.unpack_dual(t).tangent is not None for t in ts)


def mod_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, plan: MaskPlan, softcap: float = 0.0,
                  slopes: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                  deterministic: bool = False) -> torch.Tensor:
    """Attention with modified scores over bf16 [B, N, H, d] queries and
    [B, N, Hkv, d] keys and values; differentiable in q, k, v.
    deterministic=True makes the gradients bitwise reproducible."""
    if isinstance(q, torch.Tensor) and q.dim() == 4:
        _slopes(slopes, q.shape[2])  # inside a Function no tensor asks for a gradient
    if not _differentiated(q, k, v, slopes):
        return mod_fwd(q, k, v, plan, softcap=softcap, slopes=slopes, scale=scale)[0]
    return _ModAttention.apply(q, k, v, plan, softcap, slopes, scale, bool(deterministic))
