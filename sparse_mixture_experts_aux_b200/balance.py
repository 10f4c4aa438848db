"""Torch-facing wrapper of moe_balance_loss and its gradient (include/moe.h):
argument checks and marshalling; the library computes."""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib, streams
from .layer import Workspace, dtype_code


def _need(name: str, t: torch.Tensor, dtype, shape, dev) -> None:
    if t.device != dev:
        raise RuntimeError(f"{name} must be on {dev}, got {t.device}")
    if t.dtype != dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise RuntimeError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise RuntimeError(f"{name} must be contiguous")


def _no_tangent(where: str, *tensors) -> None:
    if forward_ad._current_level < 0:  # no dual tensors outside a dual level
        return
    for t in tensors:
        if forward_ad.unpack_dual(t).tangent is not None:
            raise RuntimeError(f"{where} has no forward-mode derivative: a tangent would be lost")


def _args(logits, k, gate_mode, token_mask, cu_seqlens):
    """Checks what both directions take; returns (T, E, S, fields of moe_balance_dims)."""
    if logits.dim() != 2:
        raise RuntimeError(f"logits must be [T, E], got {tuple(logits.shape)}")
    if not logits.is_cuda:
        raise RuntimeError("logits must be a CUDA tensor (there is no CPU path)")
    T, E = logits.shape
    ld = E
    if not logits.is_contiguous():
        if E > 1 and logits.stride(1) != 1:
            raise RuntimeError("logits must have their experts next to each other (stride 1)")
        if T > 1:
            ld = logits.stride(0)
            if ld < E:
                raise RuntimeError("logits' rows must not overlap")
    dev = logits.device
    S, cu, mask = 1, None, None
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise RuntimeError("cu_seqlens must be [S + 1] with S >= 1")
        S = cu_seqlens.numel() - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, (S + 1,), dev)
        cu = cu_seqlens.data_ptr()
    if token_mask is not None:
        _need("token_mask", token_mask, (torch.bool, torch.uint8), (T,), dev)
        mask = token_mask.data_ptr() or None
    return T, E, S, (T, E, k, dtype_code(logits.dtype), int(gate_mode), ld, S, cu, mask)


def _forward(logits, topk_idx, gate_mode, token_mask, cu_seqlens, workspace, stream):
    if topk_idx.dim() != 2:
        raise RuntimeError(f"topk_idx must be [T, k], got {tuple(topk_idx.shape)}")
    k = topk_idx.shape[1]
    T, E, S, fields = _args(logits, k, gate_mode, token_mask, cu_seqlens)
    dev = logits.device
    _need("topk_idx", topk_idx, torch.int32, (T, k), dev)
    handle, side = streams.run_on(stream, dev)
    with streams.on(dev, side):
        d = _lib.moe_balance_dims(*fields, None, 0, handle)
        need = _lib.moe_balance_loss_workspace_size(d) if T > _lib.MOE_BALANCE_SMALL_T else 0
        if need:  # a call that is refused has no size: it says why below
            ws = (workspace or Workspace()).get(need, dev)
            d.workspace, d.workspace_bytes = ws.data_ptr(), ws.numel()
            streams.lend(side, ws)
        loss = torch.empty(S, dtype=torch.float32, device=dev)
        counts = torch.empty((S, E), dtype=torch.int32, device=dev)
        tokens = torch.empty(S, dtype=torch.int32, device=dev)
        rc = _lib.moe_balance_loss(d, logits, topk_idx, loss, counts, tokens)
    if rc != _lib.MOE_OK:
        raise _lib.MoeError(rc, "moe_balance_loss")
    streams.lend(side, logits, topk_idx, token_mask, cu_seqlens)
    streams.give(side, dev, loss, counts, tokens)
    return loss, counts, tokens


def balance_loss_backward(dloss: torch.Tensor, logits: torch.Tensor, counts: torch.Tensor,
                          tokens: torch.Tensor, k: int, gate_mode: int = 0,
                          token_mask: Optional[torch.Tensor] = None,
                          cu_seqlens: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of balance_loss with respect to the logits ([T, E], the logits' dtype).

    dloss fp32 [S]: the gradient of each sequence's loss; counts and tokens as
    balance_loss returned them; k = topk_idx.shape[1]; the rest as there. This is
    the call behind balance_loss's autograd, for programs that chain gradients
    themselves (it touches no autograd state, so it can be captured in a graph).
    """
    _no_tangent("balance_loss_backward", dloss, logits)
    T, E, S, fields = _args(logits, int(k), gate_mode, token_mask, cu_seqlens)
    dev = logits.device
    _need("dloss", dloss, torch.float32, (S,), dev)
    _need("counts", counts, torch.int32, (S, E), dev)
    _need("tokens", tokens, torch.int32, (S,), dev)
    handle, side = streams.run_on(stream, dev)
    with streams.on(dev, side):
        d = _lib.moe_balance_dims(*fields, None, 0, handle)
        dlogits = torch.empty((T, E), dtype=logits.dtype, device=dev)
        rc = _lib.moe_balance_loss_backward(d, dloss, logits, counts, tokens, dlogits)
    if rc != _lib.MOE_OK:
        raise _lib.MoeError(rc, "moe_balance_loss_backward")
    streams.lend(side, dloss, logits, counts, tokens, token_mask, cu_seqlens)
    streams.give(side, dev, dlogits)
    return dlogits


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk_idx, gate_mode, token_mask, cu_seqlens, workspace):
        loss, counts, tokens = _forward(logits, topk_idx, gate_mode, token_mask, cu_seqlens,
                                        workspace, None)
        ctx.mark_non_differentiable(counts, tokens)
        ctx.save_for_backward(logits, counts, tokens, token_mask, cu_seqlens)
        ctx.args = (topk_idx.shape[1], gate_mode)
        return loss, counts, tokens

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _counts, _tokens):
        logits, counts, tokens, token_mask, cu_seqlens = ctx.saved_tensors
        k, gate_mode = ctx.args
        d = balance_loss_backward(dloss.contiguous(), logits, counts, tokens, k, gate_mode,
                                  token_mask, cu_seqlens)
        return d, None, None, None, None, None


def balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, gate_mode: int = 0,
                 token_mask: Optional[torch.Tensor] = None,
                 cu_seqlens: Optional[torch.Tensor] = None,
                 workspace: Optional[Workspace] = None, stream=None):
    """Load-balance loss E sum_i f_i P_i of each sequence, with autograd.

    Returns (loss fp32 [S], counts int32 [S, E], tokens int32 [S]); S = 1 without
    cu_seqlens. counts are the routed assignments per expert, tokens the tokens
    that count; neither carries a gradient. Reverse mode only, once: a tangent of
    forward mode is refused. The loss is raw: scale it by the
    trainer's weight, and average it over sequences if there are several.

    logits [T, E] fp32 or bf16, rows may be strided: what the softmax of the layer
    sees. After `forward`, routing_views(...)["logits"] and ["topk_idx"] are
    these arguments (add router_bias to the logits if the layer has one). The views
    carry no graph: a trainer whose gradient is to reach W_r and x computes the
    logits by itself (x.float() @ W_r.t()), or chains balance_loss_backward's result.
    topk_idx int32 [T, k]: the chosen experts; entries outside [0, E), like -1 for
    a dropped slot, count for none.
    gate_mode: as in forward (2: the probabilities are normalised sigmoids).
    token_mask bool or uint8 [T]: False for padding tokens.
    cu_seqlens int32 [S + 1]: sequence s is tokens cu[s] .. cu[s + 1] - 1.
    stream: where to run instead of the current stream (not with a gradient: use
    torch.cuda.stream). The inputs must be ready there, and the results are: wait
    for it before they are used elsewhere. Both may be dropped at any time; a raw
    cudaStream_t has to outlive them.
    """
    _no_tangent("balance_loss", logits)
    if torch.is_grad_enabled() and logits.requires_grad:
        if stream is not None:
            raise RuntimeError("balance_loss with a gradient runs on the current stream: "
                               "use torch.cuda.stream(...) instead of stream=")
        return _BalanceLoss.apply(logits, topk_idx, gate_mode, token_mask, cu_seqlens, workspace)
    return _forward(logits, topk_idx, gate_mode, token_mask, cu_seqlens, workspace, stream)
