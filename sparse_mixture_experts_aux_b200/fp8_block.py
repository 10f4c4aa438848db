"""Torch-facing wrappers of the block-scaled FP8 operators (include/moe.h,
moe_*_fp8_block): argument checks and marshalling; the library computes.

stream= in each of them: where to run instead of the current stream. The inputs
must be ready there, and the results are: wait for it before they are used
elsewhere. Both may be dropped at any time; a raw cudaStream_t has to outlive them."""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import _lib, streams
from .balance import _need
from .layer import dtype_code

_CODES = (torch.uint8, torch.float8_e4m3fn)


def _ceil(n: int, b: int) -> int:
    return -(-n // b)


def _stack(t: torch.Tensor) -> int:
    return math.prod(t.shape[:-2])


def quantize_fp8_block(w: torch.Tensor, block_rows: int = 128, stream=None):
    """E4M3 codes (uint8, w's shape) and fp32 scales, one for each block of
    block_rows x 128 (include/moe.h, moe_quantize_fp8_block).

    block_rows = 1 (activations): w [..., cols], scales [..., ceil(cols / 128)];
    the rows of a 2-D w may be strided. block_rows = 128 (weights): w [..., rows,
    cols], scales [..., ceil(rows / 128), ceil(cols / 128)]. bf16 or fp32, cols a
    multiple of 16. No gradient: the results of a w that requires one do not.
    """
    if not w.is_cuda:
        raise RuntimeError("w must be a CUDA tensor (there is no CPU path)")
    if w.dim() < 2:
        raise RuntimeError(f"w must have rows and columns, got shape {tuple(w.shape)}")
    rows, cols = w.shape[-2:]
    ld = w.stride(-2) if w.dim() == 2 and rows > 1 else cols
    if not w.is_contiguous() and (w.dim() > 2 or (cols > 1 and w.stride(-1) != 1) or ld < cols):
        raise RuntimeError("w must be contiguous (the rows of a matrix may be strided)")
    dev = w.device
    handle, side = streams.run_on(stream, dev)
    with streams.on(dev, side):
        codes = torch.empty(w.shape, dtype=torch.uint8, device=dev)
        srows = rows if block_rows == 1 else _ceil(rows, max(1, block_rows))
        scales = torch.empty((*w.shape[:-2], srows, _ceil(cols, 128)), dtype=torch.float32,
                             device=dev)
        rc = _lib.moe_quantize_fp8_block(w, dtype_code(w.dtype), _stack(w), rows, cols, ld,
                                         block_rows, codes, scales, handle)
    if rc != _lib.MOE_OK:
        raise _lib.MoeError(rc, "moe_quantize_fp8_block")
    streams.lend(side, w)
    streams.give(side, dev, codes, scales)
    return codes, scales


def dequantize_fp8_block(codes: torch.Tensor, scales: torch.Tensor, block_rows: int = 128,
                         stream=None) -> torch.Tensor:
    """fp32 values code * scale of quantize_fp8_block's results
    (moe_dequantize_fp8_block). No gradient."""
    if not codes.is_cuda or not codes.is_contiguous() or codes.dim() < 2 or codes.dtype not in _CODES:
        raise RuntimeError("codes must be a contiguous CUDA tensor of E4M3 codes with rows and columns")
    rows, cols = codes.shape[-2:]
    dev = codes.device
    srows = rows if block_rows == 1 else _ceil(rows, max(1, block_rows))
    _need("scales", scales, torch.float32, codes.shape[:-2] + (srows, _ceil(cols, 128)), dev)
    handle, side = streams.run_on(stream, dev)
    with streams.on(dev, side):
        out = torch.empty(codes.shape, dtype=torch.float32, device=dev)
        rc = _lib.moe_dequantize_fp8_block(codes, scales, _stack(codes), rows, cols, block_rows, out,
                                           handle)
    if rc != _lib.MOE_OK:
        raise _lib.MoeError(rc, "moe_dequantize_fp8_block")
    streams.lend(side, codes, scales)
    streams.give(side, dev, out)
    return out


def _product_dims(a, a_scales, weights, scales, offsets, wait_timeout_ns):
    """Checks what the two products share; returns (dims, M, N)."""
    if not a.is_cuda:
        raise RuntimeError("a must be a CUDA tensor (there is no CPU path)")
    if a.dim() != 2 or a.dtype not in _CODES:
        raise RuntimeError("a must be [M, K] E4M3 codes (uint8)")
    M, K = a.shape
    if (K > 1 and a.stride(1) != 1) or (M > 1 and a.stride(0) < K):
        raise RuntimeError("a must have its columns next to each other (rows may be strided)")
    dev = a.device
    w = weights[0]
    E = 0
    if offsets is not None:
        if offsets.dim() != 1 or offsets.numel() < 2:
            raise RuntimeError("offsets must be [E + 1] with E >= 1")
        E = offsets.numel() - 1
        _need("offsets", offsets, torch.int32, (E + 1,), dev)
    if w.dim() != (3 if E else 2):
        raise RuntimeError("weights must be [N, K], or [E, N, K] with offsets")
    N = w.shape[-2]
    lead = (E,) if E else ()
    for t, s in zip(weights, scales):
        _need("weights", t, _CODES, lead + (N, K), dev)
        _need("weight scales", s, torch.float32, lead + (_ceil(N, 128), _ceil(K, 128)), dev)
    _need("a_scales", a_scales, torch.float32, (M, _ceil(K, 128)), dev)
    fields = (M, N, K, E, 0, a.stride(0) if M > 1 else K, 0,
              offsets.data_ptr() if E else None, None, int(wait_timeout_ns))
    return _lib.moe_fp8_block_dims(*fields), M, N


def matmul_fp8_block(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor,
                     w_scales: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                     row_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     out_dtype: torch.dtype = torch.bfloat16, stream=None,
                     wait_timeout_ns: int = 0) -> torch.Tensor:
    """a @ w^T of block-scaled FP8 matrices, dense or grouped by expert, in fp32,
    rounded once to out's type (include/moe.h, moe_matmul_fp8_block).

    a [M, K], a_scales [M, ceil(K / 128)]: quantize_fp8_block(x, block_rows=1); rows
    may be strided. w [N, K], w_scales [ceil(N / 128), ceil(K / 128)]:
    quantize_fp8_block(W). With offsets int32 [E + 1] on the device, w is [E, N, K]
    and rows offsets[e] .. offsets[e + 1] - 1 of a meet expert e; rows of out that
    belong to no expert are left as they were (give out, or do not read them).
    row_scale fp32 [M]: a factor for each output row (the gates). out [M, N] bf16 or
    fp32 (rows may be strided), allocated in out_dtype if not given. No gradient.
    """
    d, M, N = _product_dims(a, a_scales, (w,), (w_scales,), offsets, wait_timeout_ns)
    dev = a.device
    if row_scale is not None:
        _need("row_scale", row_scale, torch.float32, (M,), dev)
        d.row_scale = row_scale.data_ptr()
    handle, side = streams.run_on(stream, dev)
    with streams.on(dev, side):
        if out is None:
            out = torch.empty(M, N, dtype=out_dtype, device=dev)
        elif out.device != dev or tuple(out.shape) != (M, N):
            raise RuntimeError(f"out must be [{M}, {N}] on {dev}")
        elif (N > 1 and out.stride(1) != 1) or (M > 1 and out.stride(0) < N):
            raise RuntimeError("out must have its columns next to each other (rows may be strided)")
        d.out_dtype = dtype_code(out.dtype)
        d.ld_out = out.stride(0) if M > 1 else N
        d.stream = handle or None
        rc = _lib.moe_matmul_fp8_block(d, a, a_scales, w, w_scales, out)
    if rc != _lib.MOE_OK:
        raise _lib.MoeError(rc, "moe_matmul_fp8_block")
    if side is not None:  # out may be the caller's or the call's own
        streams.lend(side, a, a_scales, w, w_scales, offsets, row_scale, out)
        streams.give(side, dev, out)
    return out


def swiglu_fp8_block(a: torch.Tensor, a_scales: torch.Tensor, W_g: torch.Tensor, W_u: torch.Tensor,
                     g_scales: torch.Tensor, u_scales: torch.Tensor,
                     offsets: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
                     scales: Optional[torch.Tensor] = None, stream=None, wait_timeout_ns: int = 0):
    """The first half of SwiGLU experts on block-scaled FP8: SiLU(a W_g^T) * (a W_u^T),
    quantised with one scale for each 128 columns (include/moe.h, moe_swiglu_fp8_block).

    a, a_scales, W_g, W_u, their scales and offsets as in matmul_fp8_block (N a
    multiple of 16). Returns (codes uint8 [M, N], scales fp32 [M, ceil(N / 128)]), the
    next matmul_fp8_block's a and a_scales; rows that belong to no expert are left as
    they were in codes and scales. No gradient.
    """
    d, M, N = _product_dims(a, a_scales, (W_g, W_u), (g_scales, u_scales), offsets, wait_timeout_ns)
    dev = a.device
    handle, side = streams.run_on(stream, dev)
    with streams.on(dev, side):
        if codes is None:
            codes = torch.empty(M, N, dtype=torch.uint8, device=dev)
        else:
            _need("codes", codes, _CODES, (M, N), dev)
        if scales is None:
            scales = torch.empty(M, _ceil(N, 128), dtype=torch.float32, device=dev)
        else:
            _need("scales", scales, torch.float32, (M, _ceil(N, 128)), dev)
        d.stream = handle or None
        rc = _lib.moe_swiglu_fp8_block(d, a, a_scales, W_g, W_u, g_scales, u_scales, codes, scales)
    if rc != _lib.MOE_OK:
        raise _lib.MoeError(rc, "moe_swiglu_fp8_block")
    if side is not None:  # codes and scales may be the caller's or the call's own
        streams.lend(side, a, a_scales, W_g, W_u, g_scales, u_scales, offsets, codes, scales)
        streams.give(side, dev, codes, scales)
    return codes, scales
