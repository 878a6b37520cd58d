"""Norm and gated feed-forward operators of libfp8q: marshalling, as the rest of the binding.

Entry points with the C names (caller-provided outputs, nothing allocated):
    fp8q_rms_norm_quant, fp8q_rms_norm_bwd

Allocating helpers:
    rms_norm               residual addition and root-mean-square norm (differentiable)
    rms_norm_cast_to_fp8   the same with the result cast to 1 x G fp8 groups
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import (E4M3FN, SCALE_IEEE, _FMT_DTYPE, _check, _dev_ptr, _dtype_code, _fmt_of, _need, _rule_of, _stream, lib)

__all__ = [
    "fp8q_rms_norm_quant", "fp8q_rms_norm_bwd", "fp8q_rms_norm_bwd_workspace_bytes",
    "rms_norm", "rms_norm_cast_to_fp8",
]


# ---------------------------------------------------------------------------
# root-mean-square norm
# ---------------------------------------------------------------------------
def _rows(x: torch.Tensor, weight: torch.Tensor):
    """(rows, width) of x[..., n] normed over its last dimension by weight[n]."""
    if x.dim() < 1 or weight.dim() != 1 or x.shape[-1] != weight.shape[0]:
        raise ValueError(f"x must be [..., n] and weight [n], got {tuple(x.shape)} and {tuple(weight.shape)}")
    n = weight.shape[0]
    return (x.numel() // n if n else 0), n


def _like(t: Optional[torch.Tensor], x: torch.Tensor, name: str) -> None:
    if t is not None and (t.shape != x.shape or t.dtype != x.dtype):
        raise ValueError(f"{name} must have x's shape and dtype, got {tuple(t.shape)} {t.dtype}")


def fp8q_rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, y: Optional[torch.Tensor] = None,
                        q: Optional[torch.Tensor] = None, scale_inv: Optional[torch.Tensor] = None,
                        residual: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
                        rstd: Optional[torch.Tensor] = None, eps: float = 1e-6, group: int = 128, fmt=E4M3FN,
                        rule=SCALE_IEEE, stream=None) -> None:
    """r = x + residual into residual_out (which may be residual or x itself), its norm over the last
    dimension times weight into y (x's dtype), into fp8 codes q with scale_inv per 1 x group, or both;
    rstd [rows] fp32 is what fp8q_rms_norm_bwd takes."""
    m, n = _rows(x, weight)
    dev = x.device
    _like(residual, x, "residual")
    _like(residual_out, x, "residual_out")
    if (residual is None) != (residual_out is None):
        raise ValueError("residual and residual_out go together")
    if y is None and q is None:
        raise ValueError("y or q must be given")
    if y is not None:
        _need(y, m * n, "y", dtype=x.dtype)
    if q is not None:
        _need(q, m * n, "q", byte=True)
        if scale_inv is None:
            raise ValueError("q needs scale_inv")
        if group > 0 and n % group == 0:
            _need(scale_inv, m * (n // group), "scale_inv", dtype=torch.float32)
    if rstd is not None:
        _need(rstd, m, "rstd", dtype=torch.float32)
    _check(lib().fp8q_rms_norm_quant(
        _dev_ptr(x, "x"), _dtype_code(x, "x"), _dev_ptr(residual, "residual", dev),
        _dev_ptr(residual_out, "residual_out", dev), _dev_ptr(weight, "weight", dev), _dtype_code(weight, "weight"),
        m, n, eps, group, _fmt_of(fmt), _rule_of(rule), _dev_ptr(y, "y", dev), _dev_ptr(q, "q", dev),
        _dev_ptr(scale_inv, "scale_inv", dev), _dev_ptr(rstd, "rstd", dev), _stream(stream, dev)),
        "fp8q_rms_norm_quant")


def fp8q_rms_norm_bwd_workspace_bytes(m: int, n: int) -> int:
    """Workspace of fp8q_rms_norm_bwd on the current device."""
    L = lib()
    return int(L.fp8q_rms_norm_bwd_workspace_bytes(int(m), int(n)))


def fp8q_rms_norm_bwd(dy: torch.Tensor, r: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, dx: torch.Tensor,
                      dweight: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      dres: Optional[torch.Tensor] = None, stream=None) -> None:
    """The gradient of fp8q_rms_norm_quant's y (dy) and r (dres, optional): dx for x and the residual,
    dweight (optional) for the weight.  r and rstd are the forward's; workspace holds
    fp8q_rms_norm_bwd_workspace_bytes(rows, n) bytes when dweight is given."""
    m, n = _rows(dy, weight)
    dev = dy.device
    _like(r, dy, "r")
    _like(dres, dy, "dres")
    _need(dx, m * n, "dx", dtype=dy.dtype)
    _need(rstd, m, "rstd", dtype=torch.float32)
    if dweight is not None:
        _need(dweight, n, "dweight", dtype=weight.dtype)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().fp8q_rms_norm_bwd(
        _dev_ptr(dy, "dy"), _dev_ptr(r, "r", dev), _dtype_code(dy, "dy"), _dev_ptr(weight, "weight", dev),
        _dtype_code(weight, "weight"), _dev_ptr(rstd, "rstd", dev), _dev_ptr(dres, "dres", dev), m, n,
        _dev_ptr(dx, "dx", dev), _dev_ptr(dweight, "dweight", dev), _dev_ptr(workspace, "workspace", dev), wbytes,
        _stream(stream, dev)), "fp8q_rms_norm_bwd")


class _RmsNorm(torch.autograd.Function):
    """rms_norm and its gradient; saves the summed rows, the weight and one rstd per row."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        x, weight = x.contiguous(), weight.contiguous()
        m, _ = _rows(x, weight)
        y = torch.empty_like(x)
        rstd = torch.empty((m,), dtype=torch.float32, device=x.device)
        r = None
        if residual is not None:
            residual = residual.contiguous()
            r = torch.empty_like(x)
        fp8q_rms_norm_quant(x, weight, y=y, residual=residual, residual_out=r, rstd=rstd, eps=eps)
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x if r is None else r, weight, rstd)
        return (y, r) if ctx.has_residual else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dr=None):
        r, weight, rstd = ctx.saved_tensors
        if dy is None:                       # only the sum was used
            return dr, None, dr if ctx.has_residual else None, None
        dy = dy.contiguous()
        dr = dr.contiguous() if dr is not None else None
        dx = torch.empty_like(r)
        dw = ws = None
        if ctx.needs_input_grad[1]:
            dw = torch.empty_like(weight)
            # a workspace of this call's own: the caching allocator orders it by stream and by graph
            ws = torch.empty(fp8q_rms_norm_bwd_workspace_bytes(*_rows(r, weight)), dtype=torch.uint8, device=r.device)
        fp8q_rms_norm_bwd(dy, r, weight, rstd, dx, dw, ws, dr)
        return dx, dw, dx if ctx.has_residual else None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """Root-mean-square norm over the last dimension, times weight (x's dtype or fp32): returns y, or
    (y, x + residual) when a residual is given.  Differentiable in x, weight and residual."""
    return _RmsNorm.apply(x, weight, residual, eps)


def rms_norm_cast_to_fp8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                         eps: float = 1e-6, group: int = 128, fmt=E4M3FN, rule=SCALE_IEEE):
    """per_token_cast_to_fp8(rms_norm(x + residual)) in one pass, the norm cast before any rounding to
    x's dtype: (q, scale_inv), or (q, scale_inv, x + residual) when a residual is given."""
    x, weight = x.contiguous(), weight.contiguous()
    f = _fmt_of(fmt)
    n = x.shape[-1]
    q = torch.empty(x.shape, dtype=_FMT_DTYPE[f], device=x.device)
    s = torch.empty((*x.shape[:-1], n // group if group > 0 else 0), dtype=torch.float32, device=x.device)
    r = None
    if residual is not None:
        residual = residual.contiguous()
        r = torch.empty_like(x)
    fp8q_rms_norm_quant(x, weight, q=q, scale_inv=s, residual=residual, residual_out=r, eps=eps, group=group, fmt=f,
                        rule=rule)
    return (q, s) if r is None else (q, s, r)
