"""Norm and gated feed-forward operators of libfp8q: marshalling, as the rest of the binding.

Entry points with the C names (caller-provided outputs, nothing allocated):
    fp8q_rms_norm_quant, fp8q_rms_norm_bwd
    fp8q_gated_mm, fp8q_gated_mm_blockwise, fp8q_gated_mm_blockwise_quant, fp8q_gated_bwd_cast

Allocating helpers:
    rms_norm                     residual addition and root-mean-square norm (differentiable)
    rms_norm_cast_to_fp8         the same with the result cast to 1 x G fp8 groups
    gated_linear_fp8             act(x Wg^T) * (x Wu^T) with linear_fp8's casts (differentiable)
    gated_linear_fp8_blockwise   the same on block-scaled weights
    ffn_fp8, ffn_fp8_blockwise   the whole block: the gated products, then the down projection
"""
from __future__ import annotations

import functools
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import (E4M3FN, E5M2, K_MAJOR, MN_MAJOR, SCALE_IEEE, _FMT_DTYPE, _FP8_DTYPES, _check, _dev_ptr, _dtype_code,
               _fmt_of, _need, _rule_of, _status_word, _stream, fp8q_cast_per_tensor_workspace_bytes,
               fp8q_scaled_mm_blockwise, lib, linear_fp8, per_token_cast_to_fp8)

__all__ = [
    "fp8q_rms_norm_quant", "fp8q_rms_norm_bwd", "fp8q_rms_norm_bwd_workspace_bytes",
    "rms_norm", "rms_norm_cast_to_fp8",
    "ACT_SILU", "ACT_GELU_TANH", "fp8q_gated_mm", "fp8q_gated_mm_blockwise", "fp8q_gated_mm_blockwise_quant",
    "fp8q_gated_bwd_cast", "gated_linear_fp8", "gated_linear_fp8_blockwise", "ffn_fp8", "ffn_fp8_blockwise",
]

ACT_SILU, ACT_GELU_TANH = 0, 1
_CAST_WORKSPACE = functools.cache(fp8q_cast_per_tensor_workspace_bytes)      # a constant of the library


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


# The autograd functions call the library directly: what they allocate themselves needs no checks, and
# a small training step is bound by the host's time between launches.
def _on_device(x: torch.Tensor, *others) -> int:
    """The stream of a call on x's device; every tensor given must be on it."""
    if not x.is_cuda:
        raise ValueError("the input must be a CUDA tensor (libfp8q takes device pointers)")
    for t in others:
        if t is not None and t.device != x.device:
            raise ValueError(f"a tensor is on {t.device}, expected {x.device}")
    return _stream(None, x.device)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


class _RmsNorm(torch.autograd.Function):
    """rms_norm and its gradient; saves the summed rows, the weight and one rstd per row."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        st = _on_device(x, weight, residual)
        _like(residual, x, "residual")
        x, weight = x.contiguous(), weight.contiguous()
        m, n = _rows(x, weight)
        y = torch.empty_like(x)
        rstd = torch.empty((m,), dtype=torch.float32, device=x.device)
        r = None
        if residual is not None:
            residual = residual.contiguous()
            r = torch.empty_like(x)
        _check(lib().fp8q_rms_norm_quant(
            x.data_ptr(), _dtype_code(x, "x"), _ptr(residual), _ptr(r), weight.data_ptr(),
            _dtype_code(weight, "weight"), m, n, eps, 1, E4M3FN, SCALE_IEEE, y.data_ptr(), None, None, rstd.data_ptr(),
            st), "fp8q_rms_norm_quant")
        ctx.has_residual = r is not None
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x if r is None else r, weight, rstd)
        return y if r is None else (y, r)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dr=None):
        r, weight, rstd = ctx.saved_tensors
        if dy is None:                       # only the sum was used
            return dr, None, dr if ctx.has_residual else None, None
        st = _on_device(r, dy, dr)
        dy = dy.contiguous()
        dr = dr.contiguous() if dr is not None else None
        m, n = _rows(r, weight)
        dx = torch.empty_like(r)
        dw = ws = None
        nbytes = 0
        if ctx.needs_input_grad[1]:
            dw = torch.empty_like(weight)
            # a workspace of this call's own: the caching allocator orders it by stream and by graph
            nbytes = fp8q_rms_norm_bwd_workspace_bytes(m, n)
            ws = torch.empty((nbytes,), dtype=torch.uint8, device=r.device)
        _check(lib().fp8q_rms_norm_bwd(
            dy.data_ptr(), r.data_ptr(), _dtype_code(r, "x"), weight.data_ptr(), _dtype_code(weight, "weight"),
            rstd.data_ptr(), _ptr(dr), m, n, dx.data_ptr(), _ptr(dw), _ptr(ws), nbytes, st), "fp8q_rms_norm_bwd")
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


# ---------------------------------------------------------------------------
# gated feed-forward block
# ---------------------------------------------------------------------------
def _act_of(act) -> int:
    if isinstance(act, str):
        return {"silu": ACT_SILU, "gelu_tanh": ACT_GELU_TANH}[act]
    return int(act)


def _gated_operands(a, w_gate, w_up, fa, fb):
    if a.dim() != 2 or w_gate.dim() != 2 or w_up.shape != w_gate.shape or a.shape[1] != w_gate.shape[1]:
        raise ValueError(f"a must be [M, K], w_gate and w_up [I, K], got {tuple(a.shape)}, {tuple(w_gate.shape)} and "
                         f"{tuple(w_up.shape)}")
    M, K = a.shape
    I = w_gate.shape[0]
    if w_gate.dtype != w_up.dtype:
        raise TypeError("w_gate and w_up must have one dtype")
    _need(a, M * K, "a", byte=True)
    _need(w_gate, I * K, "w_gate", byte=True)
    fa = _fmt_of(fa) if fa is not None else _FP8_DTYPES.get(a.dtype, E4M3FN)
    fb = _fmt_of(fb) if fb is not None else _FP8_DTYPES.get(w_gate.dtype, E4M3FN)
    return M, I, K, fa, fb


def fp8q_gated_mm(a: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, scale_a: torch.Tensor,
                  scale_gate: torch.Tensor, scale_up: torch.Tensor, out: torch.Tensor,
                  gate_up: Optional[torch.Tensor] = None, act=ACT_SILU, fa=None, fb=None,
                  status: Optional[torch.Tensor] = None, stream=None) -> None:
    """out[M, I] = act(gate) * up with gate = a @ w_gate.t() and up = a @ w_up.t() of fp8 codes a [M, K],
    w_gate and w_up [I, K] and per-tensor scales (fp32 [1] each).  gate_up: optional [M, 2 I] of out's
    dtype that receives gate and up for fp8q_gated_bwd_cast.  act: "silu" or "gelu_tanh"."""
    M, I, K, fa, fb = _gated_operands(a, w_gate, w_up, fa, fb)
    dev = a.device
    for t, name in ((scale_a, "scale_a"), (scale_gate, "scale_gate"), (scale_up, "scale_up")):
        _need(t, 1, name, dtype=torch.float32)
    _need(out, M * I, "out")
    if gate_up is not None:
        _need(gate_up, 2 * M * I, "gate_up", dtype=out.dtype)
    _check(lib().fp8q_gated_mm(
        _dev_ptr(a, "a"), fa, _dev_ptr(w_gate, "w_gate", dev), _dev_ptr(w_up, "w_up", dev), fb, M, I, K,
        _dev_ptr(scale_a, "scale_a", dev), _dev_ptr(scale_gate, "scale_gate", dev), _dev_ptr(scale_up, "scale_up", dev),
        _act_of(act), _dtype_code(out, "out"), _dev_ptr(out, "out", dev), _dev_ptr(gate_up, "gate_up", dev),
        _dev_ptr(_status_word(status), "status", dev), _stream(stream, dev)), "fp8q_gated_mm")


def _fine_scales(M, I, K, scale_a, scale_gate, scale_up):
    kb, ib = -(-K // 128), -(-I // 128)
    _need(scale_a, M * kb, "scale_a", dtype=torch.float32)
    _need(scale_gate, ib * kb, "scale_gate", dtype=torch.float32)
    _need(scale_up, ib * kb, "scale_up", dtype=torch.float32)
    return ib


def fp8q_gated_mm_blockwise(a: torch.Tensor, scale_a: torch.Tensor, w_gate: torch.Tensor, scale_gate: torch.Tensor,
                            w_up: torch.Tensor, scale_up: torch.Tensor, out: torch.Tensor, act=ACT_SILU, fa=None,
                            fb=None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """fp8q_gated_mm with fine-grained scales: scale_a [M, ceil(K/128)] per 1 x 128 group, scale_gate and
    scale_up [ceil(I/128), ceil(K/128)] per 128 x 128 block."""
    M, I, K, fa, fb = _gated_operands(a, w_gate, w_up, fa, fb)
    dev = a.device
    _fine_scales(M, I, K, scale_a, scale_gate, scale_up)
    _need(out, M * I, "out")
    _check(lib().fp8q_gated_mm_blockwise(
        _dev_ptr(a, "a"), fa, _dev_ptr(scale_a, "scale_a", dev), _dev_ptr(w_gate, "w_gate", dev),
        _dev_ptr(scale_gate, "scale_gate", dev), _dev_ptr(w_up, "w_up", dev), _dev_ptr(scale_up, "scale_up", dev), fb,
        M, I, K, _act_of(act), _dtype_code(out, "out"), _dev_ptr(out, "out", dev),
        _dev_ptr(_status_word(status), "status", dev), _stream(stream, dev)), "fp8q_gated_mm_blockwise")


def fp8q_gated_mm_blockwise_quant(a: torch.Tensor, scale_a: torch.Tensor, w_gate: torch.Tensor,
                                  scale_gate: torch.Tensor, w_up: torch.Tensor, scale_up: torch.Tensor,
                                  q: torch.Tensor, scale_inv: torch.Tensor, act=ACT_SILU, fa=None, fb=None, fmt=E4M3FN,
                                  rule=SCALE_IEEE, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """fp8q_gated_mm_blockwise with the result cast, unrounded, to fp8 codes q [M, I] and scale_inv
    [M, ceil(I/128)]: the activations of the fp8q_scaled_mm_blockwise that follows."""
    M, I, K, fa, fb = _gated_operands(a, w_gate, w_up, fa, fb)
    dev = a.device
    ib = _fine_scales(M, I, K, scale_a, scale_gate, scale_up)
    _need(q, M * I, "q", byte=True)
    _need(scale_inv, M * ib, "scale_inv", dtype=torch.float32)
    _check(lib().fp8q_gated_mm_blockwise_quant(
        _dev_ptr(a, "a"), fa, _dev_ptr(scale_a, "scale_a", dev), _dev_ptr(w_gate, "w_gate", dev),
        _dev_ptr(scale_gate, "scale_gate", dev), _dev_ptr(w_up, "w_up", dev), _dev_ptr(scale_up, "scale_up", dev), fb,
        M, I, K, _act_of(act), _fmt_of(fmt), _rule_of(rule), _dev_ptr(q, "q", dev),
        _dev_ptr(scale_inv, "scale_inv", dev), _dev_ptr(_status_word(status), "status", dev), _stream(stream, dev)),
        "fp8q_gated_mm_blockwise_quant")


def fp8q_gated_bwd_cast(dh: torch.Tensor, gate_up: torch.Tensor, q: torch.Tensor, scale_inv: torch.Tensor,
                        workspace: torch.Tensor, act=ACT_SILU, fmt=E5M2, rule=SCALE_IEEE, stream=None) -> None:
    """The gradients of gate and up from dh [M, I] and fp8q_gated_mm's gate_up [M, 2 I], cast with one
    scale into codes q [M, 2 I] and scale_inv [1]; workspace as fp8q_cast_per_tensor's."""
    if dh.dim() != 2 or gate_up.dim() != 2 or gate_up.shape != (dh.shape[0], 2 * dh.shape[1]):
        raise ValueError(f"dh must be [M, I] and gate_up [M, 2 I], got {tuple(dh.shape)} and {tuple(gate_up.shape)}")
    if gate_up.dtype != dh.dtype:
        raise TypeError("dh and gate_up must have one dtype")
    M, I = dh.shape
    dev = dh.device
    _need(q, 2 * M * I, "q", byte=True)
    _need(scale_inv, 1, "scale_inv", dtype=torch.float32)
    _check(lib().fp8q_gated_bwd_cast(
        _dev_ptr(dh, "dh"), _dev_ptr(gate_up, "gate_up", dev), _dtype_code(dh, "dh"), M, I, _act_of(act), _fmt_of(fmt),
        _dev_ptr(q, "q", dev), _dev_ptr(scale_inv, "scale_inv", dev), _dev_ptr(workspace, "workspace", dev),
        workspace.numel() * workspace.element_size(), _rule_of(rule), _stream(stream, dev)), "fp8q_gated_bwd_cast")


def _offsets(*sizes):
    """Offsets of parts of the given byte sizes in one buffer, 256-byte aligned, and its size."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + (n + 255 & ~255))
    return at


class _GatedLinearFp8(torch.autograd.Function):
    """gated_linear_fp8: _LinearFp8's casts and products around the gated kernel and its gradient.
    Keeps one buffer for the backward pass: the input's and the weight's codes and scales, and gate
    and up in the input's dtype.  Workspaces are the call's own, so that streams and graphs share none."""

    @staticmethod
    def forward(ctx, x, w, act):
        if x.dtype not in (torch.bfloat16, torch.float16) or x.dtype != w.dtype:
            raise TypeError("Only float16 and bfloat16 are allowed.")
        if w.dim() != 2 or w.shape[0] % 16 or x.shape[-1] != w.shape[1] or w.shape[1] % 16:
            raise ValueError(f"weight must be [2 I, K] with 2 I and K multiples of 16 and K the input's width, got "
                             f"{tuple(w.shape)} for an input of {tuple(x.shape)}")
        st = _on_device(x, w)
        L, code = lib(), _dtype_code(x, "input")
        x, w = x.contiguous(), w.contiguous()
        I, K = w.shape[0] // 2, w.shape[1]
        T = x.numel() // K if K else 0
        h = torch.empty((*x.shape[:-1], I), dtype=x.dtype, device=x.device)
        keep = ctx.needs_input_grad[0] or ctx.needs_input_grad[1]
        nws = _CAST_WORKSPACE()
        at = _offsets(T * K, 2 * I * K, 4, 4, nws, 4 * T * I if keep else 0)
        buf = torch.empty((at[-1],), dtype=torch.uint8, device=x.device)
        x8, w8, sx, sw, ws, gu, _ = (buf.data_ptr() + o for o in at)
        _check(L.fp8q_cast_per_tensor_ex(x.data_ptr(), code, T * K, E4M3FN, x8, sx, ws, nws, SCALE_IEEE, st),
               "fp8q_cast_per_tensor")
        _check(L.fp8q_cast_per_tensor_ex(w.data_ptr(), code, 2 * I * K, E4M3FN, w8, sw, ws, nws, SCALE_IEEE, st),
               "fp8q_cast_per_tensor")
        _check(L.fp8q_gated_mm(x8, E4M3FN, w8, w8 + I * K, E4M3FN, T, I, K, sx, sw, sw, act, code, h.data_ptr(),
                               gu if keep else None, None, st), "fp8q_gated_mm")
        ctx.sizes = act, T, I, K, at, x.shape, w.shape
        ctx.save_for_backward(buf)
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        (buf,) = ctx.saved_tensors
        st = _on_device(buf, dh)
        act, T, I, K, at, x_shape, w_shape = ctx.sizes
        x8, w8, sx, sw, _, gu, _ = (buf.data_ptr() + o for o in at)
        L, code = lib(), _dtype_code(dh, "the gradient")
        dh = dh.contiguous()
        nws = _CAST_WORKSPACE()
        to = _offsets(2 * T * I, 4, nws)
        tmp = torch.empty((to[-1],), dtype=torch.uint8, device=buf.device)
        d8, sd, ws, _ = (tmp.data_ptr() + o for o in to)
        _check(L.fp8q_gated_bwd_cast(dh.data_ptr(), gu, code, T, I, act, E5M2, d8, sd, ws, nws, SCALE_IEEE, st),
               "fp8q_gated_bwd_cast")
        dx = dw = None
        if ctx.needs_input_grad[0]:
            # dx[T, K] = d[T, 2 I] @ w[2 I, K], one product over gate's and up's columns together
            dx = torch.empty(x_shape, dtype=dh.dtype, device=buf.device)
            _check(L.fp8q_scaled_mm_ex(d8, E5M2, K_MAJOR, w8, E4M3FN, MN_MAJOR, T, K, 2 * I, sd, sw, None, code,
                                       dx.data_ptr(), None, st), "fp8q_scaled_mm_ex")
        if ctx.needs_input_grad[1]:
            # dw[2 I, K] = d^T[2 I, T] @ x[T, K], any token count
            dw = torch.empty(w_shape, dtype=dh.dtype, device=buf.device)
            _check(L.fp8q_scaled_mm_ex(d8, E5M2, MN_MAJOR, x8, E4M3FN, MN_MAJOR, 2 * I, K, T, sd, sx, None, code,
                                       dw.data_ptr(), None, st), "fp8q_scaled_mm_ex")
        return dx, dw, None


def gated_linear_fp8(input: torch.Tensor, weight: torch.Tensor, act="silu") -> torch.Tensor:
    """act(input @ Wg.t()) * (input @ Wu.t()) for weight = [Wg; Wu] of shape [2 I, K] (fp16 or bf16), with
    linear_fp8's per-tensor e4m3 casts of input and weight; differentiable, the gradients of gate and
    up cast together to e5m2.  The output has the input's dtype and last dimension I."""
    return _GatedLinearFp8.apply(input, weight, _act_of(act))


def gated_linear_fp8_blockwise(input: torch.Tensor, w_gate: torch.Tensor, scale_gate: torch.Tensor,
                               w_up: torch.Tensor, scale_up: torch.Tensor, act="silu") -> torch.Tensor:
    """act(input @ w_gate.t()) * (input @ w_up.t()) on fp8 weights [I, K] with 128 x 128 block scales: the
    input is quantised per token, as linear_fp8_blockwise does; the output has the input's dtype."""
    x = input.contiguous().reshape(-1, input.shape[-1])
    q, s = per_token_cast_to_fp8(x)
    h = torch.empty((x.shape[0], w_gate.shape[0]), dtype=input.dtype, device=input.device)
    fp8q_gated_mm_blockwise(q, s, w_gate, scale_gate, w_up, scale_up, h, act)
    return h.reshape(*input.shape[:-1], w_gate.shape[0])


def ffn_fp8(input: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor, act="silu") -> torch.Tensor:
    """A gated feed-forward block with per-tensor fp8 casts, differentiable:
    linear_fp8(gated_linear_fp8(input, w_gate_up), w_down)."""
    return linear_fp8(gated_linear_fp8(input, w_gate_up, act), w_down)


def ffn_fp8_blockwise(input: torch.Tensor, w_gate: torch.Tensor, scale_gate: torch.Tensor, w_up: torch.Tensor,
                      scale_up: torch.Tensor, w_down: torch.Tensor, scale_down: torch.Tensor,
                      norm_weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                      eps: float = 1e-6, act="silu"):
    """A gated feed-forward block on fp8 weights with 128 x 128 block scales, three launches from the
    input to the output: (with norm_weight) the residual's addition, the norm and its cast; the gated
    products and the cast of their result; the down projection w_down [N, I].  Returns the output in
    the input's dtype, or (output, input + residual) when a residual is given."""
    x = input.contiguous().reshape(-1, input.shape[-1])
    r = None
    if norm_weight is None:
        if residual is not None:
            raise ValueError("a residual needs norm_weight")
        q, s = per_token_cast_to_fp8(x)
    elif residual is None:
        q, s = rms_norm_cast_to_fp8(x, norm_weight, eps=eps)
    else:
        q, s, r = rms_norm_cast_to_fp8(x, norm_weight, residual.reshape(x.shape), eps)
    M, I = x.shape[0], w_gate.shape[0]
    h = torch.empty((M, I), dtype=torch.float8_e4m3fn, device=x.device)
    sh = torch.empty((M, -(-I // 128)), dtype=torch.float32, device=x.device)
    fp8q_gated_mm_blockwise_quant(q, s, w_gate, scale_gate, w_up, scale_up, h, sh, act)
    out = torch.empty((M, w_down.shape[0]), dtype=input.dtype, device=x.device)
    fp8q_scaled_mm_blockwise(h, sh, w_down, scale_down, out)
    out = out.reshape(*input.shape[:-1], w_down.shape[0])
    return out if r is None else (out, r.reshape(input.shape))
