"""Norm and gated feed-forward operators of libfp8q: marshalling, as the rest of the binding.  The
calls that a step makes between launches (the norms, the fine-grained gated products, the two autograd
functions) have theirs in C++ (csrc/torch_ops.cpp), where it costs a third.

Entry points with the C names (caller-provided outputs, nothing allocated):
    fp8q_rms_norm_quant, fp8q_rms_norm_bwd, fp8q_cast_per_tensor_pair
    fp8q_gated_mm, fp8q_gated_mm_blockwise, fp8q_gated_mm_blockwise_quant, fp8q_gated_bwd_cast

Allocating helpers:
    rms_norm                     residual addition and root-mean-square norm (differentiable)
    rms_norm_cast_to_fp8         the same with the result cast to 1 x G fp8 groups
    gated_linear_fp8             act(x Wg^T) * (x Wu^T) with linear_fp8's casts (differentiable)
    gated_linear_fp8_blockwise   the same on block-scaled weights
    ffn_fp8, ffn_fp8_blockwise   the whole block: the gated products, then the down projection
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (E4M3FN, E5M2, SCALE_IEEE, _FMT_DTYPE, _FP8_DTYPES, _check, _dev_ptr, _dtype_code, _fmt_of, _need, _rule_of,
               _status_word, _stream, fp8q_scaled_mm_blockwise, lib, linear_fp8, per_token_cast_to_fp8)

__all__ = [
    "fp8q_rms_norm_quant", "fp8q_rms_norm_bwd", "fp8q_rms_norm_bwd_workspace_bytes",
    "rms_norm", "rms_norm_cast_to_fp8",
    "fp8q_cast_per_tensor_pair", "ACT_SILU", "ACT_GELU_TANH", "fp8q_gated_mm", "fp8q_gated_mm_blockwise", "fp8q_gated_mm_blockwise_quant",
    "fp8q_gated_bwd_cast", "gated_linear_fp8", "gated_linear_fp8_blockwise", "ffn_fp8", "ffn_fp8_blockwise",
]

ACT_SILU, ACT_GELU_TANH = 0, 1
_ops = None


def _native():
    """The binding's C++ part (raises if it has not been built)."""
    global _ops
    if _ops is None:
        lib()
        try:
            from . import _fp8q_torch
        except ImportError as e:
            raise ImportError("_fp8q_torch.so is missing or was built against another torch; build it with "
                              "`python -m dequantisation_fp8q_token_b200.build` (needs g++)") from e
        _ops = _fp8q_torch
    return _ops


def _handle(stream) -> Optional[int]:
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


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
    _native().rms_norm_quant(x, weight, y, q, scale_inv, residual, residual_out, rstd, eps, group, _fmt_of(fmt),
                             _rule_of(rule), _handle(stream))


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


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """Root-mean-square norm over the last dimension, times weight (x's dtype or fp32): returns y, or
    (y, x + residual) when a residual is given.  Differentiable in x, weight and residual."""
    return _native().rms_norm(x, weight, residual, eps)


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
_ACTS = {"silu": ACT_SILU, "gelu_tanh": ACT_GELU_TANH}


def _act_of(act) -> int:
    if isinstance(act, str):
        if act not in _ACTS:
            raise ValueError(f'act must be "silu" or "gelu_tanh", got {act!r}')
        return _ACTS[act]
    code = int(act)
    return code if 0 <= code <= 0x7FFFFFFF else -1           # an unknown number is refused by the library, uncut


def fp8q_cast_per_tensor_pair(x0: torch.Tensor, q0: torch.Tensor, scale_inv0: torch.Tensor, x1: torch.Tensor,
                              q1: torch.Tensor, scale_inv1: torch.Tensor, workspace: torch.Tensor, fmt=E4M3FN,
                              rule=SCALE_IEEE, stream=None) -> None:
    """fp8q_cast_per_tensor_ex of two tensors of one dtype (a product's operands), with the same bytes, in two
    launches where they are 16 MB together at most, start on 16 bytes and are whole 16-byte vectors;
    workspace as fp8q_cast_per_tensor's."""
    if x0.dtype != x1.dtype:
        raise TypeError("the two tensors must have one dtype")
    dev = x0.device
    for q, s, x in ((q0, scale_inv0, x0), (q1, scale_inv1, x1)):
        _need(q, x.numel(), "q", byte=True)
        _need(s, 1, "scale_inv", dtype=torch.float32)
    _check(lib().fp8q_cast_per_tensor_pair(
        _dev_ptr(x0, "x0"), x0.numel(), _dev_ptr(q0, "q0", dev), _dev_ptr(scale_inv0, "scale_inv0", dev),
        _dev_ptr(x1, "x1", dev), x1.numel(), _dev_ptr(q1, "q1", dev), _dev_ptr(scale_inv1, "scale_inv1", dev),
        _dtype_code(x0, "x0"), _fmt_of(fmt), _dev_ptr(workspace, "workspace", dev),
        workspace.numel() * workspace.element_size(), _rule_of(rule), _stream(stream, dev)), "fp8q_cast_per_tensor_pair")


def _fmt_or_none(fmt) -> Optional[int]:
    return None if fmt is None else _fmt_of(fmt)


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
    act = _act_of(act)
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
        act, _dtype_code(out, "out"), _dev_ptr(out, "out", dev), _dev_ptr(gate_up, "gate_up", dev),
        _dev_ptr(_status_word(status), "status", dev), _stream(stream, dev)), "fp8q_gated_mm")


def fp8q_gated_mm_blockwise(a: torch.Tensor, scale_a: torch.Tensor, w_gate: torch.Tensor, scale_gate: torch.Tensor,
                            w_up: torch.Tensor, scale_up: torch.Tensor, out: torch.Tensor, act=ACT_SILU, fa=None,
                            fb=None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """fp8q_gated_mm with fine-grained scales: scale_a [M, ceil(K/128)] per 1 x 128 group, scale_gate and
    scale_up [ceil(I/128), ceil(K/128)] per 128 x 128 block."""
    _native().gated_mm_blockwise(a, scale_a, w_gate, scale_gate, w_up, scale_up, out, _act_of(act), _fmt_or_none(fa),
                                 _fmt_or_none(fb), status, _handle(stream))


def fp8q_gated_mm_blockwise_quant(a: torch.Tensor, scale_a: torch.Tensor, w_gate: torch.Tensor,
                                  scale_gate: torch.Tensor, w_up: torch.Tensor, scale_up: torch.Tensor,
                                  q: torch.Tensor, scale_inv: torch.Tensor, act=ACT_SILU, fa=None, fb=None, fmt=E4M3FN,
                                  rule=SCALE_IEEE, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """fp8q_gated_mm_blockwise with the result cast, unrounded, to fp8 codes q [M, I] and scale_inv
    [M, ceil(I/128)]: the activations of the fp8q_scaled_mm_blockwise that follows."""
    _native().gated_mm_blockwise_quant(a, scale_a, w_gate, scale_gate, w_up, scale_up, q, scale_inv, _act_of(act),
                                       _fmt_or_none(fa), _fmt_or_none(fb), _fmt_of(fmt), _rule_of(rule), status,
                                       _handle(stream))


def fp8q_gated_bwd_cast(dh: torch.Tensor, gate_up: torch.Tensor, q: torch.Tensor, scale_inv: torch.Tensor,
                        workspace: torch.Tensor, act=ACT_SILU, fmt=E5M2, rule=SCALE_IEEE, stream=None) -> None:
    """The gradients of gate and up from dh [M, I] and fp8q_gated_mm's gate_up [M, 2 I], cast with one
    scale into codes q [M, 2 I] and scale_inv [1]; workspace as fp8q_cast_per_tensor's."""
    act = _act_of(act)
    if dh.dim() != 2 or gate_up.dim() != 2 or gate_up.shape != (dh.shape[0], 2 * dh.shape[1]):
        raise ValueError(f"dh must be [M, I] and gate_up [M, 2 I], got {tuple(dh.shape)} and {tuple(gate_up.shape)}")
    if gate_up.dtype != dh.dtype:
        raise TypeError("dh and gate_up must have one dtype")
    M, I = dh.shape
    dev = dh.device
    _need(q, 2 * M * I, "q", byte=True)
    _need(scale_inv, 1, "scale_inv", dtype=torch.float32)
    _check(lib().fp8q_gated_bwd_cast(
        _dev_ptr(dh, "dh"), _dev_ptr(gate_up, "gate_up", dev), _dtype_code(dh, "dh"), M, I, act, _fmt_of(fmt),
        _dev_ptr(q, "q", dev), _dev_ptr(scale_inv, "scale_inv", dev), _dev_ptr(workspace, "workspace", dev),
        workspace.numel() * workspace.element_size(), _rule_of(rule), _stream(stream, dev)), "fp8q_gated_bwd_cast")


def gated_linear_fp8(input: torch.Tensor, weight: torch.Tensor, act="silu") -> torch.Tensor:
    """act(input @ Wg.t()) * (input @ Wu.t()) for weight = [Wg; Wu] of shape [2 I, K] (fp16 or bf16), with
    linear_fp8's per-tensor e4m3 casts of input and weight; differentiable, the gradients of gate and
    up cast together to e5m2.  The output has the input's dtype and last dimension I."""
    return _native().gated_linear_fp8(input, weight, _act_of(act))


def gated_linear_fp8_blockwise(input: torch.Tensor, w_gate: torch.Tensor, scale_gate: torch.Tensor,
                               w_up: torch.Tensor, scale_up: torch.Tensor, act="silu") -> torch.Tensor:
    """act(input @ w_gate.t()) * (input @ w_up.t()) on fp8 weights [I, K] with 128 x 128 block scales: the
    input is quantised per token, as linear_fp8_blockwise does; the output has the input's dtype."""
    act = _act_of(act)
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
    act = _act_of(act)
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
