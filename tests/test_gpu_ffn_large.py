"""The norm and gated operators on tensors of more than 2^31 elements.  The rows repeat every 4096, so
that those of an offset cut to 32 bits would show: each block of 4096 rows has the first one's bits."""
import pytest
import torch

import plain64 as P

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
B = 4096


def repeated(m, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = torch.randn(B, n, generator=g, device="cuda").to(BF16)
    out = torch.empty(m, n, dtype=BF16, device="cuda")
    for i in range(0, m, B):
        out[i:i + B] = rows[:m - i]
    return out


def same_blocks(t):
    return all(torch.equal(t[i:i + B].view(torch.uint8), t[:min(B, t.shape[0] - i)].view(torch.uint8))
               for i in range(B, t.shape[0], B))


# 2^31 elements and some rows more; rows of whole vectors and rows that are not
@pytest.mark.parametrize("n", [8192, 8191])
def test_norm_past_32_bits(fp8q, n):
    m = (1 << 31) // n + 700
    x, w = repeated(m, n, 0), (1 + 0.1 * torch.randn(n, device="cuda")).to(BF16)
    y, rstd = torch.empty_like(x), torch.empty(m, device="cuda")
    fp8q.fp8q_rms_norm_quant(x, w, y=y, rstd=rstd)
    assert same_blocks(y) and same_blocks(rstd)
    v = P.norm(x[-64:], w, None, 1e-6)[2]
    assert ((y[-64:].double() - v).abs() <= v.abs() * (64 * P.U + P.half_step(BF16)) + P.tiny(BF16)).all()
    dx, dw = y, torch.empty_like(w)                          # y is not wanted any more
    ws = torch.empty(fp8q.fp8q_rms_norm_bwd_workspace_bytes(m, n), dtype=torch.uint8, device="cuda")
    dy = repeated(m, n, 1)
    fp8q.fp8q_rms_norm_bwd(dy, x, w, rstd, dx, dw, ws)
    assert same_blocks(dx)
    r64, rstd64, _ = P.norm(x[-64:], w, None, 1e-6)
    want, _, mag, _ = P.norm_grad(r64, w, rstd64, dy[-64:], None)
    assert ((dx[-64:].double() - want).abs() <= 120 * P.U * mag + want.abs() * P.half_step(BF16) + P.tiny(BF16)).all()
    # dw: whole blocks and a rest.  A sum of m terms, of which each thread adds m / 148 at most and 296 partial sums join
    r64, rstd64, _ = P.norm(x[:B], w, None, 1e-6)
    terms = dy[:B].double() * r64 * rstd64
    whole, rest = m // B, m % B
    want, mag = whole * terms.sum(0) + terms[:rest].sum(0), whole * terms.abs().sum(0) + terms[:rest].abs().sum(0)
    assert ((dw.double() - want).abs() <= (m // 148 + 400) * P.U * mag + want.abs() * P.half_step(BF16)).all()
    if n % 128 == 0:
        q, s = torch.empty(m, n, dtype=torch.uint8, device="cuda"), torch.empty(m, n // 128, device="cuda")
        fp8q.fp8q_rms_norm_quant(x, w, q=q, scale_inv=s)
        assert same_blocks(q) and same_blocks(s)


@pytest.mark.parametrize("I", [18432, 18440])
def test_gated_past_32_bits(fp8q, I):
    K = 128
    m = (1 << 31) // I + 700
    a = repeated(m, K, 2).to(P.FP8[0])
    w = torch.randn(2 * I, K, device="cuda").to(P.FP8[0])
    sa, sw = torch.ones(m, 1, device="cuda"), torch.full((-(-I // 128), 1), 0.1, device="cuda")
    q, s = torch.empty(m, I, dtype=torch.uint8, device="cuda"), torch.empty(m, -(-I // 128), device="cuda")
    fp8q.fp8q_gated_mm_blockwise_quant(a, sa, w[:I], sw, w[I:], sw, q, s)
    assert same_blocks(q) and same_blocks(s)
    del q, s
    one, tenth = torch.ones(1, device="cuda"), torch.full((1,), 0.1, device="cuda")
    h, gu = torch.empty(m, I, dtype=BF16, device="cuda"), torch.empty(m, 2 * I, dtype=BF16, device="cuda")
    fp8q.fp8q_gated_mm(a, w[:I], w[I:], one, tenth, tenth, h, gu)
    assert same_blocks(h) and same_blocks(gu)
    gate, up, v, eg, eu, e = P.gated(a[-16:].double(), 0.1 * w[:I].double(), 0.1 * w[I:].double(), "silu", 30 * P.U)
    assert ((h[-16:].double() - v).abs() <= e + v.abs() * P.half_step(BF16) + P.tiny(BF16)).all()
    d8, sd = torch.empty(m, 2 * I, dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(fp8q.fp8q_cast_per_tensor_workspace_bytes(), dtype=torch.uint8, device="cuda")
    fp8q.fp8q_gated_bwd_cast(h, gu, d8, sd, ws)
    assert same_blocks(d8)
