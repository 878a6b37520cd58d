"""The gated feed-forward products and their gradient on a GPU against the formulas in 64 bits.

Tolerances: a tensor-core sum over K products is within (K / 32 + 1) 2^-23 of the sum of their
magnitudes (the bound of the plain products' tests); with fine-grained scales that holds per
128-deep block, and the fold adds one rounding a block; a k axis split over a cluster adds seven
more.  plain64.gated carries such an error through the activation and the product."""
import pytest
import torch

import plain64 as P
from gpu_util import Guarded

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4, E5 = 0, 1


def gen(*key):
    return torch.Generator(device="cuda").manual_seed(sum((i + 1) * 7919 * k for i, k in enumerate(key)) % (1 << 31))


def codes(g, rows, k, fmt=E4):
    """Values N(0, 1) as fp8."""
    return torch.randn(rows, k, generator=g, device="cuda").to(P.FP8[fmt])


def fine_operands(M, I, K, fa=E4, fb=E4):
    g = gen(M, I, K)
    kb, ib = -(-K // 128), -(-I // 128)
    a = codes(g, M, K, fa)
    wg, wu = codes(g, I, K, fb), codes(g, I, K, fb)
    sa = torch.exp(0.5 * torch.randn(M, kb, generator=g, device="cuda"))
    sg = torch.exp(0.5 * torch.randn(ib, kb, generator=g, device="cuda")) / max(K, 1) ** 0.5
    su = torch.exp(0.5 * torch.randn(ib, kb, generator=g, device="cuda")) / max(K, 1) ** 0.5
    return a, sa, wg, sg, wu, su


def fine_error(K):
    return (2 * (4 + 1) + -(-K // 128) + 2 + 7) * P.U


def fine_reference(a, sa, wg, sg, wu, su, act):
    (M, K), I = a.shape, wg.shape[0]
    A = a.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    G = wg.double() * sg.double().repeat_interleave(128, 0)[:I].repeat_interleave(128, 1)[:, :K]
    W = wu.double() * su.double().repeat_interleave(128, 0)[:I].repeat_interleave(128, 1)[:, :K]
    return P.gated(A, G, W, act, fine_error(K))


def group_errors(e, h):
    """The largest error of each 1 x 128 group over its amax."""
    m, n = h.shape
    nb = -(-n // 128)
    p = torch.zeros(2, m, nb * 128, dtype=torch.float64, device=h.device)
    p[0, :, :n], p[1, :, :n] = e, h.abs()
    p = p.view(2, m, nb, 128).amax(3)
    return p[0] / p[1].clamp(min=1e-4)


def check_quant(fp8q, M, I, K, act="silu", fmt=E4, rule="ieee", fa=E4, fb=E4, q_offset=0):
    ops = fine_operands(M, I, K, fa, fb)
    q, s = Guarded(M * I, torch.uint8, offset=q_offset), Guarded(M * -(-I // 128), F32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8q.fp8q_gated_mm_blockwise_quant(*ops, q.t, s.t, act=act, fmt=fmt, rule=rule, status=status)
    q.check()
    s.check()
    assert status.item() == 0
    _, _, h, _, _, e = fine_reference(*ops, act)
    P.check_groups(q.t, s.t, h, 128, fmt, group_errors(e, h))
    q2, s2 = torch.empty_like(q.t), torch.empty_like(s.t)
    fp8q.fp8q_gated_mm_blockwise_quant(*ops, q2, s2, act=act, fmt=fmt, rule=rule)
    assert torch.equal(q.t, q2) and torch.equal(s.t, s2)             # the same bits again


# one tile, clusters of 8, 4 and 2, widths and depths that end inside a tile, row counts around a
# tile's, no cluster with idle SMs, more tiles than SMs
FINE = [(1, 128, 128), (1, 2048, 7168), (2, 4096, 1024), (9, 9000, 512), (7, 1000, 256), (64, 96, 1024),
        (127, 384, 2048), (128, 384, 512), (129, 256, 656), (300, 1001, 1040), (257, 4480, 256), (513, 8192, 128),
        (130, 16384, 384), (33, 40, 16), (1, 1, 48), (5, 130, 0)]


@pytest.mark.parametrize("M,I,K", FINE)
def test_blockwise_quant(fp8q, M, I, K):
    check_quant(fp8q, M, I, K)


@pytest.mark.parametrize("M,I,K,act,fmt,rule,fa,fb,offset", [
    (40, 520, 1536, "gelu_tanh", E4, "ieee", E4, E4, 0), (40, 520, 1536, "gelu_tanh", E5, "torch", E5, E4, 0),
    (700, 4224, 256, "gelu_tanh", E5, "ieee", E4, E5, 1), (16, 256, 1024, "silu", E4, "torch", E4, E4, 3)])
def test_blockwise_quant_variants(fp8q, M, I, K, act, fmt, rule, fa, fb, offset):
    check_quant(fp8q, M, I, K, act, fmt, rule, fa, fb, offset)


@pytest.mark.parametrize("yt", [BF16, F16, F32])
@pytest.mark.parametrize("M,I,K,act", [(1, 2048, 1024, "silu"), (70, 200, 528, "gelu_tanh"), (300, 1001, 256, "silu"),
                                       (600, 8192, 128, "silu"), (3, 64, 0, "silu")])
def test_blockwise(fp8q, yt, M, I, K, act):
    ops = fine_operands(M, I, K)
    out = Guarded(M * I, yt)
    fp8q.fp8q_gated_mm_blockwise(*ops, out.t, act=act)
    out.check()
    _, _, h, _, _, e = fine_reference(*ops, act)
    assert ((out.t.view(M, I).double() - h).abs() <= e + h.abs() * P.half_step(yt) + P.tiny(yt)).all()


def tensor_operands(M, I, K, fa=E4, fb=E4):
    g = gen(M, I, K, 3)
    a, w = codes(g, M, K, fa), codes(g, 2 * I, K, fb)
    s = [torch.tensor([v], device="cuda") for v in (0.75, 1.25 / max(K, 1) ** 0.5, 2.0 / max(K, 1) ** 0.5)]
    return a, w[:I], w[I:], *s


def check_tensor(fp8q, M, I, K, yt, act="silu", fa=E4, fb=E4, with_gu=True, offset=0):
    a, wg, wu, sa, sg, su = tensor_operands(M, I, K, fa, fb)
    out = Guarded(M * I, yt, offset=offset)
    gu = Guarded(2 * M * I, yt, offset=offset) if with_gu else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8q.fp8q_gated_mm(a, wg, wu, sa, sg, su, out.t, gu.t if with_gu else None, act, status=status)
    out.check()
    assert status.item() == 0
    # the product of the scales is one rounding more
    gate, up, h, eg, eu, e = P.gated(a.double() * sa.double(), wg.double() * sg.double(), wu.double() * su.double(), act,
                                     (2 * (-(-K // 32) + 1) + 3 + 7) * P.U)
    assert ((out.t.view(M, I).double() - h).abs() <= e + h.abs() * P.half_step(yt) + P.tiny(yt)).all()
    if with_gu:
        gu.check()
        got = gu.t.view(M, 2 * I).double()
        for v, t, er in ((got[:, :I], gate, eg), (got[:, I:], up, eu)):
            assert ((v - t).abs() <= er + t.abs() * P.half_step(yt) + P.tiny(yt)).all()
    again = torch.empty_like(out.t)
    fp8q.fp8q_gated_mm(a, wg, wu, sa, sg, su, again, None, act)
    assert torch.equal(again, out.t)


# the same at the borders between the kernel's forms: at most 16, 32 and 64 rows with a cluster for a
# tile (copies of the rows) and with a tile for each CTA (operands swapped), and persistent tiles
# whose rows are no multiples of 32 bytes (words, bytes), of 16 and of an element
@pytest.mark.parametrize("M,I,K", [(16, 2048, 1024), (17, 2048, 1024), (32, 18000, 256), (33, 9000, 256), (64, 1536, 640),
                                   (64, 18432, 128), (65, 9500, 128), (3, 18944, 128), (2, 19000, 128), (30, 19072, 256),
                                   (300, 8972, 256), (300, 9001, 128), (300, 8976, 128), (140, 19001, 48),
                                   (1, 9600, 1040), (16, 10000, 640), (17, 9601, 2000), (31, 9473, 16), (9, 9472, 0)])
def test_blockwise_forms(fp8q, M, I, K):
    check_quant(fp8q, M, I, K)
    for yt in (BF16, F32):
        ops = fine_operands(M, I, K)
        out = Guarded(M * I, yt)
        fp8q.fp8q_gated_mm_blockwise(*ops, out.t)
        out.check()
        _, _, h, _, _, e = fine_reference(*ops, "silu")
        assert ((out.t.view(M, I).double() - h).abs() <= e + h.abs() * P.half_step(yt) + P.tiny(yt)).all()


@pytest.mark.parametrize("yt", [BF16, F16, F32])
@pytest.mark.parametrize("M,I,K", [(250, 9001, 128), (200, 9501, 64), (250, 9004, 128), (100, 600, 1600), (128, 2048, 2048)])
def test_per_tensor_forms(fp8q, yt, M, I, K):
    check_tensor(fp8q, M, I, K, yt)


# one CTA a tile, clusters, and (from 67 tiles of 256 rows) CTA pairs
@pytest.mark.parametrize("yt", [BF16, F16, F32])
@pytest.mark.parametrize("M,I,K", [(1, 128, 128), (300, 384, 1024), (64, 2048, 2048), (257, 1001, 256), (512, 4352, 256),
                                   (1000, 2305, 384), (256, 8576, 48), (2000, 4096, 144), (4, 16, 0), (512, 8576, 0)])
def test_per_tensor(fp8q, yt, M, I, K):
    check_tensor(fp8q, M, I, K, yt)


@pytest.mark.parametrize("M,I,K,act,fa,fb,with_gu,offset", [
    (600, 4224, 256, "gelu_tanh", E4, E4, True, 0), (600, 4224, 256, "silu", E5, E4, False, 4),
    (90, 300, 512, "gelu_tanh", E4, E5, True, 4)])
def test_per_tensor_variants(fp8q, M, I, K, act, fa, fb, with_gu, offset):
    check_tensor(fp8q, M, I, K, BF16, act, fa, fb, with_gu, offset)


@pytest.mark.parametrize("M,I,K", [(60, 300, 2048), (600, 4224, 256), (600, 200, 128)])
def test_exact_sums_give_exact_gate_and_up(fp8q, M, I, K):
    """Integer operands of magnitude up to 4: every partial sum is an fp32 number."""
    g = gen(M, I, K, 9)
    a = torch.randint(-4, 5, (M, K), generator=g, device="cuda").float().to(P.FP8[E4])
    w = torch.randint(-4, 5, (2 * I, K), generator=g, device="cuda").float().to(P.FP8[E4])
    one = torch.ones(1, device="cuda")
    h, gu = torch.empty(M, I, device="cuda"), torch.empty(M, 2 * I, device="cuda")
    fp8q.fp8q_gated_mm(a, w[:I], w[I:], one, one, one, h, gu)
    assert torch.equal(gu.double(), a.double() @ w.double().t())


def test_a_nan_stays_in_its_row_and_empty_calls_write_nothing(fp8q):
    for M, I, K in ((40, 256, 1024), (300, 4224, 256)):
        a, sa, wg, sg, wu, su = fine_operands(M, I, K)
        q, s = torch.empty(M, I, dtype=torch.uint8, device="cuda"), torch.empty(M, -(-I // 128), device="cuda")
        fp8q.fp8q_gated_mm_blockwise_quant(a, sa, wg, sg, wu, su, q, s)
        a2 = a.clone()
        a2.view(torch.uint8)[17, 5] = 0x7F
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        fp8q.fp8q_gated_mm_blockwise_quant(a2, sa, wg, sg, wu, su, q2, s2)
        rest = torch.arange(M, device="cuda") != 17
        assert torch.equal(q[rest], q2[rest]) and torch.equal(s[rest], s2[rest])
        assert s2[17].isnan().all() and (q2[17] & 0x7F == 0x7F).all()
    e = torch.empty(0, 256, dtype=P.FP8[E4], device="cuda")
    w, sw = torch.zeros(64, 256, dtype=P.FP8[E4], device="cuda"), torch.ones(1, 2, device="cuda")
    fp8q.fp8q_gated_mm_blockwise(e, torch.empty(0, 2, device="cuda"), w, sw, w, sw, torch.empty(0, 64, device="cuda"))
    assert fp8q.gated_linear_fp8(torch.empty(0, 64, dtype=BF16, device="cuda"),
                                 torch.ones(32, 64, dtype=BF16, device="cuda")).shape == (0, 16)


def test_extreme_gates(fp8q):
    """Gates of +-200 and 0: the exponential overflows or vanishes, the value does not."""
    a = torch.ones(4, 128, dtype=P.FP8[E4], device="cuda")
    g = torch.tensor([200.0, -200.0, 0.0, -88.0, 30.0, -30.0, 1e30, -1e30], device="cuda")
    one = torch.ones(4, 1, device="cuda")
    eye = torch.zeros(1024, 128, dtype=P.FP8[E4], device="cuda")
    eye[::128, 0] = 1.0                                      # one live row in each 128-row block
    up = eye.clone()
    for act in ("silu", "gelu_tanh"):
        out = torch.empty(4, 1024, device="cuda")
        fp8q.fp8q_gated_mm_blockwise(a, one, eye, g.view(8, 1), up, torch.ones(8, 1, device="cuda"), out, act=act)
        want = P.act(g.double(), act)[0]
        p = P.exponent(g.double(), act)[0].abs().clamp(max=104)
        assert ((out[:, ::128].double() - want).abs() <= (16 + 8 * p) * P.U * want.abs() + 1e-36).all(), act


# ---------------------------------------------------------------------------
# the elementwise backward
# ---------------------------------------------------------------------------
def check_bwd(fp8q, M, I, dt, act, fmt=E5, rule="ieee", offset=0, scale=1.0):
    g = gen(M, I, 11)
    n = M * I
    buf = torch.randn(3 * n + offset, generator=g, device="cuda")
    dh = (buf[:n].view(M, I) * 1e-2 * scale).to(dt)
    gu = torch.zeros(2 * n + offset, dtype=dt, device="cuda")[offset:].view(M, 2 * I)
    gu.copy_((2 * buf[n:3 * n].view(M, 2 * I)).to(dt))
    q, s = Guarded(2 * n, torch.uint8, offset=offset), Guarded(1, F32)
    ws = torch.empty(fp8q.fp8q_cast_per_tensor_workspace_bytes(), dtype=torch.uint8, device="cuda")
    fp8q.fp8q_gated_bwd_cast(dh, gu, q.t, s.t, ws, act, fmt, rule)
    q.check()
    s.check()
    gate, up, d = gu[:, :I].double(), gu[:, I:].double(), dh.double()
    v, dv = P.act(gate, act)
    p, dp = P.exponent(gate, act)
    sig = torch.sigmoid(p)
    want = torch.cat((d * up * dv, d * v), 1)
    unit = (24 + 8 * p.abs()) * P.U
    err = torch.cat((unit * (d * up).abs() * (sig + (gate * sig * (1 - sig) * dp).abs()), unit * (d * v).abs()), 1)
    amax = want.abs().max()
    e_amax = err.max()
    assert abs(s.t.item() - (amax / P.FMAX[fmt]).item()) <= (e_amax / P.FMAX[fmt]).item() + 4 * P.U * s.t.item()
    z = want * (P.FMAX[fmt] / amax)
    got = q.t.view(M, 2 * I).view(P.FP8[fmt]).double()
    tol = torch.clamp(z.abs() * P.HALF[fmt], min=P.TINY[fmt]) * (1 + 8 * P.U) + \
        err * (P.FMAX[fmt] / amax) + z.abs() * (e_amax / amax + 8 * P.U)
    assert ((got - z).abs() <= tol).all()


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,I", [(1, 16), (300, 384), (77, 1000), (5, 8), (3, 7), (1, 1), (700, 4096), (4100, 260)])
def test_gated_bwd_cast(fp8q, dt, act, M, I):
    check_bwd(fp8q, M, I, dt, act)


@pytest.mark.parametrize("M,I,dt,fmt,rule,offset", [(64, 512, BF16, E4, "torch", 0), (64, 512, F16, E5, "torch", 1),
                                                    (64, 512, F32, E4, "ieee", 4), (64, 512, BF16, E5, "ieee", 8)])
def test_gated_bwd_cast_variants(fp8q, M, I, dt, fmt, rule, offset):
    check_bwd(fp8q, M, I, dt, "silu", fmt, rule, offset)


def test_gated_bwd_cast_zero_nan_and_extremes(fp8q):
    ws = torch.empty(fp8q.fp8q_cast_per_tensor_workspace_bytes(), dtype=torch.uint8, device="cuda")
    s = torch.empty(1, device="cuda")
    for I in (64, 63):
        dh = torch.zeros(3, I, dtype=BF16, device="cuda")
        gu = torch.ones(3, 2 * I, dtype=BF16, device="cuda")
        q = torch.full((3, 2 * I), 9, dtype=torch.uint8, device="cuda")
        fp8q.fp8q_gated_bwd_cast(dh, gu, q, s, ws)
        assert (q & 0x7F == 0).all() and abs(s.item() - 1 / 57344) <= 2 * P.U / 57344      # a zero amax becomes 1
        # saturated gates: the derivative is 1 or 0, also where p' overflows
        dh.fill_(1.0)
        big = torch.tensor([3e38, -3e38, 1e20, -1e20, 200.0, -200.0], device="cuda").to(BF16)
        gu[0, :6] = big
        gu[:, I:] = 0.5
        for act in ("silu", "gelu_tanh"):
            fp8q.fp8q_gated_bwd_cast(dh * 1e-30, gu, q, s, ws, act, fp8q.E5M2)
            d = q[0, :6].view(P.FP8[E5]).double() * s.item()
            assert (d[1::2] == 0).all(), act
            assert d.isfinite().all()
        dh[1, 3] = float("nan")
        fp8q.fp8q_gated_bwd_cast(dh * 0 + dh, gu.clamp(-4, 4), q, s, ws)
        assert q[1, 3] & 0x7F == 0x7F and q[1, I + 3] & 0x7F == 0x7F                       # and the amax becomes 1
        assert abs(s.item() - 1 / 57344) <= 2 * P.U / 57344
        fp8q.fp8q_gated_bwd_cast(dh[:0], gu[:0], q, s, ws)
        assert s.item() == 1.0


# ---------------------------------------------------------------------------
# the differentiable layer, the blocks, streams and graphs
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,I,K,dt,act", [(300, 384, 1024, F16, "silu"), (37, 64, 256, BF16, "gelu_tanh"),
                                          (600, 4224, 256, BF16, "silu"), (1, 8, 16, BF16, "silu")])
def test_gated_linear_fp8_forward_and_backward(fp8q, T, I, K, dt, act):
    g = gen(T, I, K, 21)
    x = torch.randn(T, K, generator=g, device="cuda").to(dt).requires_grad_(True)
    w = (torch.randn(2 * I, K, generator=g, device="cuda") / K ** 0.5).to(dt).requires_grad_(True)
    dh = (torch.randn(T, I, generator=g, device="cuda") * 1e-2).to(dt)
    h = fp8q.gated_linear_fp8(x, w, act)
    dx, dw = torch.autograd.grad(h, (x, w), dh)
    # the casts are the library's own (tested bit for bit elsewhere)
    x8, sx = fp8q.cast_to_fp8(x.detach())
    w8, sw = fp8q.cast_to_fp8(w.detach())
    X, W = x8.double() * sx.double(), w8.double() * sw.double()
    rel = (2 * (-(-K // 32) + 1) + 3 + 7) * P.U
    _, _, want, _, _, e = P.gated(X, W[:I], W[I:], act, rel)
    assert ((h.detach().double() - want).abs() <= e + want.abs() * P.half_step(dt) + P.tiny(dt)).all()
    # the gradients from the gate, up and codes that the C calls give on the same operands
    gu, out = torch.empty(T, 2 * I, dtype=dt, device="cuda"), torch.empty(T, I, dtype=dt, device="cuda")
    fp8q.fp8q_gated_mm(x8, w8[:I], w8[I:], sx, sw, sw, out, gu, act)
    assert torch.equal(out, h.detach())
    d8, sd = torch.empty(T, 2 * I, dtype=torch.float8_e5m2, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(fp8q.fp8q_cast_per_tensor_workspace_bytes(), dtype=torch.uint8, device="cuda")
    fp8q.fp8q_gated_bwd_cast(dh, gu, d8, sd, ws, act)
    D = d8.double() * sd.double()
    for got, a, b, k in ((dx, D, W, 2 * I), (dw, D.t(), X, T)):
        exact, mag = a @ b, a.abs() @ b.abs()
        tol = (2 * (-(-k // 32) + 1) + 4) * P.U * mag + exact.abs() * P.half_step(dt) + P.tiny(dt)
        assert ((got.double() - exact).abs() <= tol).all()
    # and D itself is the formula's gradient to within half a step of e5m2 of it and of its amax's share
    gate, up = gu[:, :I].double(), gu[:, I:].double()
    v, dv = P.act(gate, act)
    f = torch.cat((dh.double() * up * dv, dh.double() * v), 1)
    tol = f.abs() * (P.HALF[E5] + 1e-4) + f.abs().max() * (P.TINY[E5] / 57344 + 1e-5)
    assert ((D - f).abs() <= tol).all()
    # one gradient alone is the same
    (only,) = torch.autograd.grad(fp8q.gated_linear_fp8(x, w.detach(), act), x, dh)
    assert torch.equal(only, dx)


def test_leading_dimensions_and_strides(fp8q):
    g = gen(5)
    x = torch.randn(64, 2, 3, generator=g, device="cuda").to(BF16).permute(1, 2, 0)        # [2, 3, 64], strided
    w = torch.randn(64, 64, generator=g, device="cuda").to(BF16).t()
    h = fp8q.gated_linear_fp8(x, w)
    assert h.shape == (2, 3, 32)
    assert torch.equal(h.reshape(6, 32), fp8q.gated_linear_fp8(x.contiguous().view(6, 64), w.contiguous()))


def block_weight(g, rows, k):
    return codes(g, rows, k), torch.exp(0.3 * torch.randn(-(-rows // 128), -(-k // 128), generator=g, device="cuda")) / k ** 0.5


@pytest.mark.parametrize("M,I,K", [(1, 2048, 1024), (70, 400, 512), (300, 4224, 384)])
@pytest.mark.parametrize("res", [False, True])
def test_ffn_blockwise_together(fp8q, M, I, K, res):
    """The serving block is its three calls, bit for bit, and each is the formula's on what it reads."""
    g = gen(M, I, K, 31)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    r = torch.randn(M, K, generator=g, device="cuda").to(BF16) if res else None
    nw = (1 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(BF16)
    (wg, sg), (wu, su), (wd, sd) = block_weight(g, I, K), block_weight(g, I, K), block_weight(g, K, I)
    got = fp8q.ffn_fp8_blockwise(x, wg, sg, wu, su, wd, sd, nw, r)
    out, total = got if res else (got, None)
    cast = fp8q.rms_norm_cast_to_fp8(x, nw, r)
    q, s = cast[:2]
    if res:
        assert torch.equal(total, cast[2]) and torch.equal(total.double(), P.norm(x, nw, r, 1e-6)[0])
    P.check_groups(q.view(torch.uint8), s, P.norm(x, nw, r, 1e-6)[2], 128, E4, 64 * P.U)
    hq, hs = torch.empty(M, I, dtype=P.FP8[E4], device="cuda"), torch.empty(M, -(-I // 128), device="cuda")
    fp8q.fp8q_gated_mm_blockwise_quant(q, s, wg, sg, wu, su, hq, hs)
    _, _, h, _, _, e = fine_reference(q, s, wg, sg, wu, su, "silu")
    P.check_groups(hq.view(torch.uint8), hs, h, 128, E4, group_errors(e, h))
    assert torch.equal(out, fp8q.scaled_mm_blockwise(hq, hs, wd, sd))
    A = hq.double() * hs.double().repeat_interleave(128, 1)[:, :I]
    D = wd.double() * sd.double().repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :I]
    exact, mag = A @ D.t(), A.abs() @ D.abs().t()
    assert ((out.double() - exact).abs() <= fine_error(I) * mag + exact.abs() * P.half_step(BF16)).all()
    plain = fp8q.ffn_fp8_blockwise(x, wg, sg, wu, su, wd, sd)
    hp = fp8q.gated_linear_fp8_blockwise(x, wg, sg, wu, su)
    assert plain.shape == x.shape and hp.shape == (M, I)
    _, _, h, _, _, e = fine_reference(*fp8q.per_token_cast_to_fp8(x), wg, sg, wu, su, "silu")
    assert ((hp.double() - h).abs() <= e + h.abs() * P.half_step(BF16) + P.tiny(BF16)).all()


def test_training_block_together(fp8q):
    """norm -> gated products -> down projection with autograd: the gradients are those of the parts."""
    g = gen(77)
    T, K, I = 130, 256, 192
    x = torch.randn(T, K, generator=g, device="cuda").to(BF16).requires_grad_(True)
    res = torch.randn(T, K, generator=g, device="cuda").to(BF16).requires_grad_(True)
    nw = torch.ones(K, device="cuda", requires_grad=True)
    w = (torch.randn(2 * I, K, generator=g, device="cuda") / K ** 0.5).to(BF16).requires_grad_(True)
    wd = (torch.randn(K, I, generator=g, device="cuda") / I ** 0.5).to(BF16).requires_grad_(True)
    y, r = fp8q.rms_norm(x, nw, res)
    out = r + fp8q.ffn_fp8(y, w, wd)
    dout = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    grads = torch.autograd.grad(out, (x, res, nw, w, wd), dout)
    assert torch.equal(grads[0], grads[1])
    # by parts
    y2 = y.detach().requires_grad_(True)
    h = fp8q.gated_linear_fp8(y2, w)
    h2 = h.detach().requires_grad_(True)
    dh, dwd = torch.autograd.grad(fp8q.linear_fp8(h2, wd), (h2, wd), dout)
    dy, dw = torch.autograd.grad(h, (y2, w), dh)
    assert torch.equal(dw, grads[3]) and torch.equal(dwd, grads[4])
    r64, rstd, _ = P.norm(x.detach(), nw.detach(), res.detach(), 1e-6)
    want, want_w, mag, mag_w = P.norm_grad(r64, nw.detach(), rstd, dy, dout)
    assert ((grads[0].double() - want).abs() <= 60 * P.U * mag + want.abs() * P.half_step(BF16)).all()
    assert ((grads[2].double() - want_w).abs() <= (T + 70) * P.U * mag_w).all()


def test_streams_and_graph_replay(fp8q):
    """Two streams at once, and a captured graph replayed on new inputs, give the eager calls' bits."""
    small, large = fine_operands(3, 1024, 2048), fine_operands(400, 4224, 384)
    outs = []
    for ops in (small, large):
        M, I = ops[0].shape[0], ops[2].shape[0]
        outs.append((torch.empty(M, I, dtype=torch.uint8, device="cuda"), torch.empty(M, I // 128, device="cuda")))
    for ops, o in zip((small, large), outs):
        fp8q.fp8q_gated_mm_blockwise_quant(*ops, *o)
    want = [[t.clone() for t in o] for o in outs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for o in outs:
        o[0].zero_()
    torch.cuda.synchronize()
    for _ in range(8):
        for st, ops, o in zip(streams, (small, large), outs):
            fp8q.fp8q_gated_mm_blockwise_quant(*ops, *o, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    a, wg, wu, sa, sg, su = tensor_operands(300, 512, 1024)
    h, gu = torch.empty(300, 512, dtype=BF16, device="cuda"), torch.empty(300, 1024, dtype=BF16, device="cuda")
    d8, sd = torch.empty(300, 1024, dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(fp8q.fp8q_cast_per_tensor_workspace_bytes(), dtype=torch.uint8, device="cuda")

    def step():
        fp8q.fp8q_gated_mm(a, wg, wu, sa, sg, su, h, gu)
        fp8q.fp8q_gated_bwd_cast(h, gu, d8, sd, ws)
        fp8q.fp8q_gated_mm_blockwise_quant(*small, *outs[0])

    with torch.cuda.stream(streams[0]):
        step()
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin()
        step()
        graph.capture_end()
    torch.cuda.synchronize()
    a.copy_(codes(gen(1, 2), 300, 1024))
    small[0].copy_(codes(gen(2, 2), 3, 2048))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (h, gu, d8, sd, *outs[0])]
    step()
    torch.cuda.synchronize()
    for x, y in zip(got, (h, gu, d8, sd, *outs[0])):
        assert torch.equal(x, y)


def test_offsets_past_32_bits(fp8q):
    """gate_up of more than 2^31 elements: rows from both ends, forward and backward."""
    M, I, K = 66000, 16512, 16
    a, wg, wu, sa, sg, su = tensor_operands(M, I, K)
    h, gu = torch.empty(M, I, dtype=BF16, device="cuda"), torch.empty(M, 2 * I, dtype=BF16, device="cuda")
    assert gu.numel() > 1 << 31
    fp8q.fp8q_gated_mm(a, wg, wu, sa, sg, su, h, gu)
    d8, sd = torch.empty(M, 2 * I, dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(fp8q.fp8q_cast_per_tensor_workspace_bytes(), dtype=torch.uint8, device="cuda")
    fp8q.fp8q_gated_bwd_cast(h, gu, d8, sd, ws)
    rows = torch.tensor([0, 1, 65023, 65024, 65999], device="cuda")
    gate, up, want, eg, eu, e = P.gated(a[rows].double() * sa.double(), wg.double() * sg.double(), wu.double() * su.double(),
                                        "silu", 16 * P.U)
    assert ((h[rows].double() - want).abs() <= e + want.abs() * P.half_step(BF16) + P.tiny(BF16)).all()
    assert ((gu[rows][:, I:].double() - up).abs() <= eu + up.abs() * P.half_step(BF16)).all()
    g64, u64, d = gu[rows][:, :I].double(), gu[rows][:, I:].double(), h[rows].double()
    v, dv = P.act(g64, "silu")
    f = torch.cat((d * u64 * dv, d * v), 1)
    D = d8[rows].view(P.FP8[E5]).double() * sd.double()
    assert ((D - f).abs() <= f.abs() * (P.HALF[E5] + 1e-4) + 57344 * sd.item() * (P.TINY[E5] / 57344 + 1e-5)).all()


# every form of the kernel that casts, with a last group shorter than 128 columns
@pytest.mark.parametrize("how", ["scale of a row", "scale of a block", "code"])
@pytest.mark.parametrize("M,I,K", [(3, 200, 256), (40, 200, 256), (100, 200, 1024), (300, 9504, 128), (300, 9001, 128),
                                   (300, 9004, 128), (4, 9672, 256), (20, 9504, 256)])
def test_an_infinite_row_has_infinite_scales_in_a_short_group_too(fp8q, M, I, K, how):
    """Positive operands, so that an infinity among them makes its row's (or block's) gate, up and h
    infinite and no value NaN; what stands past the last column is no part of its group."""
    kb, ib, row = -(-K // 128), -(-I // 128), M // 2
    fa = E5 if how == "code" else E4
    a = torch.ones(M, K, device="cuda").to(P.FP8[fa])
    w = torch.ones(I, K, device="cuda").to(P.FP8[E4])
    sa, sg = torch.ones(M, kb, device="cuda"), torch.ones(ib, kb, device="cuda")
    hit = torch.zeros(M, ib, dtype=torch.bool, device="cuda")
    if how == "scale of a row":
        sa[row, 0] = float("inf")
        hit[row] = True
    elif how == "scale of a block":
        sg[ib - 1, 0] = float("inf")
        hit[:, ib - 1] = True
    else:
        a.view(torch.uint8)[row, 7] = 0x7C
        hit[row] = True
    q, s = torch.empty(M, I, dtype=torch.uint8, device="cuda"), torch.empty(M, ib, device="cuda")
    fp8q.fp8q_gated_mm_blockwise_quant(a, sa, w, sg, w, sg, q, s, fa=fa, fb=E4)
    assert torch.equal(s.isinf(), hit) and (s > 0).all()
    # h = K * sigmoid(K) * K = K^2 elsewhere (sigmoid(128) is 1), which is a group's amax: the largest code
    cols = hit.repeat_interleave(128, 1)[:, :I]
    assert (q[~cols] == 0x7E).all() and (q[cols] == 0x7F).all()
    assert ((s[~hit].double() - K * K / 448).abs() <= 8 * P.U * K * K / 448).all()
