"""fp8q_rms_norm_quant and fp8q_rms_norm_bwd on a GPU against the formulas in 64 bits.

Tolerances count roundings (U = 2^-24, half a step of fp32).  A row's sum of squares has only
positive terms; a thread adds at most max(32, n / 256) of them and ten more additions join the
threads, so its relative error is at most C = max(32, n / 256) + 10 roundings; rstd takes half of
it and four more (mean, eps, root, reciprocal), and v two products more: REL = C / 2 + 6.  The
backward pass's mean is such a sum of terms of either sign, so its error scales with the sum of
their magnitudes; dw adds at most m terms and 64 more partial sums."""
import pytest
import torch

import plain64 as P
from gpu_util import Guarded

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def rel(n):
    return ((max(32, n / 256) + 10) / 2 + 6) * P.U


def make(m, n, dt, res, w32=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + m * 31 + n)
    x = (torch.randn(m, n, generator=g, device="cuda") * torch.exp(torch.randn(m, 1, generator=g, device="cuda"))).to(dt)
    r = torch.randn(m, n, generator=g, device="cuda").to(dt) if res else None
    w = (1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(F32 if w32 else dt)
    return x, r, w


def shifted(t, offset):
    """The same values `offset` elements past an aligned address."""
    buf = torch.zeros(t.numel() + offset, dtype=t.dtype, device=t.device)
    buf[offset:].copy_(t.reshape(-1))
    return buf[offset:].view(t.shape)


def check_forward(fp8q, x, res, w, group=128, fmt=0, rule="ieee", eps=EPS, with_y=True, q_offset=0):
    m, n = x.shape
    q = Guarded(m * n, torch.uint8, offset=q_offset)
    s = Guarded(m * (n // group), F32)
    y = Guarded(m * n, x.dtype) if with_y else None
    r = Guarded(m * n, x.dtype) if res is not None else None
    rstd = Guarded(m, F32)
    fp8q.fp8q_rms_norm_quant(x, w, y=y.t if with_y else None, q=q.t, scale_inv=s.t, residual=res,
                             residual_out=r.t.view(m, n) if r else None, rstd=rstd.t, eps=eps, group=group, fmt=fmt,
                             rule=rule)
    for g in (q, s, y, r, rstd):
        if g is not None:
            g.check()
    r64, rstd64, v = P.norm(x, w, res, eps)
    e = rel(n)
    assert ((rstd.t.double() - rstd64.view(-1)).abs() <= e * rstd64.view(-1)).all()
    if r is not None:
        assert torch.equal(r.t.view(m, n).double(), r64)
    if with_y:
        tol = v.abs() * (e + P.half_step(x.dtype)) + P.tiny(x.dtype)
        assert ((y.t.view(m, n).double() - v).abs() <= tol).all()
    P.check_groups(q.t, s.t, v, group, fmt, e)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("m,n,group", [(1, 128, 128), (1, 7168, 128), (3, 256, 64), (37, 1024, 128), (5, 1000, 8),
                                       (4, 1000, 125), (130, 384, 32), (2, 18432, 128), (3, 32768, 256),
                                       (2, 33024, 128), (9, 7, 7), (300, 16, 16), (2, 2048, 512), (2, 4096, 1024)])
def test_forward(fp8q, dt, res, m, n, group):
    x, r, w = make(m, n, dt, res)
    check_forward(fp8q, x, r, w, group)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n,group", [(2048, 128), (1000, 100), (24576, 64)])
def test_forward_fp32_weight_e5m2_and_no_y(fp8q, dt, n, group):
    x, r, w = make(21, n, dt, True, w32=True)
    check_forward(fp8q, x, r, w, group, fmt=1, rule="torch", eps=1e-5, with_y=False)


@pytest.mark.parametrize("dt,offset", [(BF16, 1), (BF16, 8), (F16, 3), (F32, 1), (F32, 4)])
def test_forward_unaligned(fp8q, dt, offset):
    x, r, w = make(17, 1024, dt, True)
    check_forward(fp8q, shifted(x, offset), shifted(r, offset), shifted(w, 1 if offset < 4 else offset), q_offset=1)
    check_forward(fp8q, shifted(x, offset), r, w)


def test_the_cast_is_the_per_token_cast_of_the_fp32_norm(fp8q):
    """With fp32 rows y is the norm itself, so codes and scales equal fp8q_per_token_group_quant's
    of y, bit for bit, under both rules and formats."""
    x, r, w = make(67, 2048, F32, True)
    for fmt, rule in ((0, "ieee"), (0, "torch"), (1, "ieee"), (1, "torch")):
        y = torch.empty_like(x)
        q, s, ro = torch.empty(67, 2048, dtype=torch.uint8, device="cuda"), torch.empty(67, 16, device="cuda"), torch.empty_like(x)
        fp8q.fp8q_rms_norm_quant(x, w, y=y, q=q, scale_inv=s, residual=r, residual_out=ro, fmt=fmt, rule=rule)
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        fp8q.fp8q_per_token_group_quant_ex(y, q2, s2, 128, fmt, rule)
        assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("n", [1024, 1001])
def test_zero_rows_nan_and_inf_stay_in_their_rows(fp8q, n):
    x, _, w = make(5, n, BF16, False)
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, 5] = float("inf")
    group = 128 if n % 128 == 0 else n
    q, s = fp8q.rms_norm_cast_to_fp8(x, w, group=group)
    y = fp8q.rms_norm(x, w)
    assert (q[1].float() == 0).all() and torch.allclose(s[1], torch.full_like(s[1], 1e-4 / 448))
    assert q[2].float().isnan().all() and s[2].isnan().all() and y[2].isnan().all()
    # an infinite row: rstd is 0, so its finite elements are 0 and the infinite one NaN
    assert y[3, 5].isnan() and (y[3, :5] == 0).all() and (y[3, 6:] == 0).all()
    good = torch.tensor([0, 4], device="cuda")
    v = P.norm(x[good], w, None, EPS)[2]
    P.check_groups(q[good].contiguous().view(torch.uint8), s[good].contiguous(), v, group, 0, rel(n))


@pytest.mark.parametrize("n", [1024, 1000, 40000])
def test_the_sum_may_be_written_in_place(fp8q, n):
    for over in ("residual", "x"):
        x, r, w = make(11, n, BF16, True)
        want_r, _, v = P.norm(x, w, r, EPS)
        q, s = torch.empty(11, n, dtype=torch.uint8, device="cuda"), torch.empty(11, n // 8, device="cuda")
        out = r if over == "residual" else x
        fp8q.fp8q_rms_norm_quant(x, w, q=q, scale_inv=s, residual=r, residual_out=out, group=8)
        assert torch.equal(out.double(), want_r)
        P.check_groups(q, s, v, 8, 0, rel(n))


def test_empty_calls_write_nothing(fp8q):
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda")
    q, s = fp8q.rms_norm_cast_to_fp8(x, w, group=32)
    assert q.shape == (0, 64) and s.shape == (0, 2)
    dw = torch.full((64,), 7.0, device="cuda")
    fp8q.fp8q_rms_norm_bwd(x, x, w, torch.empty(0, device="cuda"), torch.empty_like(x), dw)
    assert (dw == 0).all()
    assert fp8q.rms_norm(torch.empty(3, 0, device="cuda"), torch.empty(0, device="cuda")).shape == (3, 0)


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------
def check_backward(fp8q, m, n, dt, res, w32=False, offset=0):
    x, r, w = make(m, n, dt, res, w32, seed=5)
    g = torch.Generator(device="cuda").manual_seed(m + n)
    dy = torch.randn(m, n, generator=g, device="cuda").to(dt)
    dr = torch.randn(m, n, generator=g, device="cuda").to(dt) if res else None
    r64, rstd64, _ = P.norm(x, w, r, EPS)
    rows, rstd = r64.to(dt), rstd64.view(-1).float()
    if offset:
        rows, dy, w = shifted(rows, offset), shifted(dy, offset), shifted(w, offset)
    dx, dw = Guarded(m * n, dt), Guarded(n, w.dtype)
    ws = Guarded(fp8q.fp8q_rms_norm_bwd_workspace_bytes(m, n), torch.uint8)
    fp8q.fp8q_rms_norm_bwd(dy, rows, w, rstd, dx.t.view(m, n), dw.t, ws.t, dr)
    for b in (dx, dw, ws):
        b.check()
    want, want_w, mag, mag_w = P.norm_grad(r64, w, rstd64, dy, dr)
    k = (max(32, n / 256) + 20) * P.U
    tol = k * mag + want.abs() * P.half_step(dt) + P.tiny(dt)
    assert ((dx.t.view(m, n).double() - want).abs() <= tol).all()
    tol = (m + 64 + 4) * P.U * mag_w + want_w.abs() * P.half_step(w.dtype) + P.tiny(w.dtype)
    assert ((dw.t.double() - want_w).abs() <= tol).all()
    # without dweight, and again: the same bits
    dx2 = torch.empty_like(dy)
    fp8q.fp8q_rms_norm_bwd(dy, rows, w, rstd, dx2, dres=dr)
    assert torch.equal(dx2.view(torch.uint8), dx.t.view(m, n).view(torch.uint8))
    dw2 = torch.empty_like(w)
    fp8q.fp8q_rms_norm_bwd(dy, rows, w, rstd, dx2, dw2, torch.empty_like(ws.t), dr)
    assert torch.equal(dw2, dw.t)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("m,n", [(1, 64), (3, 7168), (1000, 128), (333, 1000), (7, 18432), (5, 20480), (2, 20488),
                                 (40, 33), (2000, 1), (700, 4096), (1, 5)])
def test_backward(fp8q, dt, res, m, n):
    check_backward(fp8q, m, n, dt, res)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n", [2048, 999, 12288])
def test_backward_fp32_weight(fp8q, dt, n):
    check_backward(fp8q, 77, n, dt, True, w32=True)


@pytest.mark.parametrize("dt,offset", [(BF16, 1), (F16, 4), (F32, 2)])
def test_backward_unaligned(fp8q, dt, offset):
    check_backward(fp8q, 50, 1024, dt, True, offset=offset)


def test_gradient_against_differences(fp8q):
    """The gradients along a random direction against central differences of the formula in 64
    bits, whose own error is the step squared (1e-8) times third derivatives of order one."""
    m, n = 6, 96
    x, r, w = make(m, n, F32, True)
    g = torch.Generator(device="cuda").manual_seed(3)
    dy, dr = torch.randn(m, n, generator=g, device="cuda"), torch.randn(m, n, generator=g, device="cuda")
    for t in (x, r, w):
        t.requires_grad_(True)
    y, s = fp8q.rms_norm(x, w, residual=r)
    gx, gr, gw = torch.autograd.grad((y, s), (x, r, w), (dy, dr))
    assert torch.equal(gx, gr)

    def loss(x, r, w):
        z = x + r
        v = z * (z.square().mean(1, keepdim=True) + EPS).rsqrt() * w
        return (v * dy.double()).sum() + (z * dr.double()).sum()

    for grad, i in ((gx, 0), (gr, 1), (gw, 2)):
        args = [t.detach().double() for t in (x, r, w)]
        d = torch.randn(args[i].shape, generator=g, device="cuda").double()
        h = 1e-4
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + h * d, args[i] - h * d
        want = (loss(*hi) - loss(*lo)) / (2 * h)
        got = (grad.double() * d).sum()
        # r = x + residual is rounded to fp32 by the operator and not here: m n U of each term's size
        scale = (grad.double() * d).abs().sum()
        assert (got - want).abs() <= 64 * P.U * scale * 8 + 1e-5 * (1 + scale.sqrt())


def test_autograd_uses_only_what_is_asked(fp8q):
    x, r, w = make(9, 256, BF16, True)
    x.requires_grad_(True)
    y, s = fp8q.rms_norm(x, w, residual=r)
    (gx,) = torch.autograd.grad(s, x, torch.ones_like(s), retain_graph=True)      # only the sum
    assert torch.equal(gx, torch.ones_like(gx))
    (gx,) = torch.autograd.grad(y, x, torch.ones_like(y))                          # only the norm
    r64, rstd, _ = P.norm(x.detach(), w, r, EPS)
    want, _, mag, _ = P.norm_grad(r64, w, rstd, torch.ones_like(y), None)
    assert ((gx.double() - want).abs() <= 60 * P.U * mag + want.abs() * P.half_step(BF16)).all()
    # a transposed input and leading dimensions
    xt = torch.randn(256, 6, device="cuda").to(BF16).t()
    z = fp8q.rms_norm(xt.reshape(2, 3, 256), w)
    v = P.norm(xt.contiguous(), w, None, EPS)[2]
    assert ((z.view(6, 256).double() - v).abs() <= v.abs() * (rel(256) + P.half_step(BF16))).all()


def test_side_stream_and_graph_replay(fp8q):
    """The forward and backward captured into a graph and replayed on new inputs give what the
    eager calls give, bit for bit; a call inside a stream context runs on that stream."""
    x, r, w = make(64, 1024, BF16, True)
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randn(64, 1024, generator=g, device="cuda").to(BF16)
    q, s, ro = torch.empty(64, 1024, dtype=torch.uint8, device="cuda"), torch.empty(64, 8, device="cuda"), torch.empty_like(x)
    rstd, dx, dw = torch.empty(64, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(fp8q.fp8q_rms_norm_bwd_workspace_bytes(64, 1024), dtype=torch.uint8, device="cuda")

    def step():
        fp8q.fp8q_rms_norm_quant(x, w, q=q, scale_inv=s, residual=r, residual_out=ro, rstd=rstd)
        fp8q.fp8q_rms_norm_bwd(dy, ro, w, rstd, dx, dw, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin()
        step()
        graph.capture_end()
    torch.cuda.current_stream().wait_stream(side)
    x.copy_(make(64, 1024, BF16, False, seed=99)[0])
    graph.replay()
    got = [t.clone() for t in (q, s, ro, dx, dw)]
    step()
    for a, b in zip(got, (q, s, ro, dx, dw)):
        assert torch.equal(a, b)


# more rows than the one-launch backward pass takes, one vector a thread and more, widths that end
# inside a vector, and no vectors at all; and the forward's form for many wide rows
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("m,n", [(512, 520), (513, 520), (513, 4096), (600, 7168), (514, 7176), (520, 18432), (515, 20488),
                                 (700, 33), (513, 1001), (5000, 8)])
def test_backward_many_rows(fp8q, dt, res, m, n):
    check_backward(fp8q, m, n, dt, res)


@pytest.mark.parametrize("m", [300, 600])
def test_backward_many_rows_fp32_weight_and_unaligned(fp8q, m):
    check_backward(fp8q, m, 2048, BF16, True, w32=True)
    check_backward(fp8q, m, 999, F16, False, w32=True)
    for dt, offset in ((BF16, 1), (F32, 2)):
        check_backward(fp8q, m, 1024, dt, True, offset=offset)


@pytest.mark.parametrize("m,n,group", [(443, 7168, 128), (444, 7168, 128), (500, 4112, 16), (450, 16384, 128),
                                       (446, 8192, 256), (600, 5120, 64)])
def test_forward_many_wide_rows(fp8q, m, n, group):
    for dt, res in ((BF16, True), (F16, False), (F32, True)):
        x, r, w = make(m, n, dt, res)
        check_forward(fp8q, x, r, w, group)


# widths that no vector fits: aligned vectors that begin and end in other rows
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("m,n", [(700, 1001), (520, 100), (530, 4095), (513, 4097), (515, 8191), (3, 8193), (1, 1), (600, 2)])
def test_odd_widths(fp8q, dt, res, m, n):
    x, r, w = make(m, n, dt, res)
    y, rstd = Guarded(m * n, dt), Guarded(m, F32)
    out = Guarded(m * n, dt) if res else None
    fp8q.fp8q_rms_norm_quant(x, w, y=y.t, residual=r, residual_out=out.t.view(m, n) if res else None, rstd=rstd.t, eps=EPS)
    for g in (y, rstd, out):
        if g is not None:
            g.check()
    r64, rstd64, v = P.norm(x, w, r, EPS)
    assert ((rstd.t.double() - rstd64.view(-1)).abs() <= rel(n) * rstd64.view(-1)).all()
    assert ((y.t.view(m, n).double() - v).abs() <= v.abs() * (rel(n) + P.half_step(dt)) + P.tiny(dt)).all()
    if res:
        assert torch.equal(out.t.view(m, n).double(), r64)
    check_backward(fp8q, m, n, dt, res)


# rows that are no multiple of 16 bytes, each start inside a vector, with several rows a thread and
# with one, up to the widest row and above it
@pytest.mark.parametrize("dt,w32", [(BF16, False), (F16, True), (F32, False)])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("m,n", [(1500, 2049), (1501, 2050), (1502, 2051), (1503, 2052), (1504, 2053), (1505, 2054), (1506, 2055),
                                 (9999, 9), (20001, 65), (6001, 100), (2001, 3585), (1201, 7169), (700, 18001), (520, 20473),
                                 (513, 20481), (600, 1), (601, 7)])
def test_backward_shifted_rows(fp8q, dt, w32, res, m, n):
    check_backward(fp8q, m, n, dt, res, w32=w32)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_backward_shifted_rows_keep_apart(fp8q, dt, bad):
    """What one row holds reaches no other row's gradient, though they share vectors."""
    m, n = 1300, 1003
    x, _, w = make(m, n, dt, False)
    dy = torch.randn(m, n, device="cuda").to(dt)
    _, rstd, _ = P.norm(x, w, None, EPS)
    rstd = rstd.view(-1).float()
    want, got = torch.empty_like(x), torch.empty_like(x)
    fp8q.fp8q_rms_norm_bwd(dy, x, w, rstd, want)
    dy[::2], x[::2] = bad, bad
    fp8q.fp8q_rms_norm_bwd(dy, x, w, rstd, got)
    assert torch.equal(got[1::2], want[1::2])
    assert got[::2].isnan().all()


def test_backward_shifted_rows_in_place(fp8q):
    """A part of a larger buffer: the rows before and behind it are left as they were."""
    m, n = 1201, 1001
    x, _, w = make(m, n, BF16, False)
    dy = torch.randn(m, n, device="cuda").to(BF16)
    _, rstd, _ = P.norm(x, w, None, EPS)
    rstd = rstd.view(-1).float()
    want, buf = torch.empty_like(x), torch.full((m + 16, n), 7.0, device="cuda", dtype=BF16)
    fp8q.fp8q_rms_norm_bwd(dy, x, w, rstd, want)
    fp8q.fp8q_rms_norm_bwd(dy, x, w, rstd, buf[8:8 + m])
    assert torch.equal(buf[8:8 + m], want) and (buf[:8] == 7).all() and (buf[8 + m:] == 7).all()


def check_plain_forward(fp8q, dt, res, m, n, w32=False, offset=0):
    x, r, w = make(m, n, dt, res, w32, seed=11)
    if offset:
        x = shifted(x, offset)
    y, rstd = Guarded(m * n, dt), Guarded(m, F32)
    out = Guarded(m * n, dt) if res else None
    fp8q.fp8q_rms_norm_quant(x, w, y=y.t, residual=r, residual_out=out.t.view(m, n) if res else None, rstd=rstd.t, eps=EPS)
    for g in (y, rstd, out):
        if g is not None:
            g.check()
    r64, rstd64, v = P.norm(x, w, r, EPS)
    assert ((rstd.t.double() - rstd64.view(-1)).abs() <= rel(n) * rstd64.view(-1)).all()
    assert ((y.t.view(m, n).double() - v).abs() <= v.abs() * (rel(n) + P.half_step(dt)) + P.tiny(dt)).all()
    if res:
        assert torch.equal(out.t.view(m, n).double(), r64)
        # the sum in the place of x, and of the residual
        for place in (0, 1):
            a, b, y2 = x.clone(), r.clone(), torch.empty_like(x)
            fp8q.fp8q_rms_norm_quant(a, w, y=y2, residual=b, residual_out=(a, b)[place], eps=EPS)
            assert torch.equal((a, b)[place].view(-1), out.t)
            # an aligned copy of an unaligned x is summed in another order, so its y is held to the
            # bound that holds for every order and not to the bits
            assert ((y2.double() - v).abs() <= v.abs() * (rel(n) + P.half_step(dt)) + P.tiny(dt)).all()
            assert offset or torch.equal(y2.view(-1), y.t)


@pytest.mark.parametrize("dt,w32", [(BF16, False), (F16, True), (F32, False)])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("m,n", [(1, 1), (5, 3), (17, 9), (200, 2049), (201, 2050), (202, 2051), (203, 2052), (204, 2053), (205, 2054),
                                 (206, 2055), (3001, 65), (5, 4097), (40, 8191), (31, 16385), (9, 18001), (3, 32753), (3, 32769)])
def test_forward_shifted_rows(fp8q, dt, w32, res, m, n):
    check_plain_forward(fp8q, dt, res, m, n, w32)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("m,n", [(33, 1001), (7, 8191), (5, 8193)])
def test_forward_shifted_addresses(fp8q, dt, m, n):
    check_plain_forward(fp8q, dt, True, m, n, offset=1)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_forward_shifted_rows_keep_apart(fp8q, dt):
    x, r, w = make(300, 1003, dt, True)
    want, got, out = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    fp8q.fp8q_rms_norm_quant(x, w, y=want, residual=r, residual_out=out, eps=EPS)
    x[::2] = float("nan")
    fp8q.fp8q_rms_norm_quant(x, w, y=got, residual=r, residual_out=out, eps=EPS)
    assert torch.equal(got[1::2], want[1::2])
    assert got[::2].isnan().all()


# widths between those above: two rows a CTA and one, in fp32 the width from which memory for a row
# in flight, and not threads, says how many
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("n", [8192, 9216, 9217, 9220, 10237, 10240, 10244, 12288, 16384])
def test_backward_many_wide_rows(fp8q, dt, res, n):
    check_backward(fp8q, 600, n, dt, res)


def test_gradient_of_many_wide_fp32_rows(fp8q):
    m, n = 700, 10240
    x, r, w = make(m, n, F32, True)
    g = torch.Generator(device="cuda").manual_seed(4)
    dy, dr = torch.randn(m, n, generator=g, device="cuda"), torch.randn(m, n, generator=g, device="cuda")
    for t in (x, r, w):
        t.requires_grad_(True)
    gx, gr, gw = torch.autograd.grad(fp8q.rms_norm(x, w, residual=r, eps=EPS), (x, r, w), (dy, dr))
    r64, rstd64, _ = P.norm(x.detach(), w.detach(), r.detach(), EPS)
    want, want_w, mag, mag_w = P.norm_grad(r64, w.detach(), rstd64, dy, dr)
    # the forward's rstd is within rel(n), beside the backward's own roundings; it enters dx up to three times
    k = (max(32, n / 256) + 20) * P.U + 3 * rel(n)
    assert ((gx.double() - want).abs() <= k * mag + want.abs() * P.half_step(F32) + P.tiny(F32)).all()
    assert torch.equal(gx, gr)
    tol = ((m + 64 + 4) * P.U + rel(n)) * mag_w + want_w.abs() * P.half_step(F32) + P.tiny(F32)
    assert ((gw.double() - want_w).abs() <= tol).all()
