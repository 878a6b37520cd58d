"""The norm and feed-forward entry points without a GPU: host-side validation of every argument
before any CUDA call, and the binding's refusals."""
import pytest
import torch

P = 0x1000      # a fake, never-dereferenced pointer value
A = 0x10000


@pytest.fixture(scope="module")
def L():
    from dequantisation_fp8q_token_b200 import build
    build.build()
    import dequantisation_fp8q_token_b200 as fp8q
    return fp8q.lib()


def test_rms_norm_quant_validation(L):
    # x xt residual residual_out weight wt m n eps group fmt rule y q scale_inv rstd stream
    def f(x=P, xt=2, res=None, ro=None, w=P, wt=2, m=4, n=256, eps=1e-6, group=128, fmt=0, rule=0, y=None, q=P, s=P,
          rstd=None):
        return L.fp8q_rms_norm_quant(x, xt, res, ro, w, wt, m, n, eps, group, fmt, rule, y, q, s, rstd, None)
    assert f(xt=7) == 2                                  # dtype
    assert f(wt=1) == 2                                  # fp16 weight for bf16 rows
    assert f(xt=0, wt=2) == 2                            # bf16 weight for fp32 rows
    assert f(rule=2) == 10
    assert f(fmt=5) == 3
    assert f(m=-1) == 4 and f(n=-1) == 4 and f(m=1 << 31) == 4
    assert f(eps=-1.0) == 4 and f(eps=float("nan")) == 4
    assert f(group=0) == 4 and f(group=100) == 4         # n % group
    assert f(m=(1 << 31) - 1, n=(1 << 31) - 1, xt=0, wt=0, group=1) == 4     # bytes above 2^63
    assert f(x=None) == 1 and f(w=None) == 1
    assert f(y=None, q=None) == 1                        # neither output
    assert f(s=None) == 1                                # q without scale_inv
    assert f(res=P) == 1 and f(ro=P) == 1                # residual and residual_out go together
    assert f(x=P + 1) == 5 and f(w=P + 1) == 5 and f(res=P + 1, ro=P) == 5 and f(res=P, ro=P + 1) == 5
    assert f(y=P + 1) == 5 and f(s=P + 2) == 5 and f(rstd=P + 2) == 5
    assert f(m=0, x=None, w=None, q=None) == 0 and f(n=0) == 0


def test_rms_norm_bwd_validation(L):
    assert L.fp8q_rms_norm_bwd_workspace_bytes(-1, 8) == 0
    ws = L.fp8q_rms_norm_bwd_workspace_bytes(1000, 8)
    assert ws >= 8 * 4 and ws % 4 == 0

    def f(dy=P, r=P, xt=2, w=P, wt=2, rstd=P, dres=None, m=1000, n=8, dx=P, dw=P, work=A, nbytes=ws):
        return L.fp8q_rms_norm_bwd(dy, r, xt, w, wt, rstd, dres, m, n, dx, dw, work, nbytes, None)
    assert f(xt=3) == 2 and f(wt=1) == 2
    assert f(m=-1) == 4 and f(n=1 << 31) == 4
    assert f(dy=None) == 1 and f(r=None) == 1 and f(w=None) == 1 and f(rstd=None) == 1 and f(dx=None) == 1
    assert f(dy=P + 1) == 5 and f(dres=P + 1) == 5 and f(dw=P + 1) == 5 and f(rstd=P + 2) == 5
    assert f(work=None) == 6 and f(work=A + 4) == 6 and f(nbytes=ws - 1) == 6
    assert f(n=0) == 0 and f(m=0, dw=None) == 0


def test_host_tensors_and_wrong_shapes_are_refused(L):
    import dequantisation_fp8q_token_b200 as f
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    for call in (lambda: f.fp8q_rms_norm_quant(x, w, q=q, scale_inv=s), lambda: f.rms_norm(x, w),
                 lambda: f.rms_norm_cast_to_fp8(x, w),
                 lambda: f.fp8q_rms_norm_bwd(x, x, w, torch.zeros(4), x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: f.fp8q_rms_norm_quant(x, w[:128], q=q, scale_inv=s),                # width
                 lambda: f.fp8q_rms_norm_quant(x, w),                                        # no output
                 lambda: f.fp8q_rms_norm_quant(x, w, q=q),                                   # no scale_inv
                 lambda: f.fp8q_rms_norm_quant(x, w, q=q[:2], scale_inv=s),                  # q too small
                 lambda: f.fp8q_rms_norm_quant(x, w, q=q, scale_inv=s[:1]),                  # scale_inv too small
                 lambda: f.fp8q_rms_norm_quant(x, w, y=x, residual=x),                       # no residual_out
                 lambda: f.fp8q_rms_norm_quant(x, w, y=x, residual=x.float(), residual_out=x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        f.fp8q_rms_norm_quant(x, w, y=x.float())


def test_gated_validation(L):
    def f(a=A, fa=0, wg=A, wu=A, fb=0, M=4, I=32, K=64, sa=P, sg=P, su=P, act=0, yt=2, h=P, gu=None, st=None):
        return L.fp8q_gated_mm(a, fa, wg, wu, fb, M, I, K, sa, sg, su, act, yt, h, gu, st, None)

    def b(a=A, fa=0, wg=A, wu=A, fb=0, M=4, I=32, K=64, sa=P, sg=P, su=P, act=0, yt=2, h=P, st=None):
        return L.fp8q_gated_mm_blockwise(a, fa, sa, wg, sg, wu, su, fb, M, I, K, act, yt, h, st, None)

    def q(a=A, fa=0, wg=A, wu=A, fb=0, M=4, I=32, K=64, sa=P, sg=P, su=P, act=0, fmt=0, rule=0, h=P, sinv=P, st=None):
        return L.fp8q_gated_mm_blockwise_quant(a, fa, sa, wg, sg, wu, su, fb, M, I, K, act, fmt, rule, h, sinv, st, None)

    for c in (f, b, q):
        assert c(act=2) == 4 and c(act=-1) == 4                                   # unknown activation
        assert c(fa=2) == 3 and c(fb=7) == 3
        assert c(K=24) == 4 and c(M=-1) == 4 and c(I=-1) == 4 and c(I=1 << 31) == 4
        assert c(a=None) == 1 and c(wg=None) == 1 and c(wu=None) == 1 and c(h=None) == 1
        assert c(sa=None) == 1 and c(sg=None) == 1 and c(su=None) == 1
        assert c(a=A + 8) == 5 and c(wg=A + 8) == 5 and c(wu=A + 8) == 5
        assert c(sa=P + 2) == 5 and c(sg=P + 2) == 5 and c(su=P + 2) == 5 and c(st=P + 2) == 5
        assert c(M=0, a=None, h=None) == 0 and c(I=0, wg=None, wu=None, h=None) == 0
    assert f(yt=5) == 2 and b(yt=5) == 2
    assert f(h=P + 1) == 5 and b(h=P + 1) == 5 and f(gu=P + 1) == 5
    assert f(K=0, sa=None) == 1                                                   # the epilogue reads the scales
    assert q(fmt=3) == 3 and q(rule=2) == 10
    assert q(sinv=None) == 1 and q(sinv=P + 2) == 5


def test_gated_bwd_validation(L):
    ws = 8192

    def f(dh=P, gu=P, xt=2, M=4, I=32, act=0, fmt=1, q=P, s=P, w=A, nb=ws, rule=0):
        return L.fp8q_gated_bwd_cast(dh, gu, xt, M, I, act, fmt, q, s, w, nb, rule, None)
    assert f(xt=4) == 2 and f(rule=3) == 10 and f(fmt=2) == 3
    assert f(M=-1) == 4 and f(I=-1) == 4 and f(act=5) == 4 and f(M=1 << 62, I=4) == 4
    assert f(s=None) == 1 and f(dh=None) == 1 and f(gu=None) == 1 and f(q=None) == 1
    assert f(s=P + 2) == 5 and f(dh=P + 1) == 5 and f(gu=P + 1) == 5
    assert f(w=None) == 6 and f(nb=ws - 1) == 6 and f(w=A + 8) == 6


def test_cast_pair_validation(L):
    def f(x0=P, n0=64, q0=P, s0=P, x1=P, n1=64, q1=P, s1=P, xt=2, fmt=0, w=A, nb=8192, rule=0):
        return L.fp8q_cast_per_tensor_pair(x0, n0, q0, s0, x1, n1, q1, s1, xt, fmt, w, nb, rule, None)
    assert f(xt=5) == 2 and f(rule=2) == 10 and f(fmt=4) == 3
    assert f(n0=-1) == 4 and f(n1=-1) == 4 and f(n1=1 << 62) == 4
    assert f(x0=None) == 1 and f(q0=None) == 1 and f(s0=None) == 1 and f(x1=None) == 1 and f(q1=None) == 1 and f(s1=None) == 1
    assert f(s0=P + 2) == 5 and f(s1=P + 1) == 5 and f(x0=P + 1) == 5 and f(x1=P + 1) == 5
    assert f(w=None) == 6 and f(nb=8191) == 6 and f(w=A + 8) == 6
    import dequantisation_fp8q_token_b200 as b
    x, q, s, ws = torch.zeros(64), torch.zeros(64, dtype=torch.uint8), torch.zeros(1), torch.zeros(8192, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        b.fp8q_cast_per_tensor_pair(x, q, s, x, q, s, ws)
    with pytest.raises(ValueError):
        b.fp8q_cast_per_tensor_pair(x, q, s, x, q[:3], s, ws)
    with pytest.raises(TypeError):
        b.fp8q_cast_per_tensor_pair(x, q, s, x.half(), q, s, ws)


def test_gated_binding_refuses(L):
    import dequantisation_fp8q_token_b200 as f
    e4 = torch.float8_e4m3fn
    a, w, w2 = torch.zeros(4, 256, dtype=e4), torch.zeros(64, 256, dtype=e4), torch.zeros(32, 256, dtype=e4)
    sa, sw, one = torch.ones(4, 2), torch.ones(1, 2), torch.ones(1)
    h, gu = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=e4), torch.zeros(4, 1)
    ws = torch.zeros(8192, dtype=torch.uint8)
    x, wx = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(64, 256, dtype=torch.bfloat16)
    for call in (lambda: f.fp8q_gated_mm(a, w, w, one, one, one, h, gu),
                 lambda: f.fp8q_gated_mm_blockwise(a, sa, w, sw, w, sw, h),
                 lambda: f.fp8q_gated_mm_blockwise_quant(a, sa, w, sw, w, sw, q, s),
                 lambda: f.fp8q_gated_bwd_cast(h, gu, torch.zeros(4, 128, dtype=torch.uint8), one, ws),
                 lambda: f.gated_linear_fp8(x, wx), lambda: f.ffn_fp8(x, wx, torch.zeros(256, 32, dtype=torch.bfloat16)),
                 lambda: f.gated_linear_fp8_blockwise(x, w, sw, w, sw),
                 lambda: f.ffn_fp8_blockwise(x, w, sw, w, sw, torch.zeros(256, 64, dtype=e4), torch.ones(2, 1))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: f.fp8q_gated_mm(a, w, w2, one, one, one, h),                     # I differs
                 lambda: f.fp8q_gated_mm(a, w[:, :128], w[:, :128], one, one, one, h),    # K differs
                 lambda: f.fp8q_gated_mm(a, w, w, one, one, one, h[:2]),                  # out too small
                 lambda: f.fp8q_gated_mm(a, w, w, one, one, one, h, gu[:2]),              # gate_up too small
                 lambda: f.fp8q_gated_mm_blockwise(a, sa[:2], w, sw, w, sw, h),           # scales too few
                 lambda: f.fp8q_gated_mm_blockwise(a, sa, w, sw[:, :1], w, sw, h),
                 lambda: f.fp8q_gated_mm_blockwise_quant(a, sa, w, sw, w, sw, q, s[:2]),
                 lambda: f.fp8q_gated_bwd_cast(h, h, q, one, ws),                         # gate_up's width
                 lambda: f.gated_linear_fp8(x, wx[:, :128]), lambda: f.gated_linear_fp8(x, wx[:40]),
                 lambda: f.ffn_fp8_blockwise(x, w, sw, w, sw, w, sw, residual=x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f.fp8q_gated_mm(a, w, w.view(torch.float8_e5m2), one, one, one, h),
                 lambda: f.fp8q_gated_mm(a.float(), w, w, one, one, one, h),
                 lambda: f.fp8q_gated_mm(a, w, w, one, one, one, h, gu.float()),
                 lambda: f.gated_linear_fp8(x.float(), wx.float()), lambda: f.gated_linear_fp8(x, wx.half())):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_the_plain_derivative_is_that_of_differences(act):
    """The 64-bit activation that the GPU tests compare with: value against its definition as
    g * sigmoid(p(g)), derivative against central differences (error: the step squared)."""
    import plain64
    g = torch.linspace(-12, 12, 4001, dtype=torch.float64)
    v, d = plain64.act(g, act)
    p, dp = plain64.exponent(g, act)
    s = torch.sigmoid(p)
    assert (v - g * s).abs().max() < 1e-13
    assert (d - s * (1 + g * (1 - s) * dp)).abs().max() < 1e-12
    h = 1e-5
    assert (d - (plain64.act(g + h, act)[0] - plain64.act(g - h, act)[0]) / (2 * h)).abs().max() < 1e-9


@pytest.mark.parametrize("act", ["gelu", "SiLU", ""])
def test_an_unknown_activation_is_refused(L, act):
    """By its name, before anything else is looked at."""
    import dequantisation_fp8q_token_b200 as f
    e4 = torch.float8_e4m3fn
    a, w = torch.zeros(4, 256, dtype=e4), torch.zeros(64, 256, dtype=e4)
    sa, sw, one = torch.ones(4, 2), torch.ones(1, 2), torch.ones(1)
    h, gu = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.bfloat16)
    q, s, ws = torch.zeros(4, 64, dtype=e4), torch.zeros(4, 1), torch.zeros(8192, dtype=torch.uint8)
    x, wx = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(64, 256, dtype=torch.bfloat16)
    for call in (lambda: f.fp8q_gated_mm(a, w, w, one, one, one, h, act=act),
                 lambda: f.fp8q_gated_mm_blockwise(a, sa, w, sw, w, sw, h, act=act),
                 lambda: f.fp8q_gated_mm_blockwise_quant(a, sa, w, sw, w, sw, q, s, act=act),
                 lambda: f.fp8q_gated_bwd_cast(h, gu, torch.zeros(4, 128, dtype=torch.uint8), one, ws, act=act),
                 lambda: f.gated_linear_fp8(x, wx, act), lambda: f.gated_linear_fp8_blockwise(x, w, sw, w, sw, act),
                 lambda: f.ffn_fp8(x, wx, torch.zeros(256, 32, dtype=torch.bfloat16), act),
                 lambda: f.ffn_fp8_blockwise(x, w, sw, w, sw, torch.zeros(256, 64, dtype=e4), torch.ones(2, 1), act=act)):
        with pytest.raises(ValueError, match="act must be"):
            call()


@pytest.mark.parametrize("act", [2, -1, 1 << 31, 1 << 32, (1 << 32) + 1, 1 << 70])
def test_an_unknown_number_stays_unknown(L, act):
    """What the binding hands on for it is refused by the library; nothing is cut to a number that there is."""
    import dequantisation_fp8q_token_b200 as f
    code = f.ffn._act_of(act)
    assert L.fp8q_gated_bwd_cast(P, P, 2, 4, 32, code, 1, P, P, A, 8192, 0, None) == 4
    assert [f.ffn._act_of(a) for a in ("silu", "gelu_tanh", f.ACT_SILU, f.ACT_GELU_TANH)] == [0, 1, 0, 1]
