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
