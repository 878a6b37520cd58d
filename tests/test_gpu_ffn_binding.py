"""The native part of the norm and feed-forward binding on a GPU: refusals and status errors, streams,
empty inputs, what the autograd functions leave behind, and training steps inside CUDA graphs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def rand(*shape, seed=0, dt=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=g, device="cuda").to(dt)


def fine(M, I, K):
    a, wg, wu = (rand(r, K, seed=i).to(torch.float8_e4m3fn) for i, r in enumerate((M, I, I)))
    kb, ib = -(-K // 128), -(-I // 128)
    return a, torch.ones(M, kb, device="cuda"), wg, torch.ones(ib, kb, device="cuda"), wu, torch.ones(ib, kb, device="cuda")


def test_status_errors_and_refusals(fp8q):
    x, w = rand(4, 256), rand(256)
    q, s = torch.zeros(4, 256, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, device="cuda")
    for kw, status in (({"eps": -1.0}, 4), ({"group": 0}, 4), ({"group": 100}, 4), ({"fmt": 7}, 3), ({"rule": 5}, 10),
                       ({"group": 1 << 40}, 4)):
        with pytest.raises(fp8q.Fp8qError) as e:
            fp8q.fp8q_rms_norm_quant(x, w, q=q, scale_inv=s, **kw)
        assert e.value.status == status and "fp8q_rms_norm_quant" in str(e.value)
    with pytest.raises(fp8q.Fp8qError):
        fp8q.rms_norm(x, w, eps=-1.0)
    with pytest.raises(fp8q.Fp8qError):
        fp8q.rms_norm(x, w.half())                                           # fp16 weight for bf16 rows
    ops = fine(4, 64, 256)
    h, hs = torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), torch.zeros(4, 1, device="cuda")
    for kw, status in (({"act": 5}, 4), ({"fmt": 9}, 3), ({"fa": 9}, 3), ({"rule": 4}, 10)):
        with pytest.raises(fp8q.Fp8qError) as e:
            fp8q.fp8q_gated_mm_blockwise_quant(*ops, h, hs, **kw)
        assert e.value.status == status
    with pytest.raises(fp8q.Fp8qError) as e:
        fp8q.gated_linear_fp8(x, rand(64, 256), act=3)
    assert e.value.status == 4
    for call in (lambda: fp8q.fp8q_rms_norm_quant(x, w.cpu(), q=q, scale_inv=s),
                 lambda: fp8q.fp8q_rms_norm_quant(x, w, q=q.cpu(), scale_inv=s),
                 lambda: fp8q.fp8q_rms_norm_quant(x.t().contiguous().t(), w, q=q, scale_inv=s),      # not contiguous
                 lambda: fp8q.rms_norm(x, w.cpu()), lambda: fp8q.rms_norm(x, w, residual=x.cpu()),
                 lambda: fp8q.rms_norm(x, w, residual=x[:2]),
                 lambda: fp8q.gated_linear_fp8(x, rand(64, 256).cpu()),
                 lambda: fp8q.fp8q_gated_mm_blockwise_quant(*ops[:5], ops[5].cpu(), h, hs)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fp8q.fp8q_rms_norm_quant(x.double(), w, q=q, scale_inv=s), lambda: fp8q.rms_norm(x.double(), w),
                 lambda: fp8q.fp8q_gated_mm_blockwise_quant(*ops, h, hs, status=torch.zeros(1, device="cuda")),
                 lambda: fp8q.fp8q_rms_norm_quant(x, w, q=x, scale_inv=s)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("dt", [BF16, torch.float16, torch.float32])
@pytest.mark.parametrize("n0,n1,offset", [(300 * 1024, 768 * 1024, 0), (16, 8, 0), (8, 4 << 20, 0), (1000, 2001, 0),
                                          (5000, 4096, 1), (0, 64, 0), (64, 0, 0), (0, 0, 0), (9 << 20, 9 << 20, 0)])
def test_cast_pair_is_two_casts(fp8q, dt, n0, n1, offset):
    """Bit for bit, also where one has a NaN, only zeros, or values that overflow the scale."""
    ws = torch.empty(fp8q.fp8q_cast_per_tensor_workspace_bytes(), dtype=torch.uint8, device="cuda")
    for fmt, rule, kind in ((0, "ieee", "plain"), (1, "torch", "plain"), (0, "ieee", "nan"), (1, "ieee", "zero"), (0, "torch", "tiny")):
        xs = [rand(n + offset, seed=i, dt=dt)[offset:] for i, n in enumerate((n0, n1))]
        if kind == "nan" and n1:
            xs[1][n1 // 2] = float("nan")
        if kind == "zero":
            xs[0].zero_()
        if kind == "tiny":
            xs[0].mul_(1e-39)
        got, want = [], []
        for x in xs:
            for o in (got, want):
                o += [torch.full((x.numel(),), 7, dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")]
            fp8q.fp8q_cast_per_tensor_ex(x, want[-2], want[-1], ws, fmt, rule)
        fp8q.fp8q_cast_per_tensor_pair(xs[0], got[0], got[1], xs[1], got[2], got[3], ws, fmt, rule)
        for a, b in zip(got, want):
            assert torch.equal(a, b), (fmt, rule, kind)


def test_streams_given_as_objects_and_handles(fp8q):
    x, w = rand(64, 1024), rand(1024)
    want_q, want_s = fp8q.rms_norm_cast_to_fp8(x, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, None):
        q, s = torch.zeros(64, 1024, dtype=torch.uint8, device="cuda"), torch.zeros(64, 8, device="cuda")
        torch.cuda.synchronize()
        fp8q.fp8q_rms_norm_quant(x, w, q=q, scale_inv=s, stream=stream)
        (side if stream is not None else torch.cuda.current_stream()).synchronize()
        assert torch.equal(q, want_q.view(torch.uint8)) and torch.equal(s, want_s)
    ops = fine(9, 256, 512)
    h, hs = torch.zeros(9, 256, dtype=torch.uint8, device="cuda"), torch.zeros(9, 2, device="cuda")
    fp8q.fp8q_gated_mm_blockwise_quant(*ops, h, hs)
    h2, hs2 = torch.zeros_like(h), torch.zeros_like(hs)
    torch.cuda.synchronize()
    fp8q.fp8q_gated_mm_blockwise_quant(*ops, h2, hs2, stream=side)
    side.synchronize()
    assert torch.equal(h, h2) and torch.equal(hs, hs2)


def test_empty_inputs(fp8q):
    w = rand(256).requires_grad_(True)
    x = rand(0, 256).requires_grad_(True)
    y, r = fp8q.rms_norm(x, w, residual=x.detach())
    assert y.shape == r.shape == (0, 256)
    dx, dw = torch.autograd.grad((y, r), (x, w), (y.detach(), r.detach()))
    assert dx.shape == (0, 256) and (dw == 0).all()                          # no rows: zeros
    wide = rand(64, 256, seed=3).requires_grad_(True)
    h = fp8q.gated_linear_fp8(x, wide)
    assert h.shape == (0, 32)
    dx, dw = torch.autograd.grad(h, (x, wide), h.detach())
    assert dx.shape == (0, 256) and dw.shape == (64, 256) and (dw == 0).all()
    # no products to sum: zeros, whatever the memory held
    x, none = rand(2, 5, 0).requires_grad_(True), rand(64, 0).requires_grad_(True)
    del h
    torch.full((1 << 16,), float("nan"), device="cuda", dtype=BF16)
    h = fp8q.gated_linear_fp8(x, none)
    assert h.shape == (2, 5, 32) and (h == 0).all()
    dx, dw = torch.autograd.grad(h, (x, none), torch.ones_like(h))
    assert dx.shape == (2, 5, 0) and dw.shape == (64, 0)


def test_gradients_of_leaves_are_their_own(fp8q):
    """x's and the residual's gradients are equal, and neither changes with the other; a second
    backward pass adds to both."""
    x, r, w = rand(8, 128), rand(8, 128, seed=1), rand(128)
    for t in (x, r, w):
        t.requires_grad_(True)
    y, s = fp8q.rms_norm(x, w, residual=r)
    (y.float().square().sum() + s.float().sum()).backward(retain_graph=True)
    first = x.grad.clone(), w.grad.clone()
    assert torch.equal(x.grad, r.grad)
    x.grad.zero_()
    assert torch.equal(r.grad, first[0])
    (y.float().square().sum() + s.float().sum()).backward()
    assert torch.equal(x.grad, first[0]) and torch.equal(r.grad, first[0] + first[0]) and torch.equal(w.grad, first[1] + first[1])


def test_nothing_is_kept_without_gradients(fp8q):
    x, w = rand(512, 1024), rand(2048, 1024)
    plain = fp8q.gated_linear_fp8(x, w)
    assert not plain.requires_grad
    w.requires_grad_(True)
    with torch.no_grad():
        assert not fp8q.gated_linear_fp8(x, w).requires_grad and not fp8q.rms_norm(x, w[0]).requires_grad
    h = fp8q.gated_linear_fp8(x, w)
    assert h.requires_grad and torch.equal(h.detach(), plain)
    (dw,) = torch.autograd.grad(h, w, torch.ones_like(h))
    assert dw.shape == w.shape


def test_a_second_derivative_is_refused(fp8q):
    x, w = rand(8, 128).requires_grad_(True), rand(128).requires_grad_(True)
    wide = rand(64, 128, seed=2).requires_grad_(True)
    for f in (lambda: fp8q.rms_norm(x, w), lambda: fp8q.gated_linear_fp8(x, wide)):
        y = f()
        (g,) = torch.autograd.grad(y, x, torch.ones_like(y), create_graph=True)
        (plain,) = torch.autograd.grad(f(), x, torch.ones_like(y))
        assert torch.equal(g.detach(), plain)
        with pytest.raises(RuntimeError, match="twice"):
            g.sum().backward()


def test_changed_inputs_are_noticed(fp8q):
    """An input that the backward pass reads may not be written in between."""
    x, w = rand(8, 128).requires_grad_(True), rand(128).requires_grad_(True)
    y = fp8q.rms_norm(x, w)
    with torch.no_grad():
        w.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y, x, torch.ones_like(y))


def test_training_steps_in_graphs(fp8q):
    """A block's forward and backward captured twice (two graphs, each with its own workspaces) and
    replayed in turn on new inputs gives the eager step's bits.  No eager graph of the leaves may
    live while a backward pass is captured: torch then orders the capture after that graph's
    stream, whatever the operators are, and the capture fails."""
    x, res, nw = rand(96, 256), rand(96, 256, seed=1), rand(256, seed=2)
    wg, wd = rand(256, 256, seed=3) / 16, rand(256, 128, seed=4) / 16
    leaves = [t.requires_grad_(True) for t in (x, res, nw, wg, wd)]

    def step():
        y, r = fp8q.rms_norm(x, nw, residual=res)
        out = fp8q.ffn_fp8(y, wg, wd) + r
        return (out.detach(), *torch.autograd.grad(out, leaves, torch.ones_like(out)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        step()
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = step()
            graphs.append((graph, out))
    torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        with torch.no_grad():
            x.copy_(rand(96, 256, seed=10 + i))
            res.copy_(rand(96, 256, seed=20 + i))
        graph, out = graphs[i % 2]
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_any_one_input_may_ask_for_its_gradient(fp8q):
    """The gradient of one input alone has the bits that it has beside the others'."""
    x, r, w = rand(700, 256), rand(700, 256, seed=1), rand(256, seed=2)
    dy, dr = rand(700, 256, seed=3), rand(700, 256, seed=4)
    wide = rand(64, 256, seed=5)
    dh = rand(700, 32, seed=6)

    def norm_grads(which):
        t = [v.clone().requires_grad_(i in which) for i, v in enumerate((x, r, w))]
        out = fp8q.rms_norm(t[0], t[2], residual=t[1])
        return torch.autograd.grad(out, [t[i] for i in which], (dy, dr))

    every = norm_grads((0, 1, 2))
    for i in range(3):
        assert torch.equal(norm_grads((i,))[0], every[i])

    def gated_grads(which):
        t = [v.clone().requires_grad_(i in which) for i, v in enumerate((x, wide))]
        return torch.autograd.grad(fp8q.gated_linear_fp8(*t), [t[i] for i in which], dh)

    every = gated_grads((0, 1))
    for i in range(2):
        assert torch.equal(gated_grads((i,))[0], every[i])
    # a gradient that is no memory of its own: expanded from one number
    a, b = x.clone().requires_grad_(True), x.clone().requires_grad_(True)
    fp8q.rms_norm(a, w).sum().backward()
    fp8q.rms_norm(b, w).backward(torch.ones_like(b))
    assert torch.equal(a.grad, b.grad)


def test_threads_on_streams_of_their_own(fp8q):
    """Four threads at once, each on its stream: every result has the bits of the call alone."""
    import threading
    x, w, wide = rand(600, 1024), rand(1024, seed=1), rand(512, 1024, seed=2)
    ops = fine(40, 2048, 1024)

    def work():
        a, b, c = (t.clone().requires_grad_(True) for t in (x, w, wide))
        y = fp8q.rms_norm(a, b)
        h = fp8q.gated_linear_fp8(y, c)
        grads = torch.autograd.grad(h, (a, b, c), torch.ones_like(h))
        q, s = torch.empty(40, 2048, dtype=torch.uint8, device="cuda"), torch.empty(40, 16, device="cuda")
        fp8q.fp8q_gated_mm_blockwise_quant(*ops, q, s)
        return [y.detach(), h.detach(), *grads, q, s]

    want = work()
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(5):
                    got[i] = work()
            stream.synchronize()
        except Exception as e:                      # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [0, 1, 3])
def test_blocks_of_few_tokens(fp8q, M):
    x = rand(M, 256)
    _, _, wg, sg, wu, su = fine(1, 128, 256)
    wd, sd = rand(256, 128, seed=7).to(torch.float8_e4m3fn), torch.ones(2, 1, device="cuda")
    out, r = fp8q.ffn_fp8_blockwise(x, wg, sg, wu, su, wd, sd, norm_weight=rand(256), residual=x)
    assert out.shape == r.shape == (M, 256) and out.isfinite().all() and torch.equal(r, x + x)
    assert fp8q.ffn_fp8_blockwise(x, wg, sg, wu, su, wd, sd).shape == (M, 256)
    assert fp8q.gated_linear_fp8_blockwise(x.view(M, 1, 256), wg, sg, wu, su).shape == (M, 1, 128)


def test_activation_numbers_past_32_bits(fp8q):
    ops, h, hs = fine(4, 64, 256), torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), torch.zeros(4, 1, device="cuda")
    x, w = rand(4, 256), rand(64, 256)
    for act in (1 << 32, (1 << 32) + 1, -1):
        for call in (lambda: fp8q.fp8q_gated_mm_blockwise_quant(*ops, h, hs, act=act), lambda: fp8q.gated_linear_fp8(x, w, act),
                     lambda: fp8q.ffn._native().gated_linear_fp8(x, w, act)):
            with pytest.raises(fp8q.Fp8qError) as e:
                call()
            assert e.value.status == 4
