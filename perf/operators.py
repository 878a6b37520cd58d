"""The calls that the norm and feed-forward operators are measured by, with their plain forms.

Four kinds of call, which together are one feed-forward block on fp8 operands:

    norm_fp8     residual addition, root-mean-square norm, 1 x G group cast to fp8   (serving)
    norm_train   the same norm in the input's type, forward and backward             (training)
    gated_fp8    gate and up products of fp8 operands with 128-wide block scales,
                 act(gate) * up, and the cast of the result to fp8 groups            (serving)
    gated_train  per-tensor fp8 casts, gate and up products, act(gate) * up, and the
                 gradients of the input and of the weights                           (training)

``run`` computes a call with elementary torch operations in fp32 where ``own`` is
false and through the library's public entry points where it is true; ``exact``
is the same definition in binary64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
EPS = 1e-6
CLAMP = 1e-4                       # the smallest amax of a 1 x G group
GELU = 2.0 * math.sqrt(2.0 / math.pi)


def _lib():
    import dequantisation_fp8q_token_b200 as fp8q
    return fp8q


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token between two layers while decoding: launch and latency
        {"name": "norm_fp8_1x7168", "kind": "norm_fp8", "m": 1, "n": 7168, "dtype": "bf16", "residual": True,
         "group": 128, "fmt": "e4m3"},
        # a prompt, or a batch of them: the activations that the fp8 products take
        {"name": "norm_fp8_4096x7168", "kind": "norm_fp8", "m": 4096, "n": 7168, "dtype": "bf16", "residual": True,
         "group": 128, "fmt": "e4m3"},
        # the first norm of a model (no residual yet), short fp16 rows, an odd number of them
        {"name": "norm_fp8_333x2048_f16", "kind": "norm_fp8", "m": 333, "n": 2048, "dtype": "f16", "residual": False,
         "group": 128, "fmt": "e4m3"},
        # a training step's norm with its residual stream, forward and backward
        {"name": "norm_train_4096x7168", "kind": "norm_train", "m": 4096, "n": 7168, "dtype": "bf16",
         "residual": True, "w32": False},
        # many narrow rows in fp32, no residual, a width that is no multiple of 128
        {"name": "norm_train_7000x1000_f32", "kind": "norm_train", "m": 7000, "n": 1000, "dtype": "f32",
         "residual": False, "w32": True},
        # one token through a dense block's gate and up weights: weight streaming
        {"name": "gated_fp8_1x18432x7168", "kind": "gated_fp8", "m": 1, "i": 18432, "k": 7168, "out": "fp8",
         "act": "silu"},
        # a decoding batch through one expert's weights: few tiles, a long k axis
        {"name": "gated_fp8_64x2048x7168", "kind": "gated_fp8", "m": 64, "i": 2048, "k": 7168, "out": "fp8",
         "act": "silu"},
        # a prompt through a dense block: the products bound it
        {"name": "gated_fp8_4096x18432x7168", "kind": "gated_fp8", "m": 4096, "i": 18432, "k": 7168, "out": "fp8",
         "act": "silu"},
        # ragged rows and columns, the result left in bf16, the other activation
        {"name": "gated_fp8_333x7000x1024_bf16", "kind": "gated_fp8", "m": 333, "i": 7000, "k": 1024, "out": "bf16",
         "act": "gelu_tanh"},
        # a small training step, an odd number of tokens
        {"name": "gated_train_300x384x1024_f16", "kind": "gated_train", "m": 300, "i": 384, "k": 1024,
         "dtype": "f16", "act": "silu"},
        # a dense block's training step
        {"name": "gated_train_4096x18432x7168", "kind": "gated_train", "m": 4096, "i": 18432, "k": 7168,
         "dtype": "bf16", "act": "silu"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm_fp8", "norm_train", "gated_fp8", "gated_train"])
    if kind == "norm_fp8":
        group = rng.choice([128, 128, 128, 64, 32, 256])
        n = group * max(1, _log_int(rng, 256, 18432) // group)
        m = _log_int(rng, 1, max(2, min(16384, 4096 * 7168 // n)))
        return {"kind": kind, "m": m, "n": n, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "residual": rng.random() < 0.7, "group": group, "fmt": rng.choice(["e4m3", "e4m3", "e5m2"])}
    if kind == "norm_train":
        n = _log_int(rng, 64, 18432)
        n = n if rng.random() < 0.3 else -(-n // 64) * 64
        m = _log_int(rng, 1, max(2, min(16384, 4096 * 7168 // n)))
        return {"kind": kind, "m": m, "n": n, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "residual": rng.random() < 0.7, "w32": rng.random() < 0.3}
    m = _log_int(rng, 1, 4096)
    k = 16 * _log_int(rng, 8, 448)
    act = rng.choice(["silu", "silu", "gelu_tanh"])
    if kind == "gated_fp8":
        i = _log_int(rng, 64, 18432)
        i = i if rng.random() < 0.3 else -(-i // 128) * 128
        return {"kind": kind, "m": m, "i": i, "k": k, "out": rng.choice(["fp8", "fp8", "bf16", "f32"]), "act": act}
    return {"kind": kind, "m": m, "i": 8 * _log_int(rng, 8, 2304), "k": k, "dtype": rng.choice(["bf16", "f16"]),
            "act": act}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _outliers(g, v, share=1e-3, size=20.0):
    """A thousandth of the entries far out, as trained activations have them."""
    hit = torch.rand(v.shape, generator=g, device="cuda") < share
    return torch.where(hit, v * size, v)


def _block_weight(g, rows, k):
    """e4m3 codes uniform over the finite ones, one scale per 128 x 128 block."""
    c = torch.randint(0, 254, (rows, k), generator=g, device="cuda", dtype=torch.uint8)
    w = (c + (c >= 0x7F).to(torch.uint8)).view(torch.float8_e4m3fn)
    s = torch.exp(-9.5 + 0.5 * _normal(g, -(-rows // 128), -(-k // 128)))
    return w, s


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    kind, m = case["kind"], case["m"]
    if kind in ("norm_fp8", "norm_train"):
        n, dt = case["n"], DTYPES[case["dtype"]]
        st["x"] = (_outliers(g, _normal(g, m, n)) * torch.exp(0.5 * _normal(g, m, 1))).to(dt)
        st["res"] = (2.0 * _outliers(g, _normal(g, m, n))).to(dt) if case["residual"] else None
        wdt = torch.float32 if case.get("w32") else dt
        st["w"] = (1.0 + 0.2 * _normal(g, n)).to(wdt)
        if kind == "norm_fp8":
            # the buffers that a serving program keeps
            st["q"] = torch.empty((m, n), dtype=FP8[case["fmt"]][0], device="cuda")
            st["s"] = torch.empty((m, n // case["group"]), dtype=torch.float32, device="cuda")
            st["r"] = torch.empty((m, n), dtype=dt, device="cuda") if case["residual"] else None
        else:
            st["dy"] = (1e-2 * _normal(g, m, n)).to(dt)
            st["dr"] = (1e-2 * _normal(g, m, n)).to(dt) if case["residual"] else None
            for name in ("x", "res", "w"):
                if st[name] is not None:
                    st[name].requires_grad_(True)
        return st
    i, k = case["i"], case["k"]
    if kind == "gated_fp8":
        x = _outliers(g, _normal(g, m, k))
        kb = -(-k // 128)
        p = torch.zeros((m, kb * 128), device="cuda")
        p[:, :k] = x
        amax = p.view(m, kb, 128).abs().amax(2).clamp(min=CLAMP)
        st["a"] = (p.view(m, kb, 128) * (448.0 / amax)[:, :, None]).view(m, kb * 128)[:, :k] \
            .contiguous().to(torch.float8_e4m3fn)
        st["sa"] = amax / 448.0
        st["wg"], st["sg"] = _block_weight(g, i, k)
        st["wu"], st["su"] = _block_weight(g, i, k)
        if case["out"] == "fp8":
            st["q"] = torch.empty((m, i), dtype=torch.float8_e4m3fn, device="cuda")
            st["s"] = torch.empty((m, -(-i // 128)), dtype=torch.float32, device="cuda")
        else:
            st["h"] = torch.empty((m, i), dtype=DTYPES[case["out"]], device="cuda")
        return st
    dt = DTYPES[case["dtype"]]
    st["x"] = _outliers(g, _normal(g, m, k)).to(dt).requires_grad_(True)
    st["w"] = (_normal(g, 2 * i, k) * (1.5 / math.sqrt(k))).to(dt).requires_grad_(True)
    st["dh"] = (1e-2 * _normal(g, m, i) * torch.exp(0.5 * _normal(g, m, 1))).to(dt)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _OWN[kind](state)
    return _PLAIN[kind](state)


def _own_norm_fp8(st):
    c = st["case"]
    _lib().fp8q_rms_norm_quant(st["x"], st["w"], q=st["q"], scale_inv=st["s"], residual=st["res"],
                               residual_out=st["r"], eps=EPS, group=c["group"], fmt=c["fmt"])
    return {"q": st["q"], "s": st["s"], "r": st["r"]}


def _own_norm_train(st):
    if st["res"] is None:
        y = _lib().rms_norm(st["x"], st["w"], eps=EPS)
        dx, dw = torch.autograd.grad(y, (st["x"], st["w"]), st["dy"])
        return {"y": y, "dx": dx, "dw": dw}
    y, r = _lib().rms_norm(st["x"], st["w"], residual=st["res"], eps=EPS)
    dx, dres, dw = torch.autograd.grad((y, r), (st["x"], st["res"], st["w"]), (st["dy"], st["dr"]))
    return {"y": y, "r": r, "dx": dx, "dres": dres, "dw": dw}


def _own_gated_fp8(st):
    c = st["case"]
    if c["out"] == "fp8":
        _lib().fp8q_gated_mm_blockwise_quant(st["a"], st["sa"], st["wg"], st["sg"], st["wu"], st["su"], st["q"],
                                             st["s"], act=c["act"])
        return {"q": st["q"], "s": st["s"]}
    _lib().fp8q_gated_mm_blockwise(st["a"], st["sa"], st["wg"], st["sg"], st["wu"], st["su"], st["h"], act=c["act"])
    return {"h": st["h"]}


def _own_gated_train(st):
    h = _lib().gated_linear_fp8(st["x"], st["w"], act=st["case"]["act"])
    dx, dw = torch.autograd.grad(h, (st["x"], st["w"]), st["dh"])
    return {"h": h, "dx": dx, "dw": dw}


_OWN = {"norm_fp8": _own_norm_fp8, "norm_train": _own_norm_train, "gated_fp8": _own_gated_fp8,
        "gated_train": _own_gated_train}


# the plain forms: elementary operations in fp32, each output rounded once
def _groups(v, width):
    """[m, n] -> [m, ceil(n / width), width], zeros past n."""
    m, n = v.shape
    nb = -(-n // width)
    p = torch.zeros((m, nb * width), dtype=v.dtype, device=v.device)
    p[:, :n] = v
    return p.view(m, nb, width)


def _group_cast(v, width, fmt):
    t, top = FP8[fmt]
    m, n = v.shape
    p = _groups(v, width)
    amax = p.abs().amax(2).clamp(min=CLAMP)
    q = (p * (torch.full_like(amax, top) / amax)[:, :, None]).view(m, -1)[:, :n].contiguous().to(t)
    return q, amax / top


def _tensor_cast(v, fmt):
    t, top = FP8[fmt]
    amax = v.abs().amax()
    amax = torch.where(amax > 0, amax, torch.ones_like(amax))
    scale = torch.full_like(amax, top) / amax
    return (v * scale).to(t).float(), torch.ones_like(scale) / scale


def _sigma(g, act):
    """sigmoid(p(g)) and p'(g): act(g) = g * sigmoid(p(g))."""
    if act == "silu":
        return 1.0 / (1.0 + torch.exp(-g)), torch.ones_like(g)
    p = GELU * (g + 0.044715 * g * g * g)
    return 1.0 / (1.0 + torch.exp(-p)), GELU * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_norm(st):
    x, w, res = st["x"].detach(), st["w"].detach(), st["res"]
    r = x if res is None else (x.float() + res.detach().float()).to(x.dtype)
    f = r.float()
    rstd = 1.0 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)
    return r, f, rstd, f * rstd * w.float()


def _plain_norm_fp8(st):
    c = st["case"]
    r, _, _, y = _plain_norm(st)
    q, s = _group_cast(y, c["group"], c["fmt"])
    return {"q": q, "s": s, "r": r if st["res"] is not None else None}


def _plain_norm_train(st):
    r, f, rstd, y = _plain_norm(st)
    w, dy, dt = st["w"].detach(), st["dy"].float(), st["x"].dtype
    xhat = f * rstd
    dxhat = dy * w.float()
    dx = rstd * (dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True))
    out = {"y": y.to(dt), "dw": (dy * xhat).sum(0).to(w.dtype)}
    if st["res"] is None:
        out["dx"] = dx.to(dt)
    else:
        dx = (dx + st["dr"].float()).to(dt)
        out |= {"r": r, "dx": dx, "dres": dx}
    return out


def _block_spread(s, rows, k):
    """One value per 128 x 128 block for each element."""
    return s.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :k]


def _plain_gated_fp8(st):
    c = st["case"]
    i, k = c["i"], c["k"]
    a = st["a"].float() * st["sa"].repeat_interleave(128, 1)[:, :k]
    gate = a @ (st["wg"].float() * _block_spread(st["sg"], i, k)).t()
    up = a @ (st["wu"].float() * _block_spread(st["su"], i, k)).t()
    h = gate * _sigma(gate, c["act"])[0] * up
    if c["out"] == "fp8":
        q, s = _group_cast(h, 128, "e4m3")
        return {"q": q, "s": s}
    return {"h": h.to(DTYPES[c["out"]])}


def _plain_gated_train(st):
    c = st["case"]
    i, dt = c["i"], st["x"].dtype
    x8, sx = _tensor_cast(st["x"].detach().float(), "e4m3")
    w8, sw = _tensor_cast(st["w"].detach().float(), "e4m3")
    gu = (x8 @ w8.t()) * (sx * sw)
    h = gu[:, :i] * _sigma(gu[:, :i], c["act"])[0] * gu[:, i:]
    # gate and up are kept in the input's type for the backward pass
    kept = gu.to(dt).float()
    gate, up, dh = kept[:, :i], kept[:, i:], st["dh"].float()
    sig, dp = _sigma(gate, c["act"])
    d = torch.cat((dh * up * sig * (1.0 + gate * (1.0 - sig) * dp), dh * gate * sig), 1)
    d8, sd = _tensor_cast(d, "e5m2")
    return {"h": h.to(dt), "dx": ((d8 @ w8) * (sd * sw)).to(dt), "dw": ((d8.t() @ x8) * (sd * sx)).to(dt)}


_PLAIN = {"norm_fp8": _plain_norm_fp8, "norm_train": _plain_norm_train, "gated_fp8": _plain_gated_fp8,
          "gated_train": _plain_gated_train}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    m, kind = case["m"], case["kind"]
    if kind in ("norm_fp8", "norm_train"):
        n, e = case["n"], 4 if case["dtype"] == "f32" else 2
        ew = 4 if case.get("w32") else e
        res = case["residual"]
        if kind == "norm_fp8":
            # x (and the residual) in, the sum out, codes and scales out
            return {"bytes": m * n * (e + (2 * e if res else 0) + 1) + 4 * m * (n // case["group"]) + n * ew,
                    "flops": 8 * m * n}
        # forward: x (and the residual) in, y (and the sum) out; backward: dy and the normed rows
        # (and the sum's gradient) in, dx out, dw out
        return {"bytes": m * n * e * ((4 if res else 2) + (4 if res else 3)) + 3 * n * ew, "flops": 20 * m * n}
    i, k = case["i"], case["k"]
    kb, ib = -(-k // 128), -(-i // 128)
    if kind == "gated_fp8":
        out = m * i + 4 * m * ib if case["out"] == "fp8" else m * i * (4 if case["out"] == "f32" else 2)
        return {"bytes": m * k + 4 * m * kb + 2 * (i * k + 4 * ib * kb) + out, "flops": 4.0 * m * i * k}
    # forward: x, w in, h out; backward: dh in, dx, dw out; gate and up kept in between (out and in)
    return {"bytes": 2 * (2 * m * k + 2 * 2 * i * k + 2 * m * i + 2 * 2 * m * i), "flops": 12.0 * m * i * k}


# ---------------------------------------------------------------------------
# the definitions in binary64
# ---------------------------------------------------------------------------
def _round_fp8(v, fmt):
    """Nearest value of the format, ties to even, for |v| up to its maximum."""
    mant, lowest = (3, -6) if fmt == "e4m3" else (2, -14)
    e = (torch.frexp(v)[1].to(torch.int64) - 1).clamp(min=lowest) - mant
    step = ((e + 1023) << 52).view(torch.float64)                # 2^e from its bits
    return torch.round(v / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm_fp8": _exact_norm_fp8, "norm_train": _exact_norm_train, "gated_fp8": _exact_gated_fp8,
            "gated_train": _exact_gated_train}[case["kind"]](case, st)


def _f64(t):
    return t.detach().double()


def _exact_sum(st):
    x = _f64(st["x"])
    return x if st["res"] is None else (x + _f64(st["res"])).to(st["x"].dtype).double()


def _exact_norm_fp8(case, st):
    r = _exact_sum(st)
    y = r / (r.square().mean(1, keepdim=True) + EPS).sqrt() * _f64(st["w"])
    m, n = y.shape
    top = FP8[case["fmt"]][1]
    z = y.view(m, n // case["group"], case["group"])
    amax = z.abs().amax(2, keepdim=True).clamp(min=CLAMP)
    q = _round_fp8(z / amax * top, case["fmt"]).view(m, n)
    return {"q": q, "s": (amax / top).squeeze(2), "r": r if st["res"] is not None else None}


def _exact_norm_train(case, st):
    r, w, dy = _exact_sum(st), _f64(st["w"]), _f64(st["dy"])
    n = r.shape[1]
    v = r.square().sum(1, keepdim=True) / n + EPS
    t = dy * w
    # d/dr of r * v^(-1/2): the row's own term, and v's through every element
    dx = t / v.sqrt() - r * (t * r).sum(1, keepdim=True) / (n * v * v.sqrt())
    out = {"y": r * w / v.sqrt(), "dw": (dy * r / v.sqrt()).sum(0)}
    if st["res"] is None:
        out["dx"] = dx
    else:
        out["r"] = r
        out["dx"] = out["dres"] = dx + _f64(st["dr"])
    return out


def _act64(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1.0 - s)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 0.134145 * g * g)


def _exact_gated_fp8(case, st):
    i, k = case["i"], case["k"]
    cols = torch.arange(k, device="cuda") // 128
    rows = torch.arange(i, device="cuda") // 128
    a = _f64(st["a"]) * _f64(st["sa"])[:, cols]
    gate = a @ (_f64(st["wg"]) * _f64(st["sg"])[rows][:, cols]).t()
    up = a @ (_f64(st["wu"]) * _f64(st["su"])[rows][:, cols]).t()
    h = _act64(gate, case["act"])[0] * up
    if case["out"] != "fp8":
        return {"h": h}
    m, ib = h.shape[0], -(-i // 128)
    pad = torch.cat((h, h.new_zeros(m, ib * 128 - i)), 1).view(m, ib, 128)
    amax = pad.abs().amax(2).clamp(min=CLAMP)
    q = _round_fp8(h / amax[:, rows] * 448.0, "e4m3")
    return {"q": q, "s": amax / 448.0}


def _cast64(v, fmt):
    """Per-tensor cast: the values the codes stand for.  The cast's scale is an fp32 number, and each
    product with it is rounded to fp32, by definition: an amax that FMAX shares a factor with puts
    many bf16 values exactly between two codes, and this rounding says which they take."""
    amax = v.abs().max()
    if amax.item() == 0:
        return v
    scale = (FP8[fmt][1] / amax).float().double()
    return _round_fp8((v * scale).float().double(), fmt) / scale


def _exact_gated_train(case, st):
    i, dt = case["i"], st["x"].dtype
    x, w = _cast64(_f64(st["x"]), "e4m3"), _cast64(_f64(st["w"]), "e4m3")
    gu = x @ w.t()
    h = _act64(gu[:, :i], case["act"])[0] * gu[:, i:]
    kept = gu.to(dt).double()
    a, da = _act64(kept[:, :i], case["act"])
    dh = _f64(st["dh"])
    d = _cast64(torch.cat((dh * kept[:, i:] * da, dh * a), 1), "e5m2")
    return {"h": h, "dx": d @ w, "dw": d.t() @ x}
