"""What the products and layer norms around the library's scans are measured on.

Four operators, the two of a forward pass and their gradients:

* ``linear``: y = act(x w^T + bias) + residual, of bfloat16, float32, or e4m3 codes with a scale a row,
  for prompts and for a few tokens; the value before the activation is kept where a gradient follows;
* ``linear_back``: the gradients of x, w and bias behind the activation;
* ``norm``: layer norm of x + residual, with the rows' mean and reciprocal deviation;
* ``norm_back``: the gradients of its input, weight and bias, joined by the residual's own.

``run`` computes a case in its plain form (32-bit torch operations, rounded once at the end) while
``own`` is false, and through the library's entry points while it is true.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def listed():
    """The measured cases: real work over the range of the operators."""
    return [
        # the input projection of a state space layer (64 heads of 64, one group of 128 states, width 2048)
        # for one decoded token: latency, every weight is read once
        dict(name="linear_token", op="linear", M=1, N=8512, K=2048, dtype="bf16", out="bf16", act="none", bias=False,
             residual=False, pre=False, strided=False),
        # its output projection for a decoding step of 128 sequences, joining a residual stream in 32 bits
        dict(name="linear_tokens", op="linear", M=128, N=2048, K=4096, dtype="bf16", out="f32", act="none", bias=False,
             residual=True, pre=False, strided=False),
        # the input projection of a batch of long prompts
        dict(name="linear_prompts", op="linear", M=32768, N=8512, K=2048, dtype="bf16", out="bf16", act="none",
             bias=False, residual=False, pre=False, strided=False),
        # the output projection of e4m3 codes, one scale a token and one a weight row
        dict(name="linear_prompts_e4m3", op="linear", M=16384, N=2048, K=4096, dtype="e4m3", out="bf16", act="none",
             bias=False, residual=True, pre=False, strided=False),
        # the first product of a feed-forward block in training: bias and gelu, its argument kept
        dict(name="linear_gelu", op="linear", M=8192, N=8192, K=2048, dtype="bf16", out="bf16", act="gelu", bias=True,
             residual=False, pre=True, strided=True),
        # odd sizes in 32 bits, everything in the epilogue
        dict(name="linear_f32", op="linear", M=1001, N=777, K=1161, dtype="f32", out="f32", act="silu", bias=True,
             residual=True, pre=False, strided=True),
        # the gradients behind gelu of that feed-forward product
        dict(name="linear_back_gelu", op="linear_back", M=8192, N=8192, K=2048, dtype="bf16", act="gelu", bias=True,
             strided=False),
        # gradients of odd sizes in 32 bits
        dict(name="linear_back_f32", op="linear_back", M=513, N=1001, K=520, dtype="f32", act="silu", bias=True,
             strided=True),
        # the norm over the tokens of a long prompt with the residual stream's addition
        dict(name="norm_prompt", op="norm", M=16384, D=4096, dtype="bf16", residual="bf16", bias=True),
        # a handful of tokens, the residual stream in 32 bits
        dict(name="norm_tokens", op="norm", M=24, D=5120, dtype="bf16", residual="f32", bias=True),
        # the norm's gradients in training, the residual stream's own gradient added
        dict(name="norm_back_bf16", op="norm_back", M=16384, D=4096, dtype="bf16", stream="bf16", joined=True, bias=True),
        # an odd width in 32 bits, no residual
        dict(name="norm_back_f32", op="norm_back", M=4099, D=1001, dtype="f32", stream="f32", joined=False, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges of listed(), costing no more than its largest."""
    op = rng.choice(["linear", "linear", "linear_back", "norm", "norm_back"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    flip = lambda: rng.choice([True, False])   # noqa: E731
    if op in ("norm", "norm_back"):
        D = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024)])
        M = min(_log(rng, 1, 16384), 2 ** 26 // D)
        if op == "norm":
            residual = rng.choice(["", dtype, "f32"])
            M = min(M, 2 ** (25 if "f32" in (dtype, residual) else 26) // D)
            return dict(op=op, M=M, D=D, dtype=dtype, residual=residual, bias=flip())
        stream = rng.choice([dtype, "f32"])
        M = min(M, 2 ** (26 if stream == "bf16" else 25) // D)
        return dict(op=op, M=M, D=D, dtype=dtype, stream=stream, joined=flip(), bias=flip())
    size = lambda lo: rng.choice([_log(rng, lo, 8192), 8 * _log(rng, lo // 8, 1024)])   # noqa: E731
    N, K = size(32), size(32)
    act = rng.choice(["none", "silu", "gelu"])
    most = 2 ** 36 if dtype == "f32" else 2 ** 38   # products of one pass
    rows = 2 ** (25 if dtype == "f32" else 26) // max(N, K)
    if op == "linear_back":
        M = max(1, min(_log(rng, 1, 32768), most // (2 * N * K), rows))
        return dict(op=op, M=M, N=N, K=K, dtype=dtype, act=act, bias=flip(), strided=flip())
    out = dtype
    if dtype == "bf16":
        dtype, out = rng.choice(["bf16", "bf16", "e4m3"]), rng.choice(["bf16", "bf16", "f32"])
    M = _log(rng, 1, 128) if flip() else _log(rng, 128, 32768)
    M = max(1, min(M, most // (N * K), rows if out == "bf16" else rows // 2))
    return dict(op=op, M=M, N=N, K=K, dtype=dtype, out=out, act=act, bias=flip(), residual=flip(), pre=flip(),
                strided=flip())


# ---------------------------------------------------------------------------------------------------------------------
# inputs


def _rows(rand, rows, width, strided):
    """[rows, width], as a slice of wider rows where `strided`."""
    return rand(rows, width + 24)[:, 8:8 + width] if strided else rand(rows, width)


def _codes(v):
    """e4m3 codes and scales of the rows of v, as an 8-bit norm or a quantised weight has them."""
    scale = v.abs().amax(1) / 448.0
    return (v / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    """A block's tensors in hand before the call, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    dt = _TYPES[case["dtype"]]
    st = dict(case=case, op=case["op"])
    if case["op"] in ("norm", "norm_back"):
        M, D = case["M"], case["D"]
        st["w"] = 1 + 0.2 * rand(D)
        st["b"] = 0.1 * rand(D) if case["bias"] else None
        if case["op"] == "norm":
            st["x"] = rand(M, D).to(dt)
            st["residual"] = (0.5 + 3 * rand(M, D)).to(_TYPES[case["residual"]]) if case["residual"] else None
            return st
        sdt = _TYPES[case["stream"]]
        st["x"] = (0.5 + 3 * rand(M, D)).to(sdt)
        st["dy"] = rand(M, D).to(dt)
        st["dres"] = rand(M, D).to(sdt) if case["joined"] else None
        x = st["x"].double() if M * D <= 2 ** 24 else st["x"].float()
        mean = x.mean(1, keepdim=True)
        st["stats"] = torch.cat([mean, torch.rsqrt((x - mean).square().mean(1, keepdim=True) + 1e-5)], 1).float()
        return st
    M, N, K = case["M"], case["N"], case["K"]
    st["x"], st["w"] = _rows(rand, M, K, case["strided"]), rand(N, K) / math.sqrt(K)
    st["bias"] = 0.3 * rand(N) if case["bias"] else None
    st["x_scale"] = st["w_scale"] = None
    if case["dtype"] == "e4m3":
        st["x"], st["x_scale"] = _codes(st["x"])
        st["w"], st["w_scale"] = _codes(st["w"])
    else:
        st["x"], st["w"] = st["x"].to(dt), st["w"].to(dt)
        if case["strided"]:
            st["x"] = _rows(lambda *s: torch.zeros(*s, dtype=dt, device="cuda"), M, K, True).copy_(st["x"])
    if case["op"] == "linear":
        odt = _TYPES[case["out"]]
        st["residual"] = rand(M, N).to(odt) if case["residual"] else None
        st["pre"] = torch.empty(M, N, dtype=odt, device="cuda") if case["pre"] else None
        return st
    st["dy"] = rand(M, N).to(dt)
    st["pre"] = None
    if case["act"] != "none":
        st["pre"] = st["x"] @ st["w"].t() if st["bias"] is None else (st["x"] @ st["w"].t() + st["bias"]).to(dt)
    return st


# ---------------------------------------------------------------------------------------------------------------------
# plain forms


def _plain_act(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(v * -math.sqrt(0.5))
    return v


def _plain_linear(st):
    case = st["case"]
    v = st["x"].float() @ st["w"].float().t()
    if st["x_scale"] is not None:
        v = v * st["x_scale"][:, None] * st["w_scale"]
    if st["bias"] is not None:
        v = v + st["bias"]
    got = {}
    if st["pre"] is not None:
        st["pre"].copy_(v)
        got["pre"] = st["pre"]
    v = _plain_act(v, case["act"])
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return {"y": v.to(_TYPES[case["out"]]), **got}


def _plain_linear_back(st):
    g, act, dt = st["dy"].float(), st["case"]["act"], st["dy"].dtype
    if act != "none":
        v = st["pre"].float()
        if act == "silu":
            s = torch.sigmoid(v)
            g = g * s * (1 + v * (1 - s))
        else:
            cdf = 0.5 * torch.special.erfc(v * -math.sqrt(0.5))
            g = g * (cdf + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi))
    got = {"dx": (g @ st["w"].float()).to(dt), "dw": (g.t() @ st["x"].float()).to(dt)}
    if st["bias"] is not None:
        got["db"] = g.sum(0, dtype=torch.float64).float()
    return got


def _plain_norm(st):
    r = st["x"].float()
    got = {}
    if st["residual"] is not None:
        r = r + st["residual"].float()
        st["residual"].copy_(r)
        got["residual"] = st["residual"]
    mean = r.mean(1, keepdim=True)
    c = r - mean
    rstd = torch.rsqrt(c.square().mean(1, keepdim=True) + 1e-5)
    y = c * rstd * st["w"]
    if st["b"] is not None:
        y = y + st["b"]
    return {"y": y.to(st["x"].dtype), "stats": torch.cat([mean, rstd], 1), **got}


def _plain_norm_back(st):
    dy, x = st["dy"].float(), st["x"].float()
    mean, rstd = st["stats"][:, :1], st["stats"][:, 1:]
    h = (x - mean) * rstd
    a = dy * st["w"]
    dx = rstd * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    got = {"dx": dx.to(st["x"].dtype), "dw": (dy * h).sum(0, dtype=torch.float64).float()}
    if st["b"] is not None:
        got["db"] = dy.sum(0, dtype=torch.float64).float()
    return got


# ---------------------------------------------------------------------------------------------------------------------
# the library's calls


def _own_linear(st):
    import sherman_morrison_inverse_gb300 as vla
    case = st["case"]
    y = vla.linear(st["x"], st["w"], st["bias"], st["residual"], act=case["act"], pre=st["pre"],
                   x_scale=st["x_scale"], w_scale=st["w_scale"], dtype=_TYPES[case["out"]])
    return {"y": y} if st["pre"] is None else {"y": y, "pre": st["pre"]}


def _own_linear_back(st):
    import sherman_morrison_inverse_gb300 as vla
    bias = st["bias"] is not None
    dx, dw, db = vla.linear_backward(st["dy"], st["x"], st["w"], st["pre"], act=st["case"]["act"], bias=bias)
    return {"dx": dx, "dw": dw, "db": db} if bias else {"dx": dx, "dw": dw}


def _own_norm(st):
    import sherman_morrison_inverse_gb300 as vla
    got = {} if st["residual"] is None else {"residual": st["residual"]}
    y, stats = vla.layer_norm(st["x"], st["w"], st["b"], st["residual"], eps=1e-5, stats=True)
    return {"y": y, "stats": stats, **got}


def _own_norm_back(st):
    import sherman_morrison_inverse_gb300 as vla
    bias = st["b"] is not None
    dx, dw, db = vla.layer_norm_backward(st["dy"], st["x"], st["w"], st["stats"], st["dres"], bias=bias)
    return {"dx": dx, "dw": dw, "db": db} if bias else {"dx": dx, "dw": dw}


def run(state):
    """One pass through the case's operator; residuals are updated in place."""
    if own:
        form = {"linear": _own_linear, "linear_back": _own_linear_back, "norm": _own_norm, "norm_back": _own_norm_back}
    else:
        form = {"linear": _plain_linear, "linear_back": _plain_linear_back, "norm": _plain_norm,
                "norm_back": _plain_norm_back}
    return form[state["op"]](state)


def work(case):
    """Bytes and operations that one pass cannot do without (32-bit biases and norm weights)."""
    item = {"bf16": 2, "f32": 4, "e4m3": 1}
    e = item[case["dtype"]]
    if case["op"] in ("norm", "norm_back"):
        M, D = case["M"], case["D"]
        if case["op"] == "norm":
            res = 2 * item[case["residual"]] if case["residual"] else 0
            return {"bytes": M * D * (2 * e + res) + 8 * M + 4 * D * (2 if case["bias"] else 1), "flops": 8.0 * M * D}
        s = item[case["stream"]]
        return {"bytes": M * D * (e + s * (3 if case["joined"] else 2)) + 8 * M + 4 * D * (3 if case["bias"] else 2),
                "flops": 14.0 * M * D}
    M, N, K = case["M"], case["N"], case["K"]
    bias = 4 * N if case["bias"] else 0
    if case["op"] == "linear":
        o = item[case["out"]]
        size = e * (M * K + N * K) + o * M * N * (1 + case["residual"] + case["pre"]) + bias
        return {"bytes": size + (4 * (M + N) if case["dtype"] == "e4m3" else 0), "flops": 2.0 * M * N * K}
    return {"bytes": e * (M * N * (1 if case["act"] == "none" else 2) + 2 * M * K + 2 * N * K) + bias,
            "flops": 4.0 * M * N * K}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return {"linear": _exact_linear, "linear_back": _exact_linear_back, "norm": _exact_norm,
            "norm_back": _exact_norm_back}[case["op"]](st)


def _exact_linear(st):
    act = st["case"]["act"]
    x, w = st["x"].double(), st["w"].double()
    if st["x_scale"] is not None:
        x, w = x * st["x_scale"].double()[:, None], w * st["w_scale"].double()[:, None]
    pre = torch.einsum("mk,nk->mn", x, w)
    del x, w
    if st["bias"] is not None:
        pre += st["bias"].double()
    y = pre if act == "none" else torch.empty_like(pre)
    for at in range(0, len(pre), 4096):   # a slice at a time: 64-bit copies of a large product are gigabytes
        v = pre[at:at + 4096]
        if act == "silu":
            y[at:at + 4096] = v / (1 + torch.exp(-v))
        elif act == "gelu":
            y[at:at + 4096] = v * torch.special.erfc(-v / math.sqrt(2)) / 2
    if st["pre"] is None:
        return {"y": y if st["residual"] is None else y.add_(st["residual"])}
    return {"y": y if st["residual"] is None else y + st["residual"], "pre": pre}


def _exact_linear_back(st):
    act, g = st["case"]["act"], st["dy"].double()
    if act != "none":
        v = st["pre"].double()
        if act == "silu":
            e = torch.exp(-v)
            g *= 1 / (1 + e) + v * e / (1 + e) ** 2
        else:
            g *= torch.special.erfc(-v / math.sqrt(2)) / 2 + v * torch.exp(-v ** 2 / 2) / math.sqrt(2 * math.pi)
    got = {"dx": torch.einsum("mn,nk->mk", g, st["w"].double()), "dw": torch.einsum("mn,mk->nk", g, st["x"].double())}
    if st["bias"] is not None:
        got["db"] = torch.einsum("mn->n", g)
    return got


def _exact_norm(st):
    r = st["x"].double()
    got = {}
    if st["residual"] is not None:
        r = r + st["residual"].double()
        got["residual"] = r
    D = r.shape[1]
    mean = r.sum(1) / D
    rstd = 1 / torch.sqrt((r - mean[:, None]).pow(2).sum(1) / D + 1e-5)
    y = (r - mean[:, None]) * (rstd[:, None] * st["w"].double())
    if st["b"] is not None:
        y += st["b"].double()
    return {"y": y, "stats": torch.stack([mean, rstd], 1), **got}


def _exact_norm_back(st):
    """The Jacobian of each row applied to dy w: rstd (I - 1 1^T / D - h h^T / D)."""
    D = st["x"].shape[1]
    mean, rstd = st["stats"].double().unbind(1)
    h = (st["x"].double() - mean[:, None]) * rstd[:, None]
    dy = st["dy"].double()
    a = dy * st["w"].double()
    along = torch.einsum("md,md->m", a, h) / D
    dx = (a - (a.sum(1) / D)[:, None] - along[:, None] * h) * rstd[:, None]
    if st["dres"] is not None:
        dx += st["dres"]
    got = {"dx": dx, "dw": torch.einsum("md,md->d", dy, h)}
    if st["b"] is not None:
        got["db"] = torch.einsum("md->d", dy)
    return got
