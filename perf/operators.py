"""What the operators of a state space layer are measured on.

Three operators, each in its form for prompts and for single tokens where that differs:

* ``conv``: the short causal convolution of every channel with its own K taps, with an optional
  SiLU, over dense or packed prompts, and for one token a sequence (``T == 1``);
* ``scan``: the selective state space scan with one decay a head,
  h_t = exp(A dt_t) h_{t-1} + dt_t x_t B_t^T,  y_t = (h_t C_t + D x_t) * silu(z_t),
  over dense or packed prompts, and for one token a sequence;
* ``norm``: the root-mean-square norm of x + residual, its result in 8 bits with scales or in the
  layer's own type.

``run`` computes a case in its plain form (32-bit torch operations, rounded once at the end) while
``own`` is false, and through the library's entry points while it is true.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    """The measured cases: real work over the range of the operators."""
    return [
        # a batch of long prompts through the convolution of a layer with 64 heads of 64 and one
        # group of 128 states: x | B | C is a slice of the input projection's rows
        dict(name="conv_prompts", op="conv", S=8, T=4096, C=4352, K=4, dtype="bf16", lens="", silu=True, strided=True),
        # prompts of many lengths packed one after another, an odd channel count, three taps, no
        # activation, in 32 bits
        dict(name="conv_packed_f32", op="conv", S=9, T=0, C=1161, K=3, dtype="f32",
             lens="1,2,700,33,1024,129,5,2048,311", silu=False, strided=False),
        # one decoding step of 192 sequences whose states lie in a pool
        dict(name="conv_tokens", op="conv", S=192, T=1, C=4352, K=4, dtype="bf16", lens="", silu=True, strided=True),
        # a batch of prompts through the scan: 64 heads of 64, 128 states, B and C shared by all heads
        dict(name="scan_prompts", op="scan", S=8, T=4096, H=64, P=64, G=1, N=128, dtype="bf16", lens="", gate=False,
             strided=True),
        # one long prompt, 16 heads: few rows, a long axis; gated
        dict(name="scan_long", op="scan", S=1, T=16384, H=16, P=64, G=1, N=128, dtype="bf16", lens="", gate=True,
             strided=True),
        # packed prompts of uneven lengths that continue from their states; 8 groups, 64 states, heads of 128
        dict(name="scan_packed", op="scan", S=9, T=0, H=16, P=128, G=8, N=64, dtype="bf16",
             lens="1,129,512,37,1000,2047,64,300,96", gate=True, strided=False),
        # 32-bit input and output (the precise path) at the size of a small model
        dict(name="scan_f32", op="scan", S=4, T=513, H=8, P=64, G=1, N=64, dtype="f32", lens="", gate=False,
             strided=False),
        # one decoding step of 128 sequences: every state is read and written once
        dict(name="scan_tokens", op="scan", S=128, T=1, H=64, P=64, G=1, N=128, dtype="bf16", lens="", gate=True,
             strided=True),
        # one decoding step of a single sequence: latency
        dict(name="scan_token", op="scan", S=1, T=1, H=64, P=64, G=1, N=128, dtype="bf16", lens="", gate=True,
             strided=True),
        # the norm before an 8-bit projection over the tokens of a long prompt, one scale a token
        dict(name="norm_e4m3", op="norm", M=16384, D=4096, dtype="bf16", out="e4m3", group=0, residual="bf16"),
        # the same for a handful of decoded tokens, 8-bit integers with a scale for every 128 values,
        # the residual stream in 32 bits
        dict(name="norm_int8_tokens", op="norm", M=24, D=5120, dtype="bf16", out="int8", group=128, residual="f32"),
        # an odd width in 32 bits, no residual, no quantisation
        dict(name="norm_f32", op="norm", M=4099, D=1001, dtype="f32", out="io", group=0, residual=""),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges of listed(), costing no more than its largest."""
    op = rng.choice(["conv", "scan", "scan", "norm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "norm":
        out = rng.choice(["e4m3", "int8", "io"])
        D = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024)])
        return dict(op=op, M=min(_log(rng, 1, 16384), 2 ** 26 // D), D=D, dtype=dtype, out=out,
                    group=rng.choice([0, 128]) if out != "io" else 0, residual=rng.choice(["", dtype, "f32"]))
    form = rng.choice(["dense", "packed", "token"])
    S = _log(rng, 1, 128) if form == "token" else _log(rng, 1, 12)
    T = 1 if form == "token" else _log(rng, 2, 8192)
    lens = ",".join(str(_log(rng, 1, max(2, T))) for _ in range(S)) if form == "packed" else ""
    tokens = sum(int(v) for v in lens.split(",")) if lens else S * T
    if lens:
        T = 0
    if op == "conv":
        C = rng.choice([_log(rng, 16, 8192), 8 * _log(rng, 8, 1024)])
        C = max(16, min(C, 2 ** 26 // tokens))
        return dict(op=op, S=S, T=T, C=C, K=rng.choice([2, 3, 4, 4]), dtype=dtype, lens=lens,
                    silu=rng.choice([True, False]), strided=rng.choice([True, False]))
    G = rng.choice([1, 1, 2, 4])
    H = G * _log(rng, 1, 64 // G)
    P, N = rng.choice([64, 64, 128, 32, 40]), rng.choice([128, 128, 64, 16, 96, 20])
    most = 2 ** 16 if dtype == "f32" else 2 ** 20
    H = max(G, min(H, most * 64 // (tokens * P)) // G * G)
    if tokens * H * P > most * 256:   # one long sequence of a few heads
        G, H, P = 1, 1, 32
    return dict(op=op, S=S, T=T, H=H, P=P, G=G, N=N, dtype=dtype, lens=lens, gate=rng.choice([True, False]),
                strided=rng.choice([True, False]))


# ---------------------------------------------------------------------------------------------------------------------
# inputs


def _lens(case):
    return [int(v) for v in case["lens"].split(",")] if case["lens"] else [case["T"]] * case["S"]


def _offsets(case):
    off = [0]
    for n in _lens(case):
        off.append(off[-1] + n)
    return off


def _view(rand, lead, width, before, after, dtype):
    """[..., width] as a slice of rows that hold `before` and `after` more values."""
    return rand(*lead, before + width + after).to(dtype)[..., before:before + width]


def prepare(case, seed):
    """A layer's tensors in hand before the call, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=gen, device="cuda")     # noqa: E731
    dt = _TYPES[case["dtype"]]
    st = dict(case=case, op=case["op"])
    if case["op"] == "norm":
        M, D = case["M"], case["D"]
        st["x"] = rand(M, D).to(dt)
        st["w"] = 1 + 0.2 * rand(D)
        st["residual"] = (3 * rand(M, D)).to(_TYPES[case["residual"]]) if case["residual"] else None
        return st
    S = case["S"]
    off = _offsets(case)
    packed = bool(case["lens"])
    lead = (off[-1],) if packed else (S,) if case["T"] == 1 else (S, case["T"])
    st["packed"], st["max_len"] = packed, max(_lens(case))
    st["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda") if packed else None
    slots = torch.randperm(S + 1, generator=gen, device="cuda")[:S].to(torch.int32)   # one spare slot in the pool
    st["slots"] = slots
    if case["op"] == "conv":
        C, K = case["C"], case["K"]
        more = (C // 2 + 8, C % 8 + 8) if case["strided"] else (0, 0)
        st["x"] = _view(rand, lead, C, *more, dt)
        st["w"] = rand(C, K) / math.sqrt(K)
        st["bias"] = 0.1 * rand(C)
        st["state"] = rand(S + 1, K - 1, C).to(dt)
        return st
    H, P, G, N = (case[k] for k in "HPGN")
    width = H * P + 2 * G * N
    # x | B | C as the convolution leaves them; z and dt are slices of the input projection's rows
    xbc = torch.nn.functional.silu(rand(*lead, width)).to(dt)
    if not case["strided"]:
        x, B, C = (t.contiguous() for t in (xbc[..., :H * P], xbc[..., H * P:H * P + G * N], xbc[..., H * P + G * N:]))
    else:
        x, B, C = xbc[..., :H * P], xbc[..., H * P:H * P + G * N], xbc[..., H * P + G * N:]
    st["x"], st["B"], st["C"] = x.unflatten(-1, (H, P)), B.unflatten(-1, (G, N)), C.unflatten(-1, (G, N))
    st["z"] = None
    if case["gate"]:
        st["z"] = _view(rand, lead, H * P, 0, H if case["strided"] else 0, dt).unflatten(-1, (H, P))
    st["dt"] = _view(rand, lead, H, 16 if case["strided"] else 0, 0, dt)
    step = torch.exp(uni(H) * math.log(100.0) + math.log(1e-3))     # time steps of 0.001 to 0.1
    st["dt_bias"] = step + torch.log(-torch.expm1(-step))           # softplus of it is `step`
    st["A"] = -(1 + 15 * uni(H))
    st["D"] = 1 + 0.1 * rand(H)
    st["state"] = rand(S + 1, H, P, N)
    return st


# ---------------------------------------------------------------------------------------------------------------------
# plain forms


def _padded(st, t):
    """Packed rows [tokens, ...] -> [S, max_len, ...] with the sequences' own rows, and which they are."""
    off = st["offsets"].long()
    at = off[:-1, None] + torch.arange(st["max_len"], device=t.device)
    inside = at < off[1:, None]
    return t[torch.where(inside, at, 0)], inside


def _sequences(st, *ts):
    """The tensors as [S, T, ...] in 32 bits, and the mask of real tokens (None: all)."""
    if st["packed"]:
        got = [_padded(st, t) for t in ts]
        return [g[0].float() for g in got], got[0][1]
    if st["case"]["T"] == 1:
        return [t.unsqueeze(1).float() for t in ts], None
    return [t.float() for t in ts], None


def _back(st, y, inside):
    """[S, T, ...] -> the layout of the inputs."""
    if inside is not None:
        return y[inside]
    return y[:, 0] if st["case"]["T"] == 1 else y


def _plain_conv(st):
    x, w, K = st["x"], st["w"], st["w"].shape[1]
    slots = st["slots"].long()
    (xs,), inside = _sequences(st, x)
    if inside is not None:
        xs = xs * inside[..., None]
    whole = torch.cat([st["state"][slots].float(), xs], 1)                # [S, K - 1 + T, C]
    y = (whole.unfold(1, K, 1) * w).sum(-1) + st["bias"]
    if st["case"]["silu"]:
        y = y * torch.sigmoid(y)
    n = torch.full((len(slots),), xs.shape[1], device=x.device) if inside is None else inside.sum(1)
    last = n[:, None] + torch.arange(K - 1, device=x.device)              # the K - 1 inputs before the next token
    st["state"][slots] = whole.gather(1, last[..., None].expand(-1, -1, x.shape[-1])).to(x.dtype)
    return {"y": _back(st, y, inside).to(x.dtype), "state": st["state"]}


def _segsum(a):
    """[..., L] -> [..., L, L]: the sum of a over (j, i], -inf above the diagonal."""
    L = a.shape[-1]
    ones = torch.ones(L, L, dtype=torch.bool, device=a.device)
    s = a[..., :, None].expand(*a.shape, L).masked_fill(~ones.tril(-1), 0).cumsum(-2)
    return s.masked_fill(~ones.tril(), -math.inf)


def _plain_scan(st):
    x = st["x"]
    H, G, slots = x.shape[-2], st["B"].shape[-2], st["slots"].long()
    (xs, dt, B, C), inside = _sequences(st, x, st["dt"], st["B"], st["C"])
    S, T, P, N = *xs.shape[:2], xs.shape[-1], B.shape[-1]
    dt = torch.nn.functional.softplus(dt + st["dt_bias"])
    if inside is not None:
        dt = dt * inside[..., None]
    L = min(64, T)
    n = -(-T // L)
    pad = lambda t: torch.cat([t, t.new_zeros(S, n * L - T, *t.shape[2:])], 1).unflatten(1, (n, L))   # noqa: E731
    xc, dc, Bc, Cc = pad(xs), pad(dt).transpose(2, 3), pad(B).transpose(2, 3), pad(C).transpose(2, 3)
    xc = xc.transpose(2, 3)                                               # [S, n, H, L, P], dc [S, n, H, L]
    a = dc * st["A"][:, None]
    seg = torch.exp(_segsum(a))                                           # [S, n, H, L, L]
    CB = (Cc @ Bc.transpose(-1, -2)).repeat_interleave(H // G, 2)
    y = (CB * seg * dc[..., None, :]) @ xc
    tail = seg[..., -1, :] * dc                                           # what is left of each token at the chunk's end
    new = (xc * tail[..., None]).transpose(-1, -2) @ Bc.repeat_interleave(H // G, 2)
    new = torch.cat([st["state"][slots].unsqueeze(1), new], 1)            # [S, 1 + n, H, P, N]
    run = torch.exp(_segsum(torch.cat([a.new_zeros(S, 1, H), a.sum(-1)], 1).transpose(1, 2)))
    h = (run @ new.transpose(1, 2).flatten(-2)).unflatten(-1, (P, N)).transpose(1, 2)
    inter = (Cc.repeat_interleave(H // G, 2) @ h[:, :-1].transpose(-1, -2)) * torch.exp(a.cumsum(-1))[..., None]
    y = (y + inter).transpose(2, 3).flatten(1, 2)[:, :T] + xs * st["D"][:, None]
    if st["z"] is not None:
        z = _sequences(st, st["z"])[0][0]
        y = y * z * torch.sigmoid(z)
    st["state"][slots] = h[:, -1]
    return {"y": _back(st, y, inside).to(x.dtype), "state": st["state"]}


def _groups(v, group):
    """[M, D] -> [M, groups, width], the last group filled up with zeros."""
    width = group or v.shape[1]
    n = -(-v.shape[1] // width)
    return torch.cat([v, v.new_zeros(v.shape[0], n * width - v.shape[1])], 1).unflatten(1, (n, width))


def _plain_norm(st):
    case, x = st["case"], st["x"]
    r = x.float()
    got = {}
    if st["residual"] is not None:
        r = r + st["residual"].float()
        st["residual"].copy_(r)
        got["residual"] = st["residual"]
    v = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + 1e-6) * st["w"]
    if case["out"] == "io":
        return {"y": v.to(x.dtype), **got}
    vg = _groups(v, case["group"])
    scale = vg.abs().amax(-1) / (448.0 if case["out"] == "e4m3" else 127.0)
    scale = torch.where(scale < 2.0 ** -126, torch.ones_like(scale), scale)
    q = vg * (1.0 / scale)[..., None]
    got["scale"] = scale if case["group"] else scale[:, 0]
    if case["out"] == "e4m3":
        return {"y": q.clamp(-448, 448).flatten(1)[:, :x.shape[1]].to(torch.float8_e4m3fn), **got}
    y = (q.round().clamp(-127, 127) * scale[..., None]).flatten(1)[:, :x.shape[1]]
    return {"y": y.to(torch.bfloat16), **got}


# ---------------------------------------------------------------------------------------------------------------------
# the library's calls


def _own_conv(st):
    import sherman_morrison_inverse_gb300 as vla
    if st["case"]["T"] == 1:
        y = vla.short_conv_step(st["x"], st["w"], st["bias"], st["state"], silu=st["case"]["silu"], slots=st["slots"])
    else:
        y = vla.short_conv(st["x"], st["w"], st["bias"], st["state"], silu=st["case"]["silu"], slots=st["slots"],
                           offsets=st["offsets"], max_len=st["max_len"])
    return {"y": y, "state": st["state"]}


def _own_scan(st):
    import sherman_morrison_inverse_gb300 as vla
    args = (st["x"], st["dt"], st["A"], st["B"], st["C"], st["state"])
    more = dict(D=st["D"], z=st["z"], dt_bias=st["dt_bias"], softplus=True, slots=st["slots"])
    if st["case"]["T"] == 1:
        y = vla.ssm_step(*args, **more)
    else:
        y = vla.ssm_scan(*args, **more, offsets=st["offsets"], max_len=st["max_len"])
    return {"y": y, "state": st["state"]}


def _own_norm(st):
    import sherman_morrison_inverse_gb300 as vla
    case = st["case"]
    got = {} if st["residual"] is None else {"residual": st["residual"]}
    if case["out"] == "io":
        return {"y": vla.rms_norm(st["x"], st["w"], st["residual"], eps=1e-6), **got}
    q, scale = vla.rms_norm(st["x"], st["w"], st["residual"], eps=1e-6, out=case["out"], group=case["group"])
    return {"y": q if case["out"] == "e4m3" else _stands_for(q, scale), "scale": scale, **got}


def _stands_for(q, scale):
    """The values that 8-bit integers stand for, in 16 bits."""
    y = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if scale.dim() == 1:
        return torch.mul(q, scale[:, None], out=y)
    if q.shape[1] % 128:
        return torch.mul(q, scale.repeat_interleave(128, 1)[:, :q.shape[1]], out=y)
    torch.mul(q.unflatten(1, (-1, 128)), scale[..., None], out=y.unflatten(1, (-1, 128)))
    return y


def run(state):
    """One pass through the case's operator; states and residuals are updated in place."""
    if own:
        return {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm}[state["op"]](state)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[state["op"]](state)


def work(case):
    """Bytes and operations that one pass cannot do without (32-bit weights, states read and written once)."""
    item = {"bf16": 2, "f32": 4}
    e = item[case["dtype"]]
    if case["op"] == "norm":
        M, D = case["M"], case["D"]
        out = e if case["out"] == "io" else 1
        scales = 0 if case["out"] == "io" else M * (-(-D // 128) if case["group"] else 1) * 4
        res = 2 * item[case["residual"]] if case["residual"] else 0
        return {"bytes": M * D * (e + out + res) + scales + 4 * D, "flops": 6.0 * M * D}
    lens = _lens(case)
    tokens, S = sum(lens), case["S"]
    if case["op"] == "conv":
        C, K = case["C"], case["K"]
        return {"bytes": 2 * e * tokens * C + 2 * e * S * (K - 1) * C + 4 * C * (K + 1),
                "flops": (2.0 * K + 4) * tokens * C}
    H, P, G, N = (case[k] for k in "HPGN")
    wide = tokens * H * P
    size = e * (wide * (3 if case["gate"] else 2) + tokens * (2 * G * N + H)) + 8 * S * H * P * N
    # the recurrence itself: the state's update and its product with C, 5 operations a state element
    return {"bytes": size, "flops": 5.0 * wide * N}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions, token by token in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](st)


def _starts(st):
    case = st["case"]
    off = _offsets(case)
    flat = lambda t: t if st["packed"] or case["T"] == 1 else t.flatten(0, 1)   # noqa: E731
    start = torch.tensor(off[:-1], device="cuda")
    size = torch.tensor(_lens(case), device="cuda")
    return flat, start, size


def _exact_conv(st):
    flat, start, size = _starts(st)
    x, K = flat(st["x"]), st["w"].shape[1]
    w, state = st["w"].double(), st["state"].double()
    owner = torch.repeat_interleave(torch.arange(len(size), device="cuda"), size)
    place = torch.arange(x.shape[0], device="cuda") - start[owner]
    slot = st["slots"].long()
    y = st["bias"].double().expand(x.shape[0], -1).clone()
    for j in range(K):
        back = K - 1 - j                                  # tap j meets the input `back` tokens ago
        early = place < back
        now = x[(torch.arange(x.shape[0], device="cuda") - back).clamp_min(0)].double()
        rows = torch.nonzero(early)[:, 0]
        now[rows] = state[slot[owner[rows]], place[rows] - back + K - 1]
        y += now * w[:, j]
        del now
    if st["case"]["silu"]:
        y = y / (1 + torch.exp(-y))
    new = state.clone()
    for j in range(K - 1):
        at = size - (K - 1) + j                           # place of the input kept in row j
        kept = state[slot, (at + K - 1).clamp(0, K - 2)]
        new[slot] = new[slot].index_copy(1, torch.tensor([j], device="cuda"), torch.where(
            (at >= 0)[:, None], x[(start + at).clamp(0, x.shape[0] - 1)].double(), kept)[:, None])
    return {"y": y.view(st["x"].shape), "state": new}


def _exact_scan(st):
    flat, start, size = _starts(st)
    x, dt, B, C = (flat(st[k]) for k in ("x", "dt", "B", "C"))
    if st["max_len"] * st["state"].numel() > 2 ** 40:
        return None
    H, G, slot = x.shape[1], B.shape[1], st["slots"].long()
    A, D, bias = (st[k].double() for k in ("A", "D", "dt_bias"))
    h = st["state"][slot].double()
    y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    of = torch.arange(H, device="cuda") // (H // G)
    shortest = min(_lens(st["case"]))
    for t in range(st["max_len"]):
        live = slice(None) if t < shortest else torch.nonzero(size > t)[:, 0]
        at = (start + t)[live]
        step = torch.log1p(torch.exp(dt[at].double() + bias))
        xt, bt, ct = x[at].double(), B[at].double()[:, of], C[at].double()[:, of]
        now = h[live] * torch.exp(step * A)[..., None, None] + (step[..., None] * xt)[..., None] * bt[:, :, None, :]
        h[live] = now
        y[at] = (now @ ct[..., None])[..., 0] + D[:, None] * xt
    if st["z"] is not None:
        z = flat(st["z"]).double()
        y = y * z / (1 + torch.exp(-z))
    new = st["state"].double()
    new[slot] = h
    return {"y": y.view(st["x"].shape), "state": new}


def _exact_norm(st):
    case = st["case"]
    r = st["x"].double()
    got = {}
    if st["residual"] is not None:
        r = r + st["residual"].double()
        got["residual"] = r
    v = r / torch.sqrt((r ** 2).sum(1, keepdim=True) / r.shape[1] + 1e-6) * st["w"].double()
    if case["out"] == "io":
        return {"y": v, **got}
    top, width = (448.0 if case["out"] == "e4m3" else 127.0), case["group"] or v.shape[1]
    y, scales = torch.empty_like(v), []
    for at in range(0, v.shape[1], width):
        part = v[:, at:at + width]
        scale = part.abs().max(1, keepdim=True).values / top
        q = part / scale
        y[:, at:at + width] = q.to(torch.float8_e4m3fn).double() if top == 448.0 else torch.round(q) * scale
        scales.append(scale)
    scale = torch.cat(scales, 1)
    return {"y": y, "scale": scale if case["group"] else scale[:, 0], **got}
