"""The state space layer's operators against their float64 references.

Tolerances are derived.  u32 = 2^-24 and u16 = 2^-8 are the largest relative errors of a rounding
to float32 and bfloat16; a float32 sum of n terms is off by at most n u32 times the sum of their
magnitudes, which the references return.
"""
import numpy as np
import pytest
import torch

from oracle import layer_ref as ref

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def vla():
    from _util import ensure_built
    ensure_built()
    import sherman_morrison_inverse_gb300 as m
    return m


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def rand(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows_view(gen, lead, width, before, after, dtype):
    return rand(gen, *lead, before + width + after, dtype=dtype)[..., before:before + width]


def batch(lens, packed):
    """(leading shape, offsets tensor, list of (start, length))."""
    if packed:
        off = np.concatenate([[0], np.cumsum(lens)])
        return (int(off[-1]),), torch.tensor(off, dtype=torch.int32, device="cuda"), list(zip(off[:-1], lens))
    return (len(lens), lens[0]), None, [(i * lens[0], lens[0]) for i in range(len(lens))]


def close(got, want, bound, what):
    got = np.asarray(got, np.float64)
    assert np.isfinite(got).all(), what
    worst = float(np.max(np.abs(got - want) / bound)) if got.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times its bound"


# ---------------------------------------------------------------------------------------------
# convolution

CONV = [  # lens, packed, C, K, dtype, silu, (before, after)
    ([1], False, 8, 2, "f32", False, (0, 0)),
    ([1] * 5, False, 264, 4, "bf16", True, (8, 16)),
    ([2, 1, 3, 40, 0, 33], True, 24, 4, "bf16", True, (0, 0)),
    ([2, 1, 3, 0, 65], True, 37, 3, "f32", True, (3, 2)),
    ([100, 100], False, 1161, 3, "bf16", False, (0, 0)),
    ([31, 32, 64], True, 130, 2, "bf16", True, (0, 0)),
    ([1, 1, 1], True, 4096, 4, "f32", True, (0, 0)),
    ([257] * 3, False, 2048, 4, "bf16", True, (0, 8)),
]


@pytest.mark.parametrize("lens,packed,C,K,dtype,silu,more", CONV)
def test_short_conv_matches_the_reference(vla, lens, packed, C, K, dtype, silu, more):
    gen, dt = generator(C + K), TYPES[dtype]
    lead, off, where = batch(lens, packed)
    x = rows_view(gen, lead, C, *more, dt)
    w, bias = rand(gen, C, K), rand(gen, C)
    slots = torch.randperm(len(lens) + 2, generator=gen, device="cuda")[:len(lens)].to(torch.int32)
    state = rand(gen, len(lens) + 2, K - 1, C, dtype=dt)
    before = f64(state)
    y = vla.short_conv(x, w, bias, state, silu=silu, offsets=off, slots=slots)
    after, flat, got = f64(state), f64(x).reshape(-1, C), f64(y).reshape(-1, C)
    u = U32 if dtype == "f32" else U16
    untouched = np.ones(len(before), bool)
    for s, (at, n) in enumerate(where):
        slot = int(slots[s])
        untouched[slot] = False
        yr, ya, hr = ref.short_conv(flat[at:at + n], f64(w), f64(bias), before[slot], silu)
        # K products and sums; SiLU's slope is at most 1.1, its exponential and quotient a few ulp
        # and |argument| ulp of the argument's rounding
        bound = u * np.abs(yr) + (K + 2) * U32 * ya * 1.2 + 2.0 ** -20 * (1 + ya) * np.abs(yr) + 1e-30
        close(got[at:at + n], yr, bound, f"y of sequence {s}")
        assert np.array_equal(after[slot], hr), f"state of sequence {s}"
    assert np.array_equal(after[untouched], before[untouched])


def test_short_conv_split_at_any_token_gives_the_same_bits(vla):
    gen = generator(5)
    x, w = rand(gen, 2, 77, 40, dtype=torch.bfloat16), rand(gen, 40, 4)
    s0 = torch.zeros(2, 3, 40, dtype=torch.bfloat16, device="cuda")
    whole, s1 = vla.short_conv(x, w, None, s0), torch.zeros_like(s0)
    parts = [vla.short_conv(x[:, a:b], w, None, s1) for a, b in ((0, 1), (1, 3), (3, 40), (40, 76))]
    parts.append(vla.short_conv_step(x[:, 76], w, None, s1).unsqueeze(1))
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(s0, s1)
    assert torch.equal(vla.short_conv(x, w), whole)   # no state: zeros


# ---------------------------------------------------------------------------------------------
# scan

def scan_inputs(gen, lead, H, P, G, N, dt, gate, strided):
    if strided:   # x | B | C as one row, z and dt slices of another
        row = rand(gen, *lead, H * P + 2 * G * N, dtype=dt)
        x, B, C = row.split([H * P, G * N, G * N], -1)
        proj = rand(gen, *lead, H * P + H + 3, dtype=dt)
        z, d = proj[..., :H * P], proj[..., H * P + 3:]
    else:
        x, B, C, z, d = (rand(gen, *lead, n, dtype=dt) for n in (H * P, G * N, G * N, H * P, H))
    u = lambda t, *s: t.unflatten(-1, s)   # noqa: E731
    step = torch.exp(torch.rand(H, generator=gen, device="cuda") * 4.6 - 6.9)
    return dict(x=u(x, H, P), dt=d, A=-(1 + 15 * torch.rand(H, generator=gen, device="cuda")), B=u(B, G, N),
                C=u(C, G, N), D=rand(gen, H), z=u(z, H, P) if gate else None,
                dt_bias=step + torch.log(-torch.expm1(-step)))


def check_scan(vla, gen, lens, packed, H, P, G, N, dtype, gate, strided, rel=None, change=None, **kw):
    dt = TYPES[dtype]
    lead, off, where = batch(lens, packed)
    v = scan_inputs(gen, lead, H, P, G, N, dt, gate, strided)
    if change:
        change(v)
    slots = torch.randperm(len(lens) + 1, generator=gen, device="cuda")[:len(lens)].to(torch.int32)
    state = rand(gen, len(lens) + 1, H, P, N)
    before = f64(state)
    y = vla.ssm_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], state, D=v["D"], z=v["z"], dt_bias=v["dt_bias"],
                     offsets=off, slots=slots, **kw)
    after = f64(state)
    flat = {k: f64(t).reshape(-1, *t.shape[len(lead):]) if k in ("x", "dt", "B", "C", "z") and t is not None
            else f64(t) for k, t in v.items()}
    got = f64(y).reshape(-1, H, P)
    u = U32 if dtype == "f32" else U16
    spare = np.ones(len(before), bool)
    off2, size2 = 0.0, 0.0
    for s, (at, n) in enumerate(where):
        slot = int(slots[s])
        spare[slot] = False
        cut = lambda k: None if flat[k] is None else flat[k][at:at + n]   # noqa: E731
        yr, ya, hr, ha = ref.ssm_scan(cut("x"), cut("dt"), flat["A"], cut("B"), cut("C"), before[slot], flat["D"],
                                      cut("z"), flat["dt_bias"])
        # A state element is a sum of n + 1 terms, each through at most n decays; a decay is off by
        # its own rounding, exp's (2 ulp) and the argument's (|A s| u32, twice): 8 u32 a token for
        # |A s| <= 2 (what decays faster no longer counts), 4 u32 for the input's products; the
        # tensor cores' accumulation truncates: 3 terms of 128 products a chunk, 2 u32 each.
        c = (8 * n + 4 + 6 * 128 * -(-n // 128)) * U32
        close(after[slot], hr, c * ha + 1e-30, f"state of sequence {s}")
        # bfloat16 products: the masked matrix and the state operand are each rounded once
        bound = u * np.abs(yr) + (c + (N + 8) * U32 + (U16 if dtype == "bf16" else 0)) * ya + 1e-30
        bound += 2.0 ** -20 * (1 + np.abs(cut("z"))) * np.abs(yr) if gate else 0
        close(got[at:at + n], yr, bound, f"y of sequence {s}")
        off2 += float(((got[at:at + n] - yr) ** 2).sum())
        size2 += float((yr ** 2).sum())
    # two independent roundings (operand, output), each at most u / sqrt(3) of the result in the mean
    if size2:
        assert (off2 / size2) ** 0.5 <= (1.5 * u * (2 / 3) ** 0.5 if dtype == "bf16" else 2e-6)
    assert np.array_equal(after[spare], before[spare])
    return y


SCAN = [  # lens, packed, H, P, G, N, dtype, gate, strided
    ([1], False, 2, 64, 1, 128, "bf16", True, False),
    ([1] * 7, False, 4, 64, 2, 64, "bf16", True, True),
    ([1] * 3, False, 3, 40, 1, 20, "f32", True, True),
    ([5, 5], False, 2, 33, 2, 13, "bf16", False, True),
    ([130, 130], False, 2, 64, 1, 64, "f32", False, False),
    ([3, 0, 1, 17, 50], True, 4, 16, 2, 256, "f32", True, False),
    ([127], False, 2, 64, 1, 128, "bf16", False, False),
    ([128, 128], False, 4, 64, 2, 128, "bf16", True, True),
    ([129, 129], False, 2, 64, 1, 128, "bf16", True, False),
    ([1000], False, 8, 64, 1, 128, "bf16", True, True),
    ([2050], False, 2, 128, 1, 64, "bf16", True, False),
    ([1, 300, 0, 64, 257, 128, 31], True, 4, 64, 2, 64, "bf16", True, True),
    ([700, 5, 384], True, 2, 128, 1, 128, "bf16", False, False),
    ([200, 333], True, 3, 72, 3, 88, "bf16", True, False),
    ([400], False, 2, 32, 1, 16, "bf16", True, False),
    ([260], False, 2, 64, 2, 192, "bf16", True, False),
    ([150, 70], True, 2, 64, 1, 100, "bf16", True, False),
]


@pytest.mark.parametrize("lens,packed,H,P,G,N,dtype,gate,strided", SCAN)
def test_ssm_scan_matches_the_reference(vla, lens, packed, H, P, G, N, dtype, gate, strided):
    check_scan(vla, generator(H * P + N), lens, packed, H, P, G, N, dtype, gate, strided)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 20, 300])
def test_ssm_scan_with_strong_and_with_no_decay(vla, T, dtype):
    def change(v):
        v["A"][0] = 0.0          # the state only grows
        v["A"][1] = -3000.0      # nothing is left after a token
        v["dt"][..., 2] = 30.0   # softplus is the identity there
        v["dt"][..., 3] = -30.0  # and an exponential here
    check_scan(vla, generator(T), [T, T], False, 4, 64, 1, 64, dtype, True, False, change=change)


def test_ssm_scan_with_a_few_heads_more_than_a_wave(vla):
    """160 heads on 152 SMs: the last 8 are cut into segments of their own lengths, the others are not."""
    check_scan(vla, generator(61), [700], False, 160, 8, 1, 16, "bf16", True, False)
    check_scan(vla, generator(62), [400, 400], False, 40, 128, 2, 64, "bf16", False, True)


def test_ssm_scan_of_sequences_far_shorter_than_they_may_be(vla):
    """Rows for two sequences of 700 tokens, 60 and 641 of them used: fewer segments than there is room for."""
    gen = generator(63)
    v = scan_inputs(gen, (1400,), 80, 8, 1, 16, torch.bfloat16, True, False)
    off = torch.tensor([0, 60, 701], dtype=torch.int32, device="cuda")
    state, y = rand(gen, 2, 80, 8, 16), torch.full_like(v["x"], 7.0)
    before = f64(state)
    vla.ssm_scan(**v, state=state, y=y, offsets=off, max_len=700)
    for s, (a, b) in enumerate(((0, 60), (60, 701))):
        cut = lambda k: f64(v[k][a:b])   # noqa: E731
        yr, ya, hr, ha = ref.ssm_scan(cut("x"), cut("dt"), f64(v["A"]), cut("B"), cut("C"), before[s], f64(v["D"]),
                                      cut("z"), f64(v["dt_bias"]))
        c = (8 * (b - a) + 4 + 6 * 128 * -(-(b - a) // 128)) * U32   # as in check_scan
        close(f64(state[s]), hr, c * ha + 1e-30, "state")
        bound = (U16 + 2.0 ** -20 * (1 + np.abs(cut("z")))) * np.abs(yr) + (c + (16 + 8) * U32 + U16) * ya + 1e-30
        close(f64(y[a:b]), yr, bound, "y")
    assert (y[701:] == 7).all()


def test_ssm_scan_without_options(vla):
    gen = generator(3)
    v = scan_inputs(gen, (2, 200), 2, 64, 1, 64, torch.bfloat16, False, False)
    step = torch.rand(2, 200, 2, generator=gen, device="cuda").to(torch.bfloat16)
    y = vla.ssm_scan(v["x"], step, v["A"], v["B"], v["C"], softplus=False)
    for s in range(2):
        yr, ya, _, _ = ref.ssm_scan(f64(v["x"][s]), f64(step[s]), f64(v["A"]), f64(v["B"][s]), f64(v["C"][s]),
                                    np.zeros((2, 64, 64)), softplus_on=False)
        close(f64(y[s]), yr, U16 * np.abs(yr) + (U16 + 3000 * U32) * ya + 1e-30, "y")


def test_ssm_tokens_continue_a_prompt(vla):
    """A prompt and then single tokens give what the longer prompt gives: the same state bit for bit
    (the same operations on every element), and outputs whose sums over N may run in another order."""
    gen = generator(11)
    v = scan_inputs(gen, (3, 140), 4, 64, 2, 128, torch.float32, True, False)
    part = lambda a, b: {k: t[:, a:b] if k in ("x", "dt", "B", "C", "z") else t for k, t in v.items()}   # noqa: E731
    s0 = torch.zeros(3, 4, 64, 128, device="cuda")
    s1 = s0.clone()
    whole = vla.ssm_scan(state=s0, **v)
    got = [vla.ssm_scan(state=s1, **part(0, 133))]
    for t in range(133, 140):
        one = {k: a[:, 0] if k in ("x", "dt", "B", "C", "z") else a for k, a in part(t, t + 1).items()}
        got.append(vla.ssm_step(state=s1, **one).unsqueeze(1))
    assert torch.equal(s0, s1)
    for s in range(3):
        one = lambda k: f64(v[k][s])   # noqa: E731
        _, ya, _, _ = ref.ssm_scan(one("x"), one("dt"), f64(v["A"]), one("B"), one("C"), np.zeros((4, 64, 128)),
                                   f64(v["D"]), one("z"), f64(v["dt_bias"]))
        close(f64(torch.cat(got, 1)[s]), f64(whole[s]), 2 * (128 + 8) * U32 * ya + 1e-30, "y")


@pytest.mark.parametrize("T", [1, 9, 200])
def test_skipped_and_invalid_sequences_touch_nothing(vla, T):
    gen = generator(T)
    h = vla.Handle()
    v = scan_inputs(gen, (4, T), 2, 64, 1, 64, torch.bfloat16, True, False)
    slots = torch.tensor([2, -1, 7, 0], dtype=torch.int32, device="cuda")   # 7 is outside the pool
    state = rand(gen, 3, 2, 64, 64)
    before = state.clone()
    y = torch.full_like(v["x"], 7.0)
    h.ssm_scan(state=state, y=y, slots=slots, **v)
    st = h.status()
    assert st["index"] and st["flags"] == vla.STATUS_INDEX
    assert (y[1] == 7).all() and (y[2] == 7).all() and not (y[0] == 7).all() and not (y[3] == 7).all()
    assert torch.equal(state[1], before[1]) and not torch.equal(state[0], before[0])
    w, cs = rand(gen, 64, 4), rand(gen, 3, 3, 64, dtype=torch.bfloat16)
    x = rand(gen, 4, T, 64, dtype=torch.bfloat16)
    y = torch.full_like(x, 7.0)
    before = cs.clone()
    h.short_conv(x, w, None, cs, y, slots=slots)
    assert h.status()["index"] and (y[1] == 7).all() and (y[2] == 7).all() and torch.equal(cs[1], before[1])
    off = torch.tensor([0, T, T - 1, 2 * T, 4 * T + 1], dtype=torch.int32, device="cuda")   # 1 decreases, 3 runs out
    x = x.flatten(0, 1)
    y = torch.full_like(x, 7.0)
    h.short_conv(x, w, None, None, y, offsets=off)
    assert h.status()["index"] and not (y[:2 * T] == 7).all(-1).any() and (y[2 * T:] == 7).all()
    h.close()


@pytest.mark.parametrize("T", [40, 300])
def test_neighbours_in_a_packed_batch_do_not_meet(vla, T):
    """NaN and infinity in one sequence, and in rows of no sequence, stay there."""
    gen = generator(T)
    v = scan_inputs(gen, (3 * T + 5,), 2, 64, 1, 64, torch.bfloat16, True, False)
    for k, bad in (("x", float("nan")), ("B", float("inf")), ("C", float("nan")), ("z", float("nan")), ("dt", float("nan"))):
        v[k][T:2 * T] = bad
        v[k][3 * T:] = bad
    off = torch.tensor([0, T, 2 * T, 3 * T], dtype=torch.int32, device="cuda")
    state = torch.zeros(3, 2, 64, 64, device="cuda")
    y = vla.ssm_scan(state=state, offsets=off, **v)
    assert y[:T].isfinite().all() and y[2 * T:3 * T].isfinite().all() and y[T:2 * T].isnan().any()
    assert state[0].isfinite().all() and state[2].isfinite().all() and state[1].isnan().any()
    alone = {k: t[2 * T:3 * T].unsqueeze(0) if k in ("x", "dt", "B", "C", "z") else t for k, t in v.items()}
    got, want = vla.ssm_scan(**alone)[0].double(), y[2 * T:3 * T].double()
    assert (got - want).norm() <= 2 * U16 * want.norm()   # a batch may be split along T in another way


def test_scan_is_repeatable_and_runs_on_a_side_stream_and_in_a_graph(vla):
    gen = generator(21)
    v = scan_inputs(gen, (2, 500), 4, 64, 1, 128, torch.bfloat16, True, True)
    y0 = vla.ssm_scan(**v)
    assert torch.equal(y0, vla.ssm_scan(**v))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1 = vla.ssm_scan(stream=side, **v)
    side.synchronize()
    assert torch.equal(y0, y1)
    y2 = torch.zeros_like(y0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vla.ssm_scan(y=y2, **v)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y0, y2)


# ---------------------------------------------------------------------------------------------
# norm

NORM = [  # rows, D, dtype, residual, out, group
    (1, 1, "f32", None, "io", 0),
    (5, 64, "bf16", "bf16", "e4m3", 0),
    (3, 1001, "f32", None, "io", 0),
    (7, 1001, "bf16", "f32", "int8", 128),
    (4, 5120, "bf16", "f32", "int8", 128),
    (2, 8192, "bf16", "bf16", "e4m3", 128),
    (2, 9000, "f32", "f32", "int8", 0),
    (3, 200, "f32", "bf16", "e4m3", 128),
    (2, 20001, "bf16", "bf16", "int8", 128),
    (2, 32768, "f32", None, "e4m3", 0),
    (2, 32768, "bf16", "f32", "io", 0),
    (9, 40, "bf16", None, "int8", 0),
    # rows off 16-byte boundaries, many or wide: through shared memory, by 1, 2, 4 and 8 warps a row
    (700, 1001, "bf16", "bf16", "e4m3", 0),
    (640, 1003, "bf16", "f32", "int8", 128),
    (2600, 257, "bf16", None, "io", 0),
    (333, 2003, "f32", "f32", "io", 0),
    (333, 2003, "bf16", "bf16", "int8", 128),
    (401, 2047, "f32", "bf16", "e4m3", 0),
    (3, 7195, "bf16", "bf16", "io", 0),
    (4, 4099, "f32", None, "e4m3", 128),
    (5, 20001, "f32", "f32", "int8", 128),
]


@pytest.mark.parametrize("rows,D,dtype,res,out,group", NORM)
def test_rms_norm_matches_the_reference(vla, rows, D, dtype, res, out, group):
    gen = generator(rows + D)
    x = rows_view(gen, (rows,), D, 8, 8, TYPES[dtype]) if rows % 2 else rand(gen, rows, D, dtype=TYPES[dtype])
    w = rand(gen, D)
    residual = rand(gen, rows, D, dtype=TYPES[res]) * 3 if res else None
    vr, rr = ref.rms_norm(f64(x), f64(w), f64(residual) if res else np.zeros((rows, D)), 1e-5)
    got = vla.rms_norm(x, w, residual, eps=1e-5, out=out, group=group)
    if res:
        # the kernel's float32 sum rounded to the residual's type
        close(f64(residual), rr, (U32 + (U16 if res == "bf16" else U32)) * np.abs(rr) + 1e-30, "residual")
    # r's rounding, the mean's (n + 2 sums, halved by the root), the root's and two products
    c = (D / 2 + 8) * U32
    if out == "io":
        u = U32 if dtype == "f32" else U16
        close(f64(got), vr, (c + u) * np.abs(vr) + 1e-30, "y")
        return
    codes, scale = got
    top = 448.0 if out == "e4m3" else 127.0
    sr = ref.scales(vr, top, group)
    scale = f64(scale).reshape(rows, -1)
    close(scale, sr, (c + 2 * U32) * sr, "scale")
    wide = np.repeat(scale, group or D, 1)[:, :D]
    q = f64(codes)
    assert np.abs(q).max() <= top
    # half a step: of an integer, or of an e4m3 with 3 bits after the point (2^-4 relative, 2^-10 least)
    step = 0.5 * wide if out == "int8" else np.maximum(np.abs(vr) * 2.0 ** -4, wide * 2.0 ** -10)
    close(q * wide, vr, step * (1 + 1e-3) + (c + 4 * U32) * np.abs(vr) + 1e-30, "codes * scale")


@pytest.mark.parametrize("rows,D,dtype", [(700, 1001, "bf16"), (3, 7195, "bf16"), (400, 2003, "f32"), (3, 1001, "bf16")])
def test_rms_norm_leaves_what_lies_between_rows(vla, rows, D, dtype):
    """x, residual and y at offsets of their own in wider rows: the same values, and nothing beside them changes."""
    gen = generator(rows)
    x, w, r = rand(gen, rows, D, dtype=TYPES[dtype]), rand(gen, D), rand(gen, rows, D)
    r2, y2 = torch.full((rows, D + 9), 7.0, device="cuda"), torch.full((rows, D + 6), 7.0, device="cuda", dtype=x.dtype)
    x2 = torch.full((rows, D + 4), float("nan"), device="cuda", dtype=x.dtype)
    r2[:, 5:D + 5], x2[:, 3:D + 3] = r, x
    y = vla.rms_norm(x, w, r)
    vla.rms_norm(x2[:, 3:D + 3], w, r2[:, 5:D + 5], y=y2[:, 1:D + 1])
    assert torch.equal(y2[:, 1:D + 1], y) and torch.equal(r2[:, 5:D + 5], r)
    assert (r2[:, :5] == 7).all() and (r2[:, D + 5:] == 7).all() and (y2[:, :1] == 7).all() and (y2[:, D + 1:] == 7).all()


def test_rms_norm_of_zeros_and_of_nan(vla):
    x = torch.zeros(3, 256, device="cuda", dtype=torch.bfloat16)
    x[1, 7] = float("nan")
    x[2, 200] = 5.0
    w = torch.ones(256, device="cuda")
    for out in ("e4m3", "int8"):
        q, s = vla.rms_norm(x, w, out=out)
        assert (q[0].float() == 0).all() and s[0] == 1 and s[1].isnan() and s[2] > 0
        assert q[2].float().abs().max() == (448 if out == "e4m3" else 127)
        q, s = vla.rms_norm(x, w, out=out, group=128)
        assert s.shape == (3, 2) and s[0].tolist() == [1, 1] and s[1].isnan().all() and s[2, 0] == 1
    assert vla.rms_norm(x, w)[0].float().abs().max() == 0
    w[100] = float("nan")   # of the filter: every row's scale, or its group's
    for D in (256, 255):
        xs, ws = x[:, :D].contiguous(), w[:D].contiguous()
        assert vla.rms_norm(xs, ws, out="int8")[1].isnan().all()
        s = vla.rms_norm(xs, ws, out="e4m3", group=128)[1]
        assert s[:, 0].isnan().all() and not s[2, 1].isnan()
        ws[100] = float("inf")   # times x's zero
        assert vla.rms_norm(xs, ws, out="e4m3")[1].isnan().all()


# ---------------------------------------------------------------------------------------------
# refusals

def test_refusals(vla):
    gen = generator(1)
    x, w = rand(gen, 2, 8, 16), rand(gen, 16, 4)
    conv = lambda *a, **k: pytest.raises(ValueError, vla.short_conv, *a, **k)   # noqa: E731
    conv(x[0], w)
    conv(x.half(), w)
    conv(x.transpose(1, 2), rand(gen, 8, 4))
    conv(x, w.bfloat16())
    conv(x, rand(gen, 15, 4))
    conv(x, w, state=rand(gen, 2, 4, 16))
    conv(x, w, slots=torch.zeros(2, dtype=torch.int32, device="cuda"))
    conv(x, w, y=rand(gen, 2, 8, 17))
    conv(x, w.cpu())
    with pytest.raises(vla.VlaError, match="taps"):
        vla.short_conv(x, rand(gen, 16, 5))
    with pytest.raises(vla.VlaError, match="fewer states"):
        vla.short_conv(x, w, state=rand(gen, 1, 3, 16))
    with pytest.raises(vla.VlaError, match="overlap"):
        vla.short_conv(x, w, y=rand(gen, 1, 8, 16).expand(2, 8, 16))
    v = scan_inputs(gen, (2, 8), 4, 16, 2, 16, torch.float32, True, False)
    vla.ssm_scan(**v)
    for name, bad in (("dt", v["dt"].bfloat16()), ("A", v["A"][:3]), ("C", v["C"][..., :8]), ("z", v["z"][:1]),
                      ("B", v["B"].transpose(2, 3)), ("state", rand(gen, 2, 4, 16, 17))):
        with pytest.raises(ValueError):
            vla.ssm_scan(**{**v, name: bad})
    with pytest.raises(vla.VlaError, match="multiple of G"):
        vla.ssm_scan(**{**v, "B": rand(gen, 2, 8, 3, 16), "C": rand(gen, 2, 8, 3, 16)})
    with pytest.raises(vla.VlaError, match="256"):
        vla.ssm_scan(**{**v, "B": rand(gen, 2, 8, 2, 260), "C": rand(gen, 2, 8, 2, 260)})
    with pytest.raises(ValueError):
        vla.ssm_step(**v)
    x, w = rand(gen, 4, 64), rand(gen, 64)
    for kw in (dict(out="fp4"), dict(group=64), dict(residual=rand(gen, 4, 63)), dict(residual=rand(gen, 4, 64).half())):
        with pytest.raises(ValueError):
            vla.rms_norm(x, w, **kw)
    with pytest.raises(vla.VlaError, match="eps"):
        vla.rms_norm(x, w, eps=-1.0)
    with pytest.raises(vla.VlaError, match="32768"):
        vla.rms_norm(rand(gen, 1, 40000), rand(gen, 40000))
    assert vla.rms_norm(x[:0], w).shape == (0, 64)
    assert vla.short_conv(rand(gen, 2, 0, 16), rand(gen, 16, 4)).shape == (2, 0, 16)


def test_a_layer_decodes_what_it_would_prefill(vla):
    """The example's stack: prompts, then tokens from the kept states, against longer prompts.

    The two differ by the roundings of bfloat16 activations (2^-8 each, about six in a layer) and by
    e4m3 codes that fall to the other side (2^-4 of the value, for the few that are that near)."""
    import importlib.util
    import os
    from _util import ROOT
    spec = importlib.util.spec_from_file_location("state_space_layer",
                                                  os.path.join(ROOT, "examples", "state_space_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.demo(width=256, heads=4, n_layers=2, n_tokens=5, lens=(3, 140, 29, 1)) <= 0.05


# ---------------------------------------------------------------------------------------------
# layouts and sizes away from the ordinary

@pytest.mark.parametrize("form", ["token-major", "odd start", "shared B and C"])
def test_ssm_scan_with_other_strides(vla, form):
    """Sequences interleaved token by token; rows off every 16-byte boundary (another kernel); B and C
    broadcast over the sequences.  The values are those of contiguous copies."""
    gen = generator(31)
    v = scan_inputs(gen, (3, 150), 4, 64, 2, 64, torch.bfloat16, True, False)
    if form == "token-major":
        v = {k: t.transpose(0, 1).contiguous().transpose(0, 1) if k in ("x", "dt", "B", "C", "z") else t for k, t in v.items()}
        out = torch.empty(150, 3, 4, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    elif form == "odd start":
        def shift(t):
            flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:]
            return flat.copy_(t.flatten()).view(t.shape)
        v = {k: shift(t) if k in ("x", "dt", "B", "C", "z") else t for k, t in v.items()}
        out = shift(torch.zeros(3, 150, 4, 64, dtype=torch.bfloat16, device="cuda"))
    else:
        v["B"], v["C"] = v["B"][:1].expand(3, -1, -1, -1), v["C"][:1].expand(3, -1, -1, -1)
        out = None
    state = torch.zeros(3, 4, 64, 64, device="cuda")
    y = vla.ssm_scan(state=state, y=out, **v)
    if out is not None:
        assert y.data_ptr() == out.data_ptr()
    for s in range(3):
        one = lambda k: f64(v[k][s])   # noqa: E731
        yr, ya, hr, ha = ref.ssm_scan(one("x"), one("dt"), f64(v["A"]), one("B"), one("C"), np.zeros((4, 64, 64)),
                                      f64(v["D"]), one("z"), f64(v["dt_bias"]))
        c = (8 * 150 + 4 + 6 * 256) * U32
        close(f64(state[s]), hr, c * ha + 1e-30, "state")
        close(f64(y[s]), yr, (U16 + 2.0 ** -20 * (1 + np.abs(one("z")))) * np.abs(yr) + (c + U16) * ya + 1e-30, "y")


def test_short_conv_with_interleaved_sequences(vla):
    gen = generator(32)
    x = rand(gen, 70, 3, 96, dtype=torch.bfloat16).transpose(0, 1)
    w = rand(gen, 96, 4)
    assert torch.equal(vla.short_conv(x, w), vla.short_conv(x.contiguous(), w))


@pytest.mark.parametrize("T", [1, 40, 200])
def test_states_and_rows_past_two_to_the_31(vla, T):
    """A pool and a token buffer whose last elements lie past 2^31: 64-bit offsets everywhere."""
    if torch.cuda.get_device_properties(0).total_memory < 60 * 2 ** 30:
        pytest.skip("needs 60 GB of device memory")
    gen = generator(T)
    H, P, G, N, width = 64, 64, 1, 128, 64 * 64 + 2 * 128
    slots = torch.tensor([4200, 3], dtype=torch.int32, device="cuda")
    state = torch.empty(4201, H, P, N, device="cuda")           # 2.2e9 floats
    state[3], state[4200] = 0.5, 0.25
    rows = 2 ** 31 // width + 2 * T + 1
    buf = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")
    tail = buf[rows - 2 * T:]
    tail.copy_(rand(gen, 2 * T, width))
    dt = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
    dt[rows - 2 * T:] = rand(gen, 2 * T, H).to(torch.bfloat16)
    A = -torch.rand(H, generator=gen, device="cuda")
    split = lambda t: (t[..., :4096].unflatten(-1, (H, P)), t[..., 4096:4224].unflatten(-1, (G, N)),   # noqa: E731
                       t[..., 4224:].unflatten(-1, (G, N)))
    off = torch.tensor([rows - 2 * T, rows - T, rows], dtype=torch.int32, device="cuda")
    x, B, C = split(buf)
    y = torch.empty(rows, H, P, dtype=torch.bfloat16, device="cuda")
    vla.ssm_scan(x, dt, A, B, C, state, y, offsets=off, slots=slots, max_len=T)
    small = torch.empty(2, H, P, N, device="cuda")
    small[0], small[1] = 0.25, 0.5
    xs, Bs, Cs = split(tail.clone())
    ys = vla.ssm_scan(xs, dt[rows - 2 * T:].clone(), A, Bs, Cs, small, offsets=off - (rows - 2 * T), max_len=T)
    assert torch.equal(y[rows - 2 * T:], ys) and torch.equal(state[4200], small[0]) and torch.equal(state[3], small[1])
    w = rand(gen, width, 4)
    out = torch.empty_like(buf)
    vla.short_conv(buf, w, None, None, out, offsets=off, max_len=T)
    assert torch.equal(out[rows - 2 * T:], vla.short_conv(tail.clone(), w, offsets=off - (rows - 2 * T), max_len=T))


def test_many_sequences(vla):
    """More sequences than a grid's second dimension holds."""
    gen = generator(33)
    S, H, P, N = 70001, 1, 8, 4
    x, dt, B, C = (rand(gen, S, *s) for s in ((H, P), (H,), (1, N), (1, N)))
    A, state = -torch.ones(H, device="cuda"), rand(gen, S, H, P, N)
    before = state.clone()
    y = vla.ssm_step(x, dt, A, B, C, state)
    step = torch.nn.functional.softplus(dt.double())
    h = torch.exp(-step)[..., None, None] * before.double() + step[..., None, None] * x.double()[..., None] * B.double()[:, :, None]
    assert (state - h).abs().max() <= 64 * U32 * h.abs().max()
    want = (h * C.double()[:, :, None]).sum(-1)
    assert (y - want).abs().max() <= 64 * U32 * (h * C.double()[:, :, None]).abs().sum(-1).max()
    cs, xs, w = torch.zeros(S, 1, 8, device="cuda"), rand(gen, S, 8), rand(gen, 8, 2)
    assert torch.equal(vla.short_conv_step(xs, w, None, cs, silu=False), xs * w[:, 1]) and torch.equal(cs[:, 0], xs)


def test_no_wait_runs_out_and_scratch_is_checked(vla):
    """Every form leaves the status clean, and a workspace that is too small is refused."""
    import ctypes
    h = vla.Handle()
    gen = generator(34)
    for lead, N in (((1, 3000), 128), ((2, 900), 64), ((40, 300), 128), ((3, 1), 64), ((2, 500), 20)):
        v = scan_inputs(gen, lead, 8, 64, 1, N, torch.bfloat16, True, False)
        h.ssm_scan(**v)
        assert h.status()["flags"] == 0
    need = ctypes.c_size_t()
    args = (h.ptr, 1, 3000, 3000, 0, 8, 64, 128, 1, ctypes.byref(need))
    assert h.lib.vla_ssm_workspace(*args) == 0 and need.value > 0
    x = torch.zeros(1, 3000, 8, 128, dtype=torch.bfloat16, device="cuda")
    f = torch.zeros(8, device="cuda")
    p, q = x.data_ptr(), f.data_ptr()
    strides = (ctypes.c_longlong * 12)(*[v for _ in range(6) for v in (3000 * 1024, 1024)])
    for ws, size in ((None, 0), (p, need.value - 1)):
        code = h.lib.vla_ssm_scan(h.ptr, p, p, q, p, p, None, None, None, None, p, 1, 3000, 3000, None, None, 0, 8, 64,
                                  1, 128, strides, 1, 1, ws, size, None)
        assert code == 1 and b"workspace" in h.lib.vla_last_error(h.ptr)
    h.close()


def test_misaligned_pointers_are_refused(vla):
    """Before any launch: each pointer in turn a byte off its type's alignment."""
    import ctypes
    h, p = vla.Handle(), torch.zeros(1 << 16, device="cuda").data_ptr()
    ones = lambda n: (ctypes.c_longlong * n)(*[64] * n)   # noqa: E731

    def refused(call, n):
        for i in range(n):
            assert call([p + (i == j) for j in range(n)]) == 1, i
            assert b"aligned" in h.lib.vla_last_error(h.ptr)

    refused(lambda q: h.lib.vla_short_conv(h.ptr, *q, 1, 4, 4, None, None, 1, 8, 4, ones(4), 0, 0, None), 5)
    refused(lambda q: h.lib.vla_ssm_scan(h.ptr, *q[:10], 1, 4, 4, None, None, 1, 2, 8, 1, 8, ones(12), 1, 0, None, 0,
                                         None), 10)
    refused(lambda q: h.lib.vla_rms_norm(h.ptr, *q, None, 1, 8, 8, 8, 8, 1e-6, 0, 0, 0, 0, None), 4)
    assert h.lib.vla_rms_norm(h.ptr, p, p, None, p, p + 1, 1, 8, 8, 8, 8, 1e-6, 0, 1, 0, 0, None) == 1
    h.close()
