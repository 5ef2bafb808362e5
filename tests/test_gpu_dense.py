"""Products with an epilogue, layer norm, and their gradients against their float64 references.

Tolerances are derived.  u32 = 2^-24 and u16 = 2^-8 bound the relative error of a rounding to float32 and
bfloat16.  A tensor core may cut an addition off instead of rounding it: 2 u32 of the running sum, which the sum of the
terms' magnitudes (the references return it) bounds.
"""
import numpy as np
import pytest
import torch

from oracle import dense_ref as ref

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
TINY = 2.0 ** -120
# activations: of float32 results a few ulp (expf, erfcf, a division) and the argument's rounding, which the
# exponential multiplies by the argument; of bfloat16 results 1.7e-5 by the polynomial, rounded up
FAST, PRECISE = 2.0 ** -14, 2.0 ** -20


@pytest.fixture(scope="module")
def vla():
    from _util import ensure_built
    ensure_built()
    import sherman_morrison_inverse_gb300 as m
    return m


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def rows_of(gen, rows, width, gap, dtype):
    """[rows, width] in rows that hold `gap` more values, half of them before (none: contiguous)."""
    return rand(gen, rows, width + gap).to(dtype)[:, gap // 2:gap // 2 + width]


def close(got, want, bound, what):
    got = np.asarray(got, np.float64)
    assert np.isfinite(got).all(), what
    worst = float(np.max(np.abs(got - want) / bound)) if got.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times its bound"


def product_error(K, mag, dtype):
    """Bound on a sum of K products whose magnitudes add up to `mag`."""
    terms = 0 if dtype != "f32" else 4   # float32 operands as three terms of bfloat16
    return (2 * K + 4 + terms) * U32 * mag


# ---------------------------------------------------------------------------------------------
# product

LINEAR = [  # M, N, K, in, out, act, bias, residual, pre, gap
    (1, 1, 1, "bf16", "bf16", "none", False, False, False, 0),
    (1, 8, 8, "f32", "f32", "silu", True, True, True, 0),
    (1, 264, 520, "bf16", "bf16", "gelu", True, True, False, 0),
    (1, 1001, 333, "bf16", "f32", "none", True, False, False, 1),
    (1, 777, 1000, "f32", "f32", "gelu", True, False, True, 0),
    (1, 130, 208, "e4m3", "bf16", "none", False, True, False, 0),
    (3, 4096, 64, "bf16", "bf16", "silu", False, False, True, 8),
    (5, 257, 129, "e4m3", "f32", "gelu", True, True, True, 0),
    (7, 640, 4096, "bf16", "f32", "none", False, True, False, 0),
    (9, 100, 2048, "f32", "f32", "none", False, True, False, 4),
    (16, 1024, 1024, "bf16", "bf16", "none", True, False, False, 0),
    (17, 96, 72, "bf16", "bf16", "gelu", True, True, True, 0),
    (33, 333, 77, "f32", "f32", "silu", True, False, False, 3),
    (64, 512, 4096, "e4m3", "bf16", "silu", True, True, False, 0),
    (65, 40, 8192, "bf16", "bf16", "none", False, False, False, 0),
    (100, 300, 200, "bf16", "bf16", "gelu", True, True, True, 24),
    (128, 128, 64, "bf16", "f32", "none", False, False, False, 0),
    (129, 384, 448, "e4m3", "bf16", "none", True, False, True, 16),
    (255, 513, 136, "bf16", "bf16", "silu", True, True, True, 2),
    (256, 256, 256, "bf16", "bf16", "none", False, False, False, 0),
    (257, 264, 2000, "bf16", "f32", "gelu", True, True, True, 16),
    (300, 777, 161, "f32", "f32", "gelu", True, True, True, 0),
    (512, 200, 1024, "f32", "f32", "none", False, False, False, 0),
    (513, 1032, 96, "bf16", "bf16", "gelu", True, False, True, 0),
    (1000, 24, 56, "bf16", "bf16", "none", True, True, False, 0),
    (1024, 1024, 4096, "bf16", "bf16", "none", False, True, False, 0),
    (2050, 520, 72, "e4m3", "f32", "silu", True, True, True, 0),
    (1, 16, 8192, "bf16", "bf16", "none", True, False, False, 0),      # Kd shared by the warps of a block
    (3, 20, 6001, "f32", "f32", "none", False, True, False, 0),
    (2, 4104, 4096, "e4m3", "bf16", "none", True, True, False, 0),
    (4, 2056, 1024, "bf16", "bf16", "silu", True, True, True, 0),
    (6, 131, 259, "e4m3", "bf16", "gelu", True, True, False, 0),
    (20, 300, 200, "f32", "f32", "gelu", True, True, True, 0),          # several eights of rows on CUDA cores
    (120, 70, 90, "bf16", "f32", "none", True, False, False, 0),
    (16, 1000, 2048, "bf16", "f32", "gelu", True, True, True, 0),       # a cluster's shares of Kd, every tile width
    (30, 1016, 2048, "bf16", "bf16", "none", True, True, True, 0),
    (40, 4096, 1024, "e4m3", "f32", "none", False, True, False, 0),
    (100, 1001, 4096, "bf16", "bf16", "silu", True, True, True, 0),
    (128, 8192, 4160, "bf16", "bf16", "none", True, True, False, 0),
    (127, 2048, 1024, "f32", "f32", "silu", True, True, True, 0),
    (130, 2000, 1000, "f32", "f32", "none", False, False, False, 0),
    (500, 1000, 1040, "bf16", "bf16", "gelu", True, True, True, 0),
    (600, 2000, 2048, "e4m3", "bf16", "none", True, False, False, 0),
    (530, 140, 8192, "bf16", "f32", "silu", True, True, True, 0),       # parts of Kd joined by a second kernel
    (700, 141, 4100, "bf16", "bf16", "gelu", True, True, True, 3),
    (3000, 2000, 40, "bf16", "bf16", "silu", True, True, False, 0),
]


def operands(gen, M, N, K, dtype, gap):
    """x, w, their scales, and what they stand for in 64 bits."""
    x, w = rows_of(gen, M, K, gap, TYPES[dtype]), rows_of(gen, N, K, gap, TYPES[dtype])
    if dtype != "e4m3":
        return x, w, None, None
    return x, w, rand(gen, M).abs() + 0.1, rand(gen, N).abs() + 0.1


@pytest.mark.parametrize("M,N,K,dtype,out,act,bias,residual,pre,gap", LINEAR)
def test_linear_matches_the_reference(vla, M, N, K, dtype, out, act, bias, residual, pre, gap):
    gen = generator(M + 3 * N + 7 * K)
    x, w, xs, ws = operands(gen, M, N, K, dtype, gap)
    w = (w.float() / K ** 0.5).to(w.dtype)
    b = rand(gen, N) if bias else None
    res = rows_of(gen, M, N, gap, TYPES[out]) if residual else None
    keep = rows_of(gen, M, N, gap, TYPES[out]) if pre else None
    around = keep._base.clone() if pre and gap else None
    y = vla.linear(x, w, b, res, act=act, pre=keep, x_scale=xs, w_scale=ws, dtype=TYPES[out])
    yr, v, mag = ref.linear(f64(x), f64(w), f64(b), f64(res), act, f64(xs), f64(ws))
    u, a = (U16, FAST) if out == "bf16" else (U32, PRECISE)
    off = product_error(K, mag, dtype)
    if pre:
        close(f64(keep), v, off + u * np.abs(v) + TINY, "pre")
    av = np.abs(ref.act(v, act))
    # the activations' slopes are at most 1.13
    bound = 1.2 * off + (a + PRECISE * (1 + np.abs(v)) ** 2) * av * (act != "none") + 2 * U32 * (av + np.abs(yr)) + u * np.abs(yr)
    close(f64(y), yr, bound + TINY, "y")
    if around is not None:   # what lies between the rows is left alone
        mine = torch.zeros_like(around, dtype=torch.bool)
        mine[:, gap // 2:gap // 2 + N] = True
        assert torch.equal(keep._base[~mine], around[~mine])


def test_linear_into_its_residual_and_other_shapes(vla):
    gen = generator(3)
    x, w = rand(gen, 2, 5, 64, dtype=torch.bfloat16), rand(gen, 40, 64, dtype=torch.bfloat16)
    stream = rand(gen, 2, 5, 40)
    want = vla.linear(x, w, residual=stream, dtype=torch.float32)
    assert want.shape == (2, 5, 40)
    got = vla.linear(x, w, None, stream, stream, dtype=torch.float32)
    assert got is stream and torch.equal(got, want)
    assert torch.equal(vla.linear(x[0, 0], w), vla.linear(x, w)[0, 0])   # one row without a leading dimension
    same = x[:1, :1].expand(2, 5, 64)                                    # one row ten times, without its memory
    assert torch.equal(vla.linear(same, w), vla.linear(same.contiguous(), w))


def test_linear_writes_rows_of_a_wider_tensor(vla):
    """y and the residual as slices, on 32-byte boundaries and off them; what lies between is left alone."""
    gen = generator(17)
    for M in (3, 60, 300):
        x, w = rand(gen, M, 72, dtype=torch.bfloat16), rand(gen, 96, 72, dtype=torch.bfloat16)
        res, b = rand(gen, M, 96, dtype=torch.bfloat16), rand(gen, 97)
        want = vla.linear(x, w, b[:96], res, act="silu")
        for before, width in ((16, 128), (3, 131), (8, 120)):
            wide = torch.full((M, width), 7.0, dtype=torch.bfloat16, device="cuda")
            room = torch.zeros(M, width, dtype=torch.bfloat16, device="cuda")
            room[:, before:before + 96] = res
            got = vla.linear(x, w, b[:96], room[:, before:before + 96], wide[:, before:before + 96], act="silu")
            assert torch.equal(got, want)
            assert (wide[:, :before] == 7).all() and (wide[:, before + 96:] == 7).all()
            off = torch.empty(97, device="cuda")[1:].copy_(b[:96])   # a bias on a 4-byte boundary
            assert torch.equal(vla.linear(x, w, off, room[:, before:before + 96], act="silu"), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("M", [1, 40, 200, 600])
def test_linear_gives_the_same_bits_every_time(vla, M, dtype):
    gen = generator(M)
    x, w, xs, ws = operands(gen, M, 520, 1040, dtype, 0)
    y = vla.linear(x, w, x_scale=xs, w_scale=ws)
    assert all(torch.equal(vla.linear(x, w, x_scale=xs, w_scale=ws), y) for _ in range(5))


def test_weights_and_gradients_of_repeated_rows(vla):
    """Operands whose rows lie in one place (stride 0), for every product that reads them."""
    gen = generator(23)
    for dt in (torch.bfloat16, torch.float32):
        row, x = rand(gen, 1, 64, dtype=dt), rand(gen, 300, 64, dtype=dt)
        for M in (1, 30, 300):
            assert torch.equal(vla.linear(x[:M], row.expand(48, 64)), vla.linear(x[:M], row.repeat(48, 1)))
        dy, w = rand(gen, 1, 48, dtype=dt), rand(gen, 48, 64, dtype=dt)
        a = vla.linear_backward(dy.expand(300, 48), x, w)
        b = vla.linear_backward(dy.repeat(300, 1), x, w)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert torch.equal(vla.linear(x, x), vla.linear(x, x.clone()))   # one tensor as both operands


def test_offsets_past_32_bits(vla):
    """Outputs, inputs and rows of more than 2^31 values: the last rows are those of a small call, or the reference's."""
    gen = generator(29)
    M, N, K = 530000, 4104, 40
    x, w, b = rand(gen, M, K, dtype=torch.bfloat16), rand(gen, N, K, dtype=torch.bfloat16), rand(gen, N)
    y = vla.linear(x, w, b, act="silu")
    assert torch.equal(y[-700:], vla.linear(x[-700:], w, b, act="silu"))
    pre = vla.linear(x, w, b)
    assert torch.equal(pre[-700:], vla.linear(x[-700:], w, b))
    dx, dw, db = vla.linear_backward(y, x, w, pre, act="silu")
    (want, _, _), (mag, _, _) = ref.linear_backward(f64(y[-50:]), f64(x[-50:]), f64(w), f64(pre[-50:]), "silu")
    close(f64(dx[-50:]), want, product_error(N, mag, "bf16") + (FAST + PRECISE * 30 + U16) * mag + U16 * np.abs(want) + TINY, "dx")
    parts = [vla.linear_backward(y[i:i + 53000], x[i:i + 53000], w, pre[i:i + 53000], act="silu", input=False) for i in range(0, M, 53000)]
    for got, i in ((dw, 1), (db, 2)):
        want = sum(p[i].double() for p in parts)
        # ten roundings to bfloat16 of parts of the sum and one of the whole; float32 sums of 53000 against 530000 terms, the
        # longest chain of additions 2600
        assert float((got.double() - want).norm() / want.norm()) < (2 * U16 if i == 1 else 2600 * U32 * 2)
    del dx, dw, pre
    nw, nb = rand(gen, N), rand(gen, N)
    h, stats = vla.layer_norm(y, nw, nb, stats=True)
    want, last = vla.layer_norm(y[-9:], nw, nb, stats=True)
    assert torch.equal(h[-9:], want) and torch.equal(stats[-9:], last)
    dx, dw, db = vla.layer_norm_backward(h, y, nw, stats)
    assert torch.equal(dx[-9:], vla.layer_norm_backward(h[-9:], y[-9:], nw, stats[-9:])[0])
    far = torch.empty(3, 2 ** 31 + 64, dtype=torch.bfloat16, device="cuda")[:, 7:7 + K]   # rows 4 GB apart
    far.copy_(x[:3])
    assert torch.equal(vla.linear(far, w, b), vla.linear(x[:3], w, b))


def test_linear_without_terms_and_without_rows(vla):
    x, w = torch.empty(3, 0, device="cuda"), torch.empty(5, 0, device="cuda")
    b, r = torch.randn(5, device="cuda"), torch.randn(3, 5, device="cuda")
    assert torch.equal(vla.linear(x, w, b, r), b + r)
    assert vla.linear(torch.empty(0, 8, device="cuda"), torch.ones(5, 8, device="cuda")).shape == (0, 5)
    assert vla.linear(torch.ones(3, 8, device="cuda"), torch.ones(0, 8, device="cuda")).shape == (3, 0)


@pytest.mark.parametrize("M", [1, 20, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_keeps_nan_and_infinity_to_their_rows(vla, M, dtype):
    gen = generator(M)
    x, w = rand(gen, M, 96, dtype=TYPES[dtype]), rand(gen, 200, 96, dtype=TYPES[dtype])
    clean = vla.linear(x, w)
    x[M // 2, 5], x[0, 3] = float("nan"), float("inf")
    y = vla.linear(x, w)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[M // 2] = bad[0] = True
    assert not y[bad].isfinite().any() and torch.equal(y[~bad], clean[~bad])


def test_linear_float32_keeps_small_and_large_values(vla):
    """Terms of every magnitude that float32 has, each within 2^-22 of itself where nothing else joins."""
    x = torch.diag(2.0 ** torch.arange(-100, 100, 5, device="cuda")) * 1.2345678
    w = torch.full((24, 40), 1.7654321, device="cuda")
    y = vla.linear(x, w)
    want = (f64(x) @ f64(w).T)
    assert np.max(np.abs(f64(y) / want - 1)) <= 2.0 ** -22


# ---------------------------------------------------------------------------------------------
# its gradients

BACK = [  # M, N, K, dtype, act, bias, gap
    (1, 1, 1, "f32", "gelu", True, 0),
    (1, 72, 40, "bf16", "silu", True, 0),
    (7, 129, 65, "f32", "silu", True, 1),
    (24, 256, 512, "bf16", "none", True, 0),
    (100, 333, 201, "bf16", "gelu", True, 3),
    (128, 64, 64, "bf16", "none", False, 8),
    (256, 256, 256, "bf16", "gelu", True, 0),
    (300, 520, 264, "f32", "none", True, 4),
    (513, 1001, 520, "f32", "gelu", True, 0),
    (1000, 24, 4096, "bf16", "silu", True, 0),
    (2049, 264, 136, "bf16", "gelu", True, 16),
    (4096, 512, 512, "bf16", "silu", False, 0),
    (5000, 16, 32, "f32", "silu", True, 0),
    (20000, 40, 24, "bf16", "gelu", True, 0),
    (3000, 1032, 1, "bf16", "silu", True, 0),
    (2000, 1, 1000, "bf16", "gelu", True, 0),
    (700, 300, 520, "bf16", "none", True, 5),
]


@pytest.mark.parametrize("M,N,K,dtype,act,bias,gap", BACK)
def test_linear_backward_matches_the_reference(vla, M, N, K, dtype, act, bias, gap):
    gen, dt = generator(M + N + K), TYPES[dtype]
    dy, x, w = (rows_of(gen, r, c, gap, dt) for r, c in ((M, N), (M, K), (N, K)))
    pre = rows_of(gen, M, N, gap, dt) if act != "none" else None
    dx, dw, db = vla.linear_backward(dy, x, w, pre, act=act, bias=bias)
    want, mag = ref.linear_backward(f64(dy), f64(x), f64(w), f64(pre), act)
    u = U16 if dtype == "bf16" else U32
    a = 0.0 if act == "none" else (FAST if dtype == "bf16" else PRECISE) + PRECISE * 30
    g = a + (u if act != "none" else 0.0)                          # of a term of the products
    for got, r, m, n, what in ((dx, want[0], mag[0], N, "dx"), (dw, want[1], mag[1], M, "dw")):
        close(f64(got), r, product_error(n, m, dtype) + g * m + u * np.abs(r) + TINY, what)
    if bias:
        close(f64(db), want[2], ((M + 4) * U32 + a) * mag[2] + U32 * np.abs(want[2]) + TINY, "db")
    else:
        assert db is None


def test_linear_backward_against_differences(vla):
    """d/dt of sum(c act(x(t) w(t)^T + b(t))) by central differences of the float64 formula."""
    gen = generator(11)
    M, N, K, t = 9, 20, 14, 1e-5
    x, w, b, c = rand(gen, M, K), rand(gen, N, K), rand(gen, N), rand(gen, M, N)
    for act in ("silu", "gelu"):
        pre = torch.empty(M, N, device="cuda")
        vla.linear(x, w, b, act=act, pre=pre)
        got = vla.linear_backward(c, x, w, pre, act=act)
        for i, of in enumerate((x, w, b)):
            way = f64(rand(gen, *of.shape))
            args = [f64(x), f64(w), f64(b)]
            value = []
            for sign in (1, -1):
                moved = list(args)
                moved[i] = args[i] + sign * t * way
                value.append((ref.linear(moved[0], moved[1], moved[2], None, act)[0] * f64(c)).sum())
            slope = (value[0] - value[1]) / (2 * t)
            terms = np.abs(f64(got[i]) * way).sum()
            assert abs((f64(got[i]) * way).sum() - slope) <= 1e-4 * terms


def test_linear_backward_computes_only_what_is_asked_for(vla):
    gen = generator(2)
    dy, x, w = (rand(gen, *s, dtype=torch.bfloat16) for s in ((40, 24), (40, 16), (24, 16)))
    whole = vla.linear_backward(dy, x, w)
    for i, ask in enumerate(("input", "weight", "bias")):
        part = vla.linear_backward(dy, x, w, **{a: a == ask for a in ("input", "weight", "bias")})
        assert [p is None for p in part] == [j != i for j in range(3)] and torch.equal(part[i], whole[i])
    into = tuple(torch.full_like(t, 7) for t in whole)
    back = vla.linear_backward(dy, x, w, None, *into)
    assert all(b is o and torch.equal(o, t) for b, o, t in zip(back, into, whole))


def test_linear_backward_without_terms_is_zero(vla):
    e = lambda *s: torch.empty(*s, device="cuda")   # noqa: E731
    dx, dw, db = vla.linear_backward(e(0, 5), e(0, 4), torch.ones(5, 4, device="cuda"), e(0, 5), act="gelu")
    assert dx.shape == (0, 4) and not dw.any() and dw.shape == (5, 4) and not db.any()
    dx, dw, db = vla.linear_backward(e(3, 0), torch.ones(3, 4, device="cuda"), e(0, 4))
    assert dx.shape == (3, 4) and not dx.any() and dw.shape == (0, 4) and db.shape == (0,)
    dx, dw, db = vla.linear_backward(torch.ones(3, 5, device="cuda"), e(3, 0), e(5, 0))
    assert dx.shape == (3, 0) and dw.shape == (5, 0) and torch.equal(db, torch.full((5,), 3.0, device="cuda"))


# ---------------------------------------------------------------------------------------------
# layer norm

NORM = [  # rows, D, dtype, residual, bias, gap
    (1, 1, "f32", "", True, 0),
    (1, 8, "bf16", "f32", True, 0),
    (3, 31, "f32", "f32", False, 1),
    (5, 64, "bf16", "", True, 0),
    (24, 5120, "bf16", "f32", True, 0),
    (7, 1001, "f32", "", True, 3),
    (33, 1001, "bf16", "bf16", True, 2),
    (300, 4096, "bf16", "bf16", True, 0),
    (41, 520, "f32", "bf16", False, 8),
    (2000, 264, "bf16", "f32", True, 24),
    (4, 8192, "bf16", "bf16", True, 0),
    (4, 8200, "f32", "f32", True, 0),
    (3, 16384, "bf16", "f32", True, 0),
    (3, 16385, "bf16", "", True, 0),
    (2, 32768, "f32", "f32", True, 0),
    (2, 32767, "bf16", "bf16", True, 0),
    (1000, 33, "bf16", "f32", True, 0),
]
# a row's sum: at most 128 values one after another, then two rounds of five pairs
CHAIN = 140


@pytest.mark.parametrize("rows,D,dtype,residual,bias,gap", NORM)
def test_layer_norm_matches_the_reference(vla, rows, D, dtype, residual, bias, gap):
    gen, dt = generator(rows + D), TYPES[dtype]
    x = rows_of(gen, rows, D, gap, dt)
    w, b = rand(gen, D), rand(gen, D) if bias else None
    res = (rows_of(gen, rows, D, gap, TYPES[residual]) * 3 + 1).to(TYPES[residual]) if residual else None
    want, r, mean, rstd = ref.layer_norm(f64(x), f64(w), f64(b), f64(res))
    y, stats = vla.layer_norm(x, w, b, res, stats=True)
    A = np.abs(r).mean(1)
    mean_off = CHAIN * U32 * A + U32 * np.abs(mean)
    close(f64(stats)[:, 0], mean, mean_off + TINY, "mean")
    # r - mean is off by its rounding and the mean's; rstd by half the relative error of the variance
    std = 1 / rstd
    rstd_off = (CHAIN + 8) * U32 + 2 * (mean_off + U32 * np.abs(r).max(1)) / std
    close(f64(stats)[:, 1], rstd, rstd_off * rstd + TINY, "rstd")
    h = np.abs(r - mean[:, None]) * rstd[:, None]
    off = ((mean_off[:, None] + 2 * U32 * np.abs(r)) * rstd[:, None] + h * (rstd_off[:, None] + 4 * U32)) * np.abs(f64(w))
    u = U16 if dtype == "bf16" else U32
    close(f64(y), want, off + U32 * np.abs(want) + u * np.abs(want) + TINY, "y")
    if residual:
        u = U16 if residual == "bf16" else U32
        close(f64(res), r, (u + U32) * np.abs(r) + TINY, "residual")


def test_layer_norm_far_from_zero(vla):
    """A mean of a thousand deviations: what is left is the inputs' own rounding."""
    gen = generator(9)
    x = 1000 + rand(gen, 20, 4096)
    y = vla.layer_norm(x, torch.ones(4096, device="cuda"))
    want = ref.layer_norm(f64(x), 1.0)[0]
    # the mean's error and the differences' rounding, of 1000
    assert np.max(np.abs(f64(y) - want)) <= (16 + 2) * U32 * 1000 + 2.0 ** -20 * np.abs(want).max()


def test_layer_norm_keeps_nan_and_infinity_to_their_rows(vla):
    gen = generator(4)
    x, w = rand(gen, 9, 520), rand(gen, 520)
    clean = vla.layer_norm(x, w)
    x[3, 7], x[6, 519] = float("nan"), float("inf")
    y = vla.layer_norm(x, w)
    good = [i for i in range(9) if i not in (3, 6)]
    assert y[[3, 6]].isnan().all() and torch.equal(y[good], clean[good])


NORM_BACK = [  # rows, D, dy, x, joined, bias, gap
    (1, 1, "f32", "f32", True, True, 0),
    (1, 8, "bf16", "f32", True, True, 0),
    (3, 31, "f32", "f32", False, False, 1),
    (40, 64, "bf16", "bf16", True, True, 0),
    (24, 5120, "bf16", "f32", True, True, 0),
    (7, 1001, "f32", "f32", True, True, 3),
    (300, 1001, "bf16", "bf16", False, True, 2),
    (600, 4096, "bf16", "bf16", True, True, 0),
    (41, 520, "f32", "bf16", False, True, 8),
    (2000, 264, "bf16", "f32", True, True, 24),
    (500, 8192, "bf16", "bf16", True, True, 0),
    (330, 8192, "f32", "f32", True, True, 0),
    (5, 8200, "bf16", "bf16", True, True, 0),
    (3, 16385, "bf16", "f32", True, True, 0),
    (2, 32768, "f32", "f32", True, True, 0),
    (5000, 33, "bf16", "bf16", True, True, 0),
    (3000, 128, "f32", "f32", True, True, 0),
]


@pytest.mark.parametrize("rows,D,dyt,xt,joined,bias,gap", NORM_BACK)
def test_layer_norm_backward_matches_the_reference(vla, rows, D, dyt, xt, joined, bias, gap):
    gen = generator(rows + D)
    dy, x = rows_of(gen, rows, D, gap, TYPES[dyt]), (rows_of(gen, rows, D, gap, TYPES[xt]) * 2 + 1).to(TYPES[xt])
    dres = rows_of(gen, rows, D, gap, TYPES[xt]) if joined else None
    w = rand(gen, D)
    _, _, mean, rstd = ref.layer_norm(f64(x), f64(w))
    stats = torch.tensor(np.stack([mean, rstd], 1), dtype=torch.float32, device="cuda")
    mean, rstd = f64(stats).T
    dx, dw, db = vla.layer_norm_backward(dy, x, w, stats, dres, bias=bias)
    want, mag = ref.layer_norm_backward(f64(dy), f64(x), f64(w), mean, rstd, f64(dres))
    # h is off by the rounding of x - mean, of magnitudes up to |x| + |mean|, times rstd
    far = (np.abs(f64(x)) + np.abs(mean[:, None])) * rstd[:, None]
    u = U16 if xt == "bf16" else U32
    a = np.abs(f64(dy) * f64(w))
    h_off = 2 * U32 * far
    h_share = rstd[:, None] * (h_off * (a * 1.0).mean(1, keepdims=True) * np.max(far, 1, keepdims=True) + far * (a * h_off).mean(1, keepdims=True))
    close(f64(dx), want[0], (CHAIN + 10) * U32 * mag[0] + h_share + u * np.abs(want[0]) + TINY, "dx")
    dw_off = (np.abs(f64(dy)) * h_off).sum(0)
    close(f64(dw), want[1], (rows + 6) * U32 * mag[1] + dw_off + TINY, "dw")
    if bias:
        close(f64(db), want[2], (rows + 2) * U32 * mag[2] + TINY, "db")
    else:
        assert db is None


def test_layer_norm_backward_against_differences(vla):
    gen = generator(21)
    rows, D, t = 6, 40, 1e-5
    x, w, b, c = rand(gen, rows, D), rand(gen, D), rand(gen, D), rand(gen, rows, D)
    y, stats = vla.layer_norm(x, w, b, stats=True)
    got = vla.layer_norm_backward(c, x, w, stats)
    for i, of in enumerate((x, w, b)):
        way = f64(rand(gen, *of.shape))
        value = []
        for sign in (1, -1):
            moved = [f64(x), f64(w), f64(b)]
            moved[i] = moved[i] + sign * t * way
            value.append((ref.layer_norm(*moved)[0] * f64(c)).sum())
        slope = (value[0] - value[1]) / (2 * t)
        assert abs((f64(got[i]) * way).sum() - slope) <= 1e-4 * np.abs(f64(got[i]) * way).sum()


def test_layer_norm_without_rows(vla):
    e = lambda *s: torch.empty(*s, device="cuda")   # noqa: E731
    w = torch.ones(16, device="cuda")
    y, stats = vla.layer_norm(e(0, 16), w, stats=True)
    assert y.shape == (0, 16) and stats.shape == (0, 2)
    dx, dw, db = vla.layer_norm_backward(e(0, 16), e(0, 16), w, e(0, 2))
    assert dx.shape == (0, 16) and not dw.any() and not db.any()


# ---------------------------------------------------------------------------------------------
# together

def block(vla, x, stream, p, dtype):
    """norm -> product, gelu -> product into the residual stream; returns what a gradient needs."""
    h, stats = vla.layer_norm(x, p["nw"], p["nb"], stream, stats=True)
    pre = torch.empty(*x.shape[:-1], p["w1"].shape[0], dtype=dtype, device="cuda")
    a = vla.linear(h, p["w1"], p["b1"], act="gelu", pre=pre)
    return vla.linear(a, p["w2"], p["b2"], stream if stream.dtype == dtype else None), (h, stats, pre, a)


def block_back(vla, dy, stream, p, kept):
    h, stats, pre, a = kept
    da, dw2, db2 = vla.linear_backward(dy, a, p["w2"])
    dh, dw1, db1 = vla.linear_backward(da, h, p["w1"], pre, act="gelu")
    dx, dnw, dnb = vla.layer_norm_backward(dh, stream, p["nw"], stats, dy)
    return dx, dnw, dnb, dw1, db1, dw2, db2


def parameters(gen, D, F, dtype):
    return dict(nw=1 + 0.1 * rand(gen, D), nb=0.1 * rand(gen, D), b1=0.1 * rand(gen, F), b2=0.1 * rand(gen, D),
                w1=(rand(gen, F, D) / D ** 0.5).to(dtype), w2=(rand(gen, D, F) / F ** 0.5).to(dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_feed_forward_block_and_its_gradients(vla, dtype):
    """Forward and backward of a whole block against autograd in 64 bits."""
    gen, dt = generator(8), TYPES[dtype]
    M, D, F = 200, 264, 1032
    p = parameters(gen, D, F, dt)
    x, stream, dy = rand(gen, M, D, dtype=dt), rand(gen, M, D, dtype=dt), rand(gen, M, D, dtype=dt)
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    r = (x.double() + stream.double()).requires_grad_()
    n = (r - r.mean(1, keepdim=True)) * torch.rsqrt(r.var(1, unbiased=False, keepdim=True) + 1e-5) * q["nw"] + q["nb"]
    v = n @ q["w1"].t() + q["b1"]
    y = (0.5 * v * torch.special.erfc(-v / 2 ** 0.5)) @ q["w2"].t() + q["b2"] + r
    want = torch.autograd.grad(y, [r, *(q[k] for k in ("nw", "nb", "w1", "b1", "w2", "b2"))], dy.double())
    got_y, kept = block(vla, x, stream, p, dt)
    got = block_back(vla, dy, stream, p, kept)
    # bfloat16: h, pre, a, da, dh and the residual are rounded on the way, each by up to 2^-8 of itself and mostly
    # independently; six of them add up to less than 6 x 2^-8 of the norm.  float32: 2^-20.
    tol = 6 * U16 if dtype == "bf16" else 2.0 ** -19
    for g, w in zip((got_y, *got), (y, *want)):
        assert float((g.double() - w.detach()).norm() / w.detach().norm()) <= tol


def test_a_block_captured_in_a_graph_on_another_stream(vla):
    gen = generator(12)
    M, D, F = 96, 256, 512
    p = parameters(gen, D, F, torch.bfloat16)
    x0, s0 = rand(gen, M, D, dtype=torch.bfloat16), rand(gen, M, D, dtype=torch.bfloat16)
    dy = rand(gen, M, D, dtype=torch.bfloat16)

    def step(x, stream):
        y, kept = block(vla, x, stream, p, torch.bfloat16)
        return y, *block_back(vla, dy, stream, p, kept)

    want = step(x0, s0.clone())
    x, stream = x0.clone(), s0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step(x, stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, stream)
    for seed in (1, 2):
        x.copy_(rand(generator(seed), M, D))
        stream.copy_(s0)
        graph.replay()
        again = step(x.clone(), s0.clone())
        assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_two_streams_at_once(vla):
    """Workspaces belong to the call: two streams' products do not meet."""
    gen = generator(31)
    w = rand(gen, 333, 1001)
    xs = [rand(gen, 400, 1001) for _ in range(2)]
    want = [vla.linear(x, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(20):
        for x, s, g in zip(xs, streams, got):
            g.append(vla.linear(x, w, stream=s))
    torch.cuda.synchronize()
    for g, y in zip(got, want):
        assert all(torch.equal(a, y) for a in g)


def test_the_norms_codes_go_into_the_product(vla):
    gen = generator(6)
    x, w = rand(gen, 50, 512, dtype=torch.bfloat16), rand(gen, 96, 512) / 512 ** 0.5
    codes, scale = vla.rms_norm(x, torch.ones(512, device="cuda"), out="e4m3")
    ws = w.abs().amax(1) / 448
    wq = (w / ws[:, None]).to(torch.float8_e4m3fn)
    y = vla.linear(codes, wq, x_scale=scale, w_scale=ws)
    want, v, mag = ref.linear(f64(codes), f64(wq), None, None, "none", f64(scale), f64(ws))
    assert y.dtype == torch.bfloat16
    close(f64(y), want, product_error(512, mag, "e4m3") + U16 * np.abs(want) + TINY, "y")


def test_outputs_without_torchs_short_way_to_its_allocator(vla, monkeypatch):
    """Where torch lacks it, outputs come from torch.empty: the same results."""
    gen = generator(41)
    x, w, b = rand(gen, 33, 136), rand(gen, 24, 136), rand(gen, 24)
    calls = lambda: [vla.linear(x, w, b), *vla.linear_backward(x[:, :24].contiguous(), x, w),   # noqa: E731
                     *vla.layer_norm(x, x[0].contiguous(), stats=True)]
    want = calls()
    lib = vla.load_library()
    with monkeypatch.context() as m:
        m.delattr(torch._C, "_cuda_getDevice")
        vla.layer.declare(lib)
        got = calls()
    vla.layer.declare(lib)
    for a, b in ((got, want), (calls(), want)):
        assert all(torch.equal(p, q) and p.stride() == q.stride() for p, q in zip(a, b))


# ---------------------------------------------------------------------------------------------
# refusals

def test_refusals(vla):
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
    b16 = torch.bfloat16
    x, w = z(4, 8), z(6, 8)
    bad = [
        (lambda: vla.linear(x, z(6, 9)), "w has shape"),
        (lambda: vla.linear(x, z(6, 8, dtype=b16)), "w has dtype"),
        (lambda: vla.linear(x.half(), w.half()), "float32, bfloat16 or"),
        (lambda: vla.linear(x, w, z(7)), "bias has shape"),
        (lambda: vla.linear(x, w, z(6, dtype=b16)), "bias has dtype"),
        (lambda: vla.linear(x, w, None, z(4, 5)), "residual has shape"),
        (lambda: vla.linear(x, w, None, z(4, 6, dtype=b16)), "residual has dtype"),
        (lambda: vla.linear(x, w, None, None, z(4, 6, dtype=b16)), "y has dtype"),
        (lambda: vla.linear(x, w, act="relu"), "act must be"),
        (lambda: vla.linear(x, w, dtype=torch.float16), "dtype must be"),
        (lambda: vla.linear(x, w, pre=z(4, 7)), "pre has shape"),
        (lambda: vla.linear(z(8, 4).t(), w), "adjacent"),
        (lambda: vla.linear(z(4, 4, 8)[:, ::3], w), "evenly"),
        (lambda: vla.linear(x, w.cpu()), "not on a CUDA device"),
        (lambda: vla.linear_backward(z(4, 6), x, w, act="gelu"), "pre is needed"),
        (lambda: vla.linear_backward(z(4, 7), x, w), "dy has shape"),
        (lambda: vla.linear_backward(z(5, 6), x, w), "x has shape"),
        (lambda: vla.linear_backward(z(4, 6, dtype=b16), x, w), "x has dtype"),
        (lambda: vla.linear_backward(z(4, 6), x, w, None, z(4, 9)), "dx has shape"),
        (lambda: vla.layer_norm(x, z(9)), "w has shape"),
        (lambda: vla.layer_norm(x, z(8), z(8, dtype=b16)), "b has dtype"),
        (lambda: vla.layer_norm(x, z(8), None, z(4, 9)), "residual has shape"),
        (lambda: vla.layer_norm(x, z(8), stats=z(4, 3)), "stats has shape"),
        (lambda: vla.layer_norm_backward(x, x, z(8), z(3, 2)), "stats has shape"),
        (lambda: vla.layer_norm_backward(x, x, z(8), z(4, 2), z(4, 8, dtype=b16)), "dresidual has dtype"),
    ]
    for call, text in bad:
        with pytest.raises(ValueError, match=text):
            call()
    refused = [
        (lambda: vla.linear(x, w, x_scale=z(4)), "scales go with e4m3"),
        (lambda: vla.linear(x, w, dtype=b16), "float32 operands"),
        (lambda: vla.linear(x, w, None, None, z(1, 6).expand(4, 6)), "overlap"),
        (lambda: vla.linear_backward(z(4, 6), x, w, None, z(1, 8).expand(4, 8)), "overlap"),
        (lambda: vla.layer_norm(x, z(8), eps=-1.0), "eps"),
        (lambda: vla.layer_norm(x, z(8), eps=float("nan")), "eps"),
        (lambda: vla.layer_norm(z(1, 32769), z(32769)), "32768"),
        (lambda: vla.layer_norm(x, z(8), None, z(1, 8).expand(4, 8)), "overlap"),
        (lambda: vla.layer_norm_backward(x, x, z(8), z(4, 2), None, z(1, 8).expand(4, 8)), "overlap"),
        (lambda: vla.layer_norm_backward(z(1, 32769), z(1, 32769), z(32769), z(1, 2)), "32768"),
    ]
    for call, text in refused:
        with pytest.raises(vla.VlaError, match=text):
            call()
    assert vla.default_handle().status()["flags"] == 0


@pytest.mark.parametrize("M,N,K", [(20, 4096, 2051), (300, 333, 200), (700, 130, 2048), (2000, 520, 77)])
def test_workspaces_on_16_byte_boundaries(vla, M, N, K):
    """A workspace of just the size asked for, 16 bytes off a 32-byte boundary: nothing behind it is touched."""
    import ctypes
    h, gen = vla.default_handle(), generator(M)
    x, w, dy = rand(gen, M, K), rand(gen, N, K), rand(gen, M, N)
    size, ptr = ctypes.c_size_t(), lambda t: None if t is None else t.data_ptr()   # noqa: E731

    def guarded(call):
        room = torch.full((size.value + 16 + 4096,), 7, dtype=torch.uint8, device="cuda")
        assert room.data_ptr() % 32 == 0
        torch.cuda.synchronize()
        assert call(room.data_ptr() + 16) == 0
        torch.cuda.synchronize()
        assert (room[:16] == 7).all() and (room[16 + size.value:] == 7).all()

    y = torch.empty(M, N, device="cuda")
    rows = (ctypes.c_longlong * 5)(K, K, 0, 0, N)
    assert h.lib.vla_linear_workspace(h.ptr, ptr(x), ptr(w), M, N, K, rows, 0, 0, ctypes.byref(size)) == 0 and size.value
    guarded(lambda ws: h.lib.vla_linear(h.ptr, ptr(x), ptr(w), *(None,) * 5, ptr(y), M, N, K, rows, 0, 0, 0, ws, size, None))
    assert torch.equal(y, vla.linear(x, w))
    pre, dx, dw, db = rand(gen, M, N), torch.empty(M, K, device="cuda"), torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    rows = (ctypes.c_longlong * 6)(N, K, K, N, K, K)
    assert h.lib.vla_linear_backward_workspace(h.ptr, ptr(dy), ptr(x), ptr(w), 1, 1, 1, M, N, K, rows, 2, 0, ctypes.byref(size)) == 0
    guarded(lambda ws: h.lib.vla_linear_backward(h.ptr, ptr(dy), ptr(x), ptr(w), ptr(pre), ptr(dx), ptr(dw), ptr(db), M, N, K, rows,
                                                 2, 0, ws, size, None))
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), vla.linear_backward(dy, x, w, pre, act="gelu")))
    stats = torch.stack([x.mean(1), torch.rsqrt(x.var(1, unbiased=False) + 1e-5)], 1).contiguous()
    nw, dn, dnw, dnb = rand(gen, K), torch.empty_like(x), torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
    assert h.lib.vla_layer_norm_backward_workspace(h.ptr, M, K, ctypes.byref(size)) == 0
    strides = (ctypes.c_longlong * 4)(K, K, 0, K)
    guarded(lambda ws: h.lib.vla_layer_norm_backward(h.ptr, ptr(x), ptr(x), ptr(nw), ptr(stats), None, ptr(dn), ptr(dnw), ptr(dnb), M, K,
                                                     strides, 0, 0, ws, size, None))
    assert all(torch.equal(a, b) for a, b in zip((dn, dnw, dnb), vla.layer_norm_backward(x, x, nw, stats)))


def test_c_refusals(vla):
    """Pointers and workspaces that the binding never passes."""
    import ctypes
    h = vla.default_handle()
    x, w, y = torch.zeros(300, 333, device="cuda"), torch.zeros(40, 333, device="cuda"), torch.zeros(300, 40, device="cuda")
    rows = (ctypes.c_longlong * 5)(333, 333, 0, 0, 40)
    size = ctypes.c_size_t()
    args = (300, 40, 333, rows)
    assert h.lib.vla_linear_workspace(h.ptr, x.data_ptr(), w.data_ptr(), *args, 0, 0, ctypes.byref(size)) == 0
    call = lambda x, ws, n, act=0, kind=0: h.lib.vla_linear(   # noqa: E731
        h.ptr, x, w.data_ptr(), None, None, None, None, None, y.data_ptr(), *args, act, kind, 0, ws, n, None)
    assert call(x.data_ptr() + 2, None, 0) == 1
    assert call(None, None, 0) == 1
    assert call(x.data_ptr(), None, 0, act=3) == 1
    assert call(x.data_ptr(), None, 0, kind=3) == 1
    if size.value:
        ws = torch.zeros(size.value + 16, dtype=torch.uint8, device="cuda")
        assert call(x.data_ptr(), None, size.value) == 1
        assert call(x.data_ptr(), ws.data_ptr(), size.value - 1) == 1
        assert call(x.data_ptr(), ws.data_ptr() + 8, size.value) == 1
    need = size.value   # without addresses a query may say more, never less
    assert h.lib.vla_linear_workspace(h.ptr, None, None, *args, 0, 0, ctypes.byref(size)) == 0 and size.value >= need > 0
    rows[0] = -1
    assert call(x.data_ptr(), None, 0) == 1
    assert h.lib.vla_linear(h.ptr, x.data_ptr(), w.data_ptr(), *(None,) * 5, y.data_ptr(), 2 ** 31, 40, 333, rows, 0, 0, 0, None, 0, None) == 1
    assert b"2^30" in h.lib.vla_last_error(h.ptr)
    assert h.lib.vla_linear(h.ptr, x.data_ptr(), w.data_ptr(), *(None,) * 5, y.data_ptr(), -1, 40, 333, rows, 0, 0, 0, None, 0, None) == 1
    assert h.lib.vla_layer_norm(h.ptr, x.data_ptr(), *(None,) * 3, y.data_ptr(), None, 4, 8, 8, 0, 8, 1e-5, 0, 0, None) == 1   # no w
    assert h.lib.vla_layer_norm_backward(h.ptr, *(x.data_ptr(),) * 4, None, y.data_ptr(), x.data_ptr(), None, 4, 8,
                                         (ctypes.c_longlong * 4)(8, 8, 0, 8), 0, 0, None, 0, None) == 1                     # no workspace
