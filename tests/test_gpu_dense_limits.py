"""Products and norms where they end early, at the ends of their ranges, and form by form."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import dense_ref as ref

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def vla():
    from _util import ensure_built
    ensure_built()
    import sherman_morrison_inverse_gb300 as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def launches(call):
    """What a call launches, from a graph captured of it: the kernels' names in order, and whether each may start before what
    lies before it on the stream is done."""
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    cu, graph = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(g.raw_cuda_graph())

    class Params(ctypes.Structure):   # CUDA_KERNEL_NODE_PARAMS
        _fields_ = [("func", ctypes.c_void_p), ("sizes", ctypes.c_uint * 7), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                    ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]

    class Edge(ctypes.Structure):     # CUgraphEdgeData
        _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte), ("rest", ctypes.c_ubyte * 5)]

    n = ctypes.c_size_t()
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    names = {}
    for node in nodes:
        kind, p, text = ctypes.c_int(), Params(), ctypes.c_char_p()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            if p.func:
                assert cu.cuFuncGetName(ctypes.byref(text), ctypes.c_void_p(p.func)) == 0
            else:
                assert cu.cuKernelGetName(ctypes.byref(text), ctypes.c_void_p(p.kern)) == 0
            names[node] = text.value.decode()
        else:
            names[node] = "no kernel"
    assert cu.cuGraphGetEdges_v2(graph, None, None, None, ctypes.byref(n)) == 0
    a, b, edges = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (Edge * n.value)()
    assert n.value == 0 or cu.cuGraphGetEdges_v2(graph, a, b, edges, ctypes.byref(n)) == 0
    before = {y: (x, e.type) for x, y, e in zip(a, b, edges)}
    order = [m for m in nodes if m not in before]
    assert len(order) == (1 if len(nodes) else 0) and len(before) == len(nodes) - len(order)   # one stream: a chain
    after = {x: y for y, (x, _) in before.items()}
    while order and order[-1] in after:
        order.append(after[order[-1]])
    return [(names[m], m in before and before[m][1] == 1) for m in order]


# ---------------------------------------------------------------------------------------------
# waits that run out

PRODUCTS = [  # M, N, K, dtype, gradient
    (20, 300, 2048, "bf16", False),       # few weights: CUDA cores, where nothing is waited for
    (20, 2000, 2048, "bf16", False),      # w's rows in the long dimension, shares over a cluster
    (128, 8192, 2048, "f32", False),
    (100, 1000, 4096, "e4m3", False),
    (1000, 2000, 2048, "bf16", False),    # CTA pairs
    (700, 130, 4096, "f32", False),       # parts of Kd, joined
    (2000, 2048, 1024, "e4m3", False),
    (300, 520, 264, "f32", True),
    (4096, 1024, 2048, "bf16", True),
]


@pytest.mark.parametrize("M,N,K,dtype,gradient", PRODUCTS)
def test_a_products_wait_that_runs_out_ends_the_call(vla, M, N, K, dtype, gradient):
    """Without time to wait every tensor-core product gives up before its sums are there, with copies and products under
    way: the call ends with its status, and the next ones are right."""
    gen, h = generator(M), vla.Handle(0)
    flags = vla.STATUS_TIMEOUT if gradient or N * K > 2 ** 21 // 3 or dtype == "f32" else 0
    x, w = rand(gen, M, K, dtype=TYPES[dtype]), rand(gen, N, K, dtype=TYPES[dtype])
    dy = rand(gen, M, N, dtype=TYPES[dtype]) if gradient else None

    def call():
        return h.linear_backward(dy, x, w) if gradient else [h.linear(x, w)]

    want = call()
    assert h.status()["flags"] == 0
    for _ in range(3):
        h.wait_limit(0)
        for _ in range(5):
            call()
            assert h.status()["flags"] == flags
        h.wait_limit(2000)
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(call(), want))
        assert h.status()["flags"] == 0
    h.close()


@pytest.mark.parametrize("rows,D,dtype,flagged", [(4096, 4096, "bf16", True), (3000, 128, "f32", True), (330, 8192, "f32", True),
                                                  (2, 264, "bf16", True), (300, 1001, "f32", False), (5, 8200, "bf16", False)])
def test_a_norms_wait_that_runs_out_ends_the_call(vla, rows, D, dtype, flagged):
    """The same for the norm's gradient: rows that are copied ahead are waited for, others are read directly."""
    gen, h = generator(rows), vla.Handle(0)
    dy, x, res = (rand(gen, rows, D, dtype=TYPES[dtype]) for _ in range(3))
    w = rand(gen, D)
    _, stats = h.layer_norm(x, w, stats=True)
    want = h.layer_norm_backward(dy, x, w, stats, res)
    assert h.status()["flags"] == 0
    for _ in range(3):
        h.wait_limit(0)
        for _ in range(5):
            h.layer_norm_backward(dy, x, w, stats, res)
            assert h.status()["flags"] == (vla.STATUS_TIMEOUT if flagged else 0)
        h.wait_limit(2000)
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(h.layer_norm_backward(dy, x, w, stats, res), want))
        assert h.status()["flags"] == 0
    h.close()


def test_calls_that_give_up_leave_others_alone(vla):
    """Calls that give up on one stream, with copies under way into shared memory that the next block gets, beside calls on another
    stream whose results are known."""
    gen, quick, h = generator(1), vla.Handle(0), vla.Handle(0)
    quick.wait_limit(0)
    a, aw = rand(gen, 1000, 2048, dtype=torch.bfloat16), rand(gen, 2000, 2048, dtype=torch.bfloat16)
    n, nw, stats = rand(gen, 3000, 4096, dtype=torch.bfloat16), rand(gen, 4096), rand(gen, 3000, 2).abs()
    x, w, dy = rand(gen, 700, 1032, dtype=torch.bfloat16), rand(gen, 1000, 1032, dtype=torch.bfloat16), rand(gen, 700, 1000, dtype=torch.bfloat16)
    few, codes, wc = x[:40], x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)

    def right():
        y, st = h.layer_norm(x, nw[:1032].contiguous(), stats=True)
        return [h.linear(x, w), h.linear(few, w), h.linear(x.float(), w.float()), h.linear(codes, wc), y, *h.linear_backward(dy, x, w),
                *h.layer_norm_backward(x, x, nw[:1032].contiguous(), st)]

    want, got = right(), []
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(30):
        with torch.cuda.stream(sides[0]):
            for _ in range(3):
                quick.linear(a, aw)
                quick.linear(a[:100], aw)
                quick.linear_backward(n[:1000, :2000], a, aw)
                quick.layer_norm_backward(n, n, nw, stats)
        with torch.cuda.stream(sides[1]):
            got.append(right())
    torch.cuda.synchronize()
    for outs in got:
        assert all(torch.equal(p, q) for p, q in zip(outs, want))
    assert quick.status()["flags"] == vla.STATUS_TIMEOUT and h.status()["flags"] == 0
    quick.close()
    h.close()


def test_the_wait_limit_has_a_range(vla):
    h = vla.Handle(0)
    with pytest.raises(vla.VlaError, match="0..5000"):
        h.wait_limit(5001)
    h.close()


# ---------------------------------------------------------------------------------------------
# rows far from zero

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [264, 1001, 4096, 8191, 8200])
def test_layer_norm_backward_far_from_zero(vla, D, dtype):
    """A mean of a thousand deviations.  x - mean is exact there (both within a factor of two of one another), so h is off
    by two roundings of itself, whatever the mean; dy follows h, so that the rows' mean of a h counts."""
    gen, rows = generator(D), 4
    x, w = 1000 + rand(gen, rows, D), 1 + 0.2 * rand(gen, D)
    dy = (x - 1000 + 0.1 * rand(gen, rows, D)).to(TYPES[dtype])
    _, _, mean, rstd = ref.layer_norm(f64(x), f64(w))
    stats = torch.tensor(np.stack([mean, rstd], 1), dtype=torch.float32, device="cuda")
    mean, rstd = f64(stats).T
    got = vla.layer_norm_backward(dy, x, w, stats)
    want, mag = ref.layer_norm_backward(f64(dy), f64(x), f64(w), mean, rstd)
    # sums over a row: chains of at most 140 additions (128 values, or 16 pairs and ten folds); over the rows: four
    for g, r, m, n, what in zip(got, want, mag, (150, rows + 8, rows + 2), ("dx", "dw", "db")):
        worst = np.max(np.abs(f64(g) - r) / (n * U32 * m))
        assert worst <= 1.0, f"{what}: {worst:.3g} times its bound"


# ---------------------------------------------------------------------------------------------
# long sums

def same_sign(gen, rows, cols, along, dtype):
    """[rows, cols] of positive values in `dtype`, every row (along 1) or column (0) with a size of its own; its sums over the other
    dimension in 64 bits."""
    size = 1 + torch.rand(rows if along else cols, generator=gen, device="cuda")
    x, total = torch.empty(rows, cols, dtype=dtype, device="cuda"), []
    for i in range(0, rows, 4096):
        part = 0.5 + torch.rand(min(4096, rows - i), cols, generator=gen, device="cuda")
        x[i:i + 4096] = part * (size[i:i + 4096, None] if along else size)
        total.append(x[i:i + 4096].double().sum(along))
    return x, torch.cat(total) if along else sum(total)


# Terms of one sign, whose sums a tensor core cuts off towards zero: two units of 2^-23 of the running sum an addition at most, four
# additions a stage.  A chain of 64 stages, its running sum half of the whole on the mean: 4 x 64 x 2^-23; of up to 128, which is not
# cut into parts, twice that.  Over the parts float32 additions round to the nearest.  The roundings to bfloat16, 2^-8 / sqrt(3) at most
# and of either sign, leave four times that over the square root of the number of distinct outputs, of which there are
# 128 sizes (values of bfloat16 between 1 and 2) times the sums.
def mean_bound(stages, sums):
    return 4 * (64 if stages > 128 else stages) * 2.0 ** -23 + 2.0 ** -22 + 4 * U16 / 3 ** 0.5 / (128 * sums) ** 0.5


@pytest.mark.parametrize("M", [8192, 16384, 262144 + 40, 524288])
def test_weight_gradients_of_many_tokens_keep_their_sums(vla, M):
    """dw sums over the tokens, in one share each of more tiles than there are clusters."""
    gen, N, K = generator(M), 2048, 2432
    x, total = same_sign(gen, M, K, 0, torch.bfloat16)
    dy = (1 + torch.rand(N, generator=gen, device="cuda")).bfloat16()
    _, dw, _ = vla.linear_backward(dy.expand(M, N), x, torch.zeros(N, K, dtype=torch.bfloat16, device="cuda"), input=False, bias=False)
    off = dw.double() / (dy.double()[:, None] * total) - 1
    assert abs(float(off.mean())) <= mean_bound(M / 64, K)
    assert float(off.abs().max()) <= U16 + 4 * 128 * 2.0 ** -22 + M / 4096 * U32


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("K", [8192, 65536 + 72])
def test_products_of_long_rows_keep_their_sums(vla, K, dtype):
    gen, M, N = generator(K), 2048, 2560
    x, total = same_sign(gen, M, K, 1, TYPES[dtype])
    w = (1 + torch.rand(N, generator=gen, device="cuda")).to(TYPES[dtype])
    y = vla.linear(x, w[:, None].expand(N, K).contiguous(), dtype=torch.bfloat16)
    off = y.double() / (total[:, None] * w.double()) - 1
    assert abs(float(off.mean())) <= mean_bound(K / (64 if dtype == "bf16" else 128), M / (16 if dtype == "e4m3" else 1))


def test_a_long_gradient_beside_a_short_one(vla):
    """One launch whose products differ in length: dx sums over few columns, dw over many rows."""
    gen, M, N, K = generator(77), 40000, 1500, 2500
    dy, x, w = (rand(gen, *s, dtype=torch.bfloat16) for s in ((M, N), (M, K), (N, K)))
    dx, dw, db = vla.linear_backward(dy, x, w)
    for got, left, right, stages in ((dw[:100], dy[:, :100].double().t(), x.double(), 64), (dx[-500:], dy[-500:].double(), w.double(), N / 64 + 1)):
        want, mag = left @ right, left.abs() @ right.abs()
        # a part's additions are cut off, each by 2^-22 of its sum of magnitudes at most; parts are rounded to the nearest
        bound = (4 * stages * 2.0 ** -22 + (M / 4096 + 2) * U32) * mag + U16 * want.abs()
        assert bool(((got.double() - want).abs() <= bound).all())
        assert float((got.double() - want).norm() / want.norm()) <= U16 / 3 ** 0.5


# ---------------------------------------------------------------------------------------------
# what a call launches

def test_only_launches_of_one_call_overlap(vla):
    """A call's first launch waits for all that lies before it on the stream, whatever that is; the later ones may start early."""
    gen = generator(5)
    t, e = rand(gen, 100), lambda *s: torch.empty(*s, device="cuda")   # noqa: E731
    x, w, dy = rand(gen, 700, 77), rand(gen, 130, 77), rand(gen, 700, 130)
    calls = [
        (lambda: vla.linear(x, w), True),                                                        # copies, products
        (lambda: vla.linear_backward(dy, x, w), True),                                           # db, copies, products
        (lambda: vla.layer_norm_backward(x, x, t[:77].contiguous(), e(700, 2)), True),           # rows, sums
        (lambda: vla.linear(e(3, 0), e(5, 0)), False),                                           # no terms: nothing but the epilogue
        (lambda: vla.linear_backward(e(0, 5), e(0, 4), w[:5, :4].contiguous(), bias=False), False),
        (lambda: vla.linear_backward(e(3, 0), x[:3, :4].contiguous(), e(0, 4), weight=False), False),
    ]
    for call, several in calls:
        def one():
            t.add_(1)
            call()
        got = launches(one)
        first = [early for name, early in got if "vla" in name or name == "no kernel"][0]
        assert not first and (several == any(early for _, early in got)), got


# ---------------------------------------------------------------------------------------------
# gradients that torch records

def test_products_within_an_autograd_function(vla):
    """Parameters are taken where gradients are not recorded: under no_grad, and in an autograd.Function, whose gradients
    are those of torch."""
    gen = generator(19)
    x, w, b = (rand(gen, *s).requires_grad_() for s in ((30, 72), (40, 72), (40,)))

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            pre = torch.empty(x.shape[0], w.shape[0], device="cuda")
            y = vla.linear(x, w, b, act="silu", pre=pre)
            ctx.save_for_backward(x, w, pre)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, w, pre = ctx.saved_tensors
            return vla.linear_backward(dy.contiguous(), x, w, pre, act="silu")

    with pytest.raises(ValueError, match="x requires a gradient"):
        vla.linear(x, w, b)
    with torch.no_grad():
        assert not vla.linear(x, w, b).requires_grad
    y, dy = Linear.apply(x, w, b), rand(gen, 30, 40)
    got = torch.autograd.grad(y, (x, w, b), dy)
    t = [v.detach().double().requires_grad_() for v in (x, w, b)]
    want = torch.autograd.grad(torch.nn.functional.silu(t[0] @ t[1].t() + t[2]), t, dy.double())
    for g, r in zip(got, want):
        # pre is off by 2^-24 of its 72 terms' magnitudes, some 60 for values of its own size, and the slope follows it;
        # the sums of 30 to 72 terms as much again
        assert float((g.double() - r).norm() / r.norm()) <= 2 * 72 * U32


# ---------------------------------------------------------------------------------------------
# where outputs come from

def test_a_dispatch_mode_sees_the_outputs(vla):
    """A mode that watches torch's dispatcher sees what a call allocates, its workspace among it, as of the other operators."""
    from torch.utils._python_dispatch import TorchDispatchMode

    class Watch(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.made = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if "empty" in str(func):
                self.made.append(out.data_ptr())
            return out

    gen = generator(3)
    x, w, nw = rand(gen, 700, 77), rand(gen, 130, 77), rand(gen, 77)
    want = vla.linear(x, w)
    with Watch() as watch:
        y = vla.linear(x, w)
        h, stats = vla.layer_norm(x, nw, stats=True)
        grads = [*vla.linear_backward(y, x, w), *vla.layer_norm_backward(x, x, nw, stats)]
    assert torch.equal(y, want) and {t.data_ptr() for t in (y, h, stats, *grads)} <= set(watch.made)
    assert len(watch.made) == 9 + 3   # two products' and a norm's workspaces


def test_outputs_that_are_an_input_are_refused(vla):
    """They were read while they were written: with rows wider than 8192 the norm's dw came from dx, a product's y from y."""
    gen = generator(13)
    x, w, r, pre = rand(gen, 64, 64), rand(gen, 64, 64), rand(gen, 64, 64), torch.empty(64, 64, device="cuda")
    wide, nw, stats = rand(gen, 5, 9000), rand(gen, 9000), rand(gen, 5, 2).abs()
    bad = [
        lambda: vla.linear(x, w, y=x), lambda: vla.linear(x, w, y=w), lambda: vla.linear(x, w, y=pre, pre=pre, act="silu"),
        lambda: vla.linear(x, w, pre=x, act="silu"), lambda: vla.linear(x, w, None, r, pre=r, act="silu"),
        lambda: vla.linear_backward(r, x, w, dx=r), lambda: vla.linear_backward(r, x, w, dx=x), lambda: vla.linear_backward(r, x, w, dw=w),
        lambda: vla.linear_backward(r, x, w, dw=x), lambda: vla.linear_backward(r, x, w, dx=pre, dw=pre),
        lambda: vla.linear_backward(r, x, w, pre, act="gelu", dx=pre),
        lambda: vla.layer_norm(x, nw[:64], None, r, r),
        lambda: vla.layer_norm_backward(wide, wide.clone(), nw, stats, dx=wide), lambda: vla.layer_norm_backward(wide.clone(), wide, nw, stats, dx=wide),
    ]
    kept = [t.clone() for t in (x, w, r, wide)]
    for call in bad:
        with pytest.raises(vla.VlaError, match="must not be"):
            call()
    assert all(torch.equal(a, b) for a, b in zip(kept, (x, w, r, wide)))
    vla.linear(x, w, None, r, r)   # the residual as y stays
    e = torch.empty(0, 64, device="cuda")
    assert vla.linear(e, w, y=torch.empty(0, 64, device="cuda")).shape == (0, 64)


# ---------------------------------------------------------------------------------------------
# every form of a product against its reference, float32 above all: which form a call takes is part of the test

FORMS = [  # M, N, K, dtype, out, act, everything (bias, residual, pre in rows with gaps), kernels
    (16, 1000, 2000, "f32", "f32", "silu", True, ["few_rows"]),
    (100, 2000, 1100, "f32", "f32", "gelu", True, ["pack", "tokens"]),
    (30, 8200, 1030, "f32", "f32", "none", False, ["pack", "tokens"]),
    (300, 777, 1161, "f32", "f32", "silu", True, ["pack", "tokens"]),
    (300, 3001, 3000, "f32", "f32", "silu", True, ["pack", "gemm", "join"]),       # more weights than that takes
    (513, 1000, 4000, "f32", "f32", "none", False, ["pack", "gemm", "join"]),      # few tiles, a long Kd
    (700, 141, 4100, "f32", "f32", "gelu", True, ["pack", "gemm", "join"]),
    (1001, 777, 1161, "f32", "f32", "silu", True, ["pack", "gemm", "join"]),
    (6000, 2501, 72, "f32", "f32", "gelu", True, ["pack", "gemm"]),                # rows of y through shared memory
    (6000, 2504, 200, "f32", "f32", "silu", False, ["pack", "gemm"]),              # and directly
    (6000, 2504, 200, "bf16", "f32", "silu", True, ["gemm"]),
    (6000, 2504, 208, "e4m3", "bf16", "gelu", True, ["gemm"]),
    (513, 1000, 8200, "bf16", "bf16", "gelu", True, ["pack", "gemm", "join"]),
]


def forms_of(call):
    names = ("few_rows", "tokens", "gemm", "join", "pack", "slope_sum", "slope")
    return [next(n for n in names if n + "_kernel" in name) for name, _ in launches(call) if "vla" in name]


def gaps(gen, rows, width, everything, dtype):
    return rand(gen, rows, width + 3).to(dtype)[:, 1:1 + width] if everything else rand(gen, rows, width).to(dtype)


@pytest.mark.parametrize("M,N,K,dtype,out,act,everything,forms", FORMS)
def test_products_form_by_form(vla, M, N, K, dtype, out, act, everything, forms):
    gen = generator(M + N + K)
    odd = everything and dtype != "e4m3" and (dtype == "f32" or K == 8200)
    x, w = gaps(gen, M, K, odd, TYPES[dtype]), (gaps(gen, N, K, odd, torch.float32) / K ** 0.5).to(TYPES[dtype])
    b = rand(gen, N) if everything else None
    res, pre = (gaps(gen, M, N, True, TYPES[out]) if everything else None for _ in range(2))
    scales = dict(x_scale=rand(gen, M).abs() + 0.1, w_scale=rand(gen, N).abs() + 0.1) if dtype == "e4m3" else {}
    call = lambda: vla.linear(x, w, b, res, act=act, pre=pre, dtype=TYPES[out], **scales)   # noqa: E731
    assert forms_of(call) == forms
    y = call()
    f = {k: f64(v) for k, v in scales.items()}
    want, v, mag = ref.linear(f64(x), f64(w), None if b is None else f64(b), None if res is None else f64(res), act, f.get("x_scale"), f.get("w_scale"))
    # the sums: K products and their additions, cut off or rounded, and of three terms of bfloat16 what the six products leave
    # out; the activations' own error (of bfloat16 results 2^-19 of their terms, see the slopes below) and slopes, at most 1.13
    u, own = (U16, 2.0 ** -18) if out == "bf16" else (U32, 2.0 ** -20)
    off = (2 * K + 8) * U32 * mag
    av = np.abs(ref.act(v, act))
    bound = 1.2 * off + own * (1 + np.abs(v)) ** 2 * (av + 2.0 ** -20) * (act != "none") + 2 * U32 * (av + np.abs(want)) + u * np.abs(want)
    assert np.max(np.abs(f64(y) - want) / bound) <= 1.0
    if everything:
        assert np.max(np.abs(f64(pre) - v) / (off + u * np.abs(v))) <= 1.0
    if out == "f32" and dtype == "f32":
        # In the 2-norm the terms' errors are independent.  What six of nine products leave out is 2^-24 of each, and a chain of
        # 16 additions that are cut off takes 16 x 2^-24 of its sum at most (half of 2^-23 each, the running sum half of the
        # whole, twice over for terms that are cut off before they are added): 2^-20.  Without one of the six it is 2.4e-6.
        assert np.linalg.norm((f64(pre) if everything else f64(y)) - (v if everything else want)) <= 2.0 ** -20 * np.linalg.norm(v)


@pytest.mark.parametrize("M,N,forms", [(200, 24, ["pack", "tokens"]), (600, 24, ["pack", "gemm"]), (6000, 2504, ["pack", "gemm"])])
def test_float32_terms_of_every_magnitude(vla, M, N, forms):
    """One product a sum, of values from 2^-100 to 2^95: three terms of bfloat16 hold them to 2^-24 each, the six products leave
    3 x 2^-25 out."""
    x = (torch.diag(2.0 ** torch.arange(-100, 100, 5, device="cuda")) * 1.2345678).repeat(M // 40 + 1, 1)[:M].contiguous()
    w = torch.full((N, 40), 1.7654321, device="cuda") * (1 + torch.arange(N, device="cuda") / 9999)[:, None]
    assert forms_of(lambda: vla.linear(x, w)) == forms
    want = f64(x) @ f64(w).T
    assert np.max(np.abs(f64(vla.linear(x, w)) / want - 1)) <= 2.0 ** -22
    # the same values through a gradient: dx = dy w and dw = dy^T x
    dx = vla.linear_backward(x, w[0, 0].expand(M, N).contiguous(), torch.full((40, N), 1.7654321, device="cuda"), bias=False)[0]
    assert np.max(np.abs(f64(dx) / (f64(x) @ np.full((40, N), f64(w)[0, 0])) - 1)) <= 2.0 ** -22
    one = x[:40]
    dw = vla.linear_backward(one, w[0, 0].expand(40, N).contiguous(), torch.zeros(40, N, device="cuda"), input=False, bias=False)[1]
    assert np.max(np.abs(f64(dw) / (f64(one).T @ np.full((40, N), f64(w)[0, 0])) - 1)) <= 2.0 ** -22


@pytest.mark.parametrize("M,N,K,forms", [(700, 300, 520, ["slope", "slope_sum", "pack", "gemm", "join"]),
                                         (6000, 1501, 2003, ["slope", "slope_sum", "pack", "gemm", "join"]),
                                         (7, 300, 200, ["slope", "slope_sum", "pack", "gemm", "join"]),
                                         (3000, 2500, 2600, ["slope", "slope_sum", "pack", "gemm"])])
def test_float32_gradients_in_the_2_norm(vla, M, N, K, forms):
    """The bounds of single values leave room for a whole term; the 2-norm does not (see above)."""
    gen = generator(M + N)
    dy, x, w = rand(gen, M, N), rand(gen, M, K), rand(gen, N, K)
    got = vla.linear_backward(dy, x, w)
    assert forms_of(lambda: vla.linear_backward(dy, x, w)) == forms
    for g, r in zip(got, ref.linear_backward(f64(dy), f64(x), f64(w))[0]):
        assert np.linalg.norm(f64(g) - r) <= 2.0 ** -20 * np.linalg.norm(r)


# ---------------------------------------------------------------------------------------------
# the activations' slopes behind bfloat16, where a bias gradient of one row shows them in float32

@pytest.mark.parametrize("spare", [0, 3])   # eight columns a lane, or one
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_slopes_of_every_bfloat16_value(vla, act, spare):
    """dy = 1, one row: db is act'(pre) itself.  Relative to the slope's two terms.  gelu: the polynomial and its evaluation 6.4e-7, the
    approximate exponential and reciprocal 2^-22 each, and v^2 / 2 rounded twice before the exponential, 2^-24 v^2.  silu: the
    exponential, the reciprocal and the addition between them, 2^-21, and its argument's rounding, |v| 2^-24; 1 - s is off
    by a rounding of s, which v multiplies."""
    v = torch.arange(0x4180, dtype=torch.int16, device="cuda")   # 0 to 16
    v = torch.cat([v, v | -0x8000]).view(torch.bfloat16)
    v = v[:v.numel() // 8 * 8 - spare]
    one = torch.ones(1, v.numel(), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(v.numel(), 1, dtype=torch.bfloat16, device="cuda")
    db = vla.linear_backward(one, one[:, :1], w, v[None], act=act, input=False, weight=False)[2]
    slope, terms = ref.slope(f64(v), act)
    size = np.abs(f64(v))
    bound = (2.0 ** -19 + size ** 2 * U32 if act == "gelu" else 2.0 ** -20 + size * 4 * U32) * terms
    # where an exponential falls below 2^-126 it is 0
    assert np.max(np.abs(f64(db) - slope) / (bound + 16 * 2.0 ** -126)) <= 1.0
