"""The state space layer's operators where their numbers run to the ends of their ranges, against the
float64 references and the bounds of test_gpu_layer.py."""
import math

import numpy as np
import pytest
import torch

from oracle import layer_ref as ref
from test_gpu_layer import TYPES, U16, U32, check_scan, close, f64, generator, rand, scan_inputs, vla  # noqa: F401

pytestmark = pytest.mark.gpu


def set_step(v, head, step):
    """softplus(dt + dt_bias) of a head is (about) `step` at every token."""
    v["dt_bias"][head] = 0
    v["dt"][..., head] = step if step > 20 else math.log(math.expm1(step))


# ---------------------------------------------------------------------------------------------
# scan: decays

RESETS = [  # lens, packed, N, A, an ordinary step, the resetting step, tokens that reset
    ([300], False, 128, -16.0, 0.05, 1e3, (5,)),
    ([300, 300], False, 64, -16.0, 0.05, 1e4, (5, 131)),
    ([300], False, 128, -16.0, 0.05, 1e5, (5, 40, 70, 131, 170)),
    ([300], False, 64, -16.0, 0.05, 1e6, (5, 40, 131)),
    ([300], False, 64, -16.0, 0.01, 1e4, tuple(range(1, 128, 9))),
    ([300], False, 64, -3000.0, 0.01 * 16 / 3000, 30.0, (7, 140)),
    ([200, 333, 64], True, 128, -16.0, 0.05, 1e5, (31, 32, 140, 210, 575)),
    ([2500], False, 64, -1.0, 0.01, 1e6, tuple(range(20, 2500, 77))),
]


@pytest.mark.parametrize("lens,packed,N,A,small,large,at", RESETS)
def test_ssm_scan_after_tokens_that_reset_the_state(vla, lens, packed, N, A, small, large, at):  # noqa: F811
    """A few tokens of enormous steps among ordinary ones: what follows them decays as if they were not
    there.  Their own input is zero, so that it does not hide the others'."""
    def change(v):
        for head in range(2):
            v["A"][head] = A
            set_step(v, head, small)
        for t in at:
            v["dt"][t if packed else (slice(None), t)] = large
            v["x"][t if packed else (slice(None), t)] = 0
    check_scan(vla, generator(N + len(at)), lens, packed, 2, 64, 1, N, "bf16", False, False, change=change)


def test_ssm_scan_of_large_values_under_strong_decay(vla):  # noqa: F811
    """Products C B^T of 1e12 and blocks of 32 tokens that decay by 2^92: every factor's inverse is near the end
    of float32's range, the outputs are not."""
    def change(v):
        v["B"] *= 1e6
        v["C"] *= 1e6
        for head in range(2):
            v["A"][head] = -16.0
            set_step(v, head, 0.125)
    for lens, N in (([200], 128), ([140, 140], 64)):
        check_scan(vla, generator(N), lens, False, 2, 64, 1, N, "bf16", True, False, change=change)


# ---------------------------------------------------------------------------------------------
# norm: tiny rows

@pytest.mark.parametrize("out,group", [("e4m3", 0), ("e4m3", 128), ("int8", 0), ("int8", 128)])
@pytest.mark.parametrize("dtype,rows,D", [("f32", 6, 256), ("bf16", 6, 384), ("f32", 6, 255), ("bf16", 900, 1003), ("f32", 900, 2203)])
def test_rms_norm_codes_of_tiny_rows(vla, dtype, rows, D, out, group):  # noqa: F811
    """Rows near the least normal float32 (1.2e-38), with zeros and both signs: 1 / sqrt(eps) carries them to
    ordinary scales, and their codes are those of larger rows.  Rows with aligned and with odd starts."""
    gen = generator(rows + D)
    size = torch.tensor([2e-38, 1e-37, 1e-36, 3e-36, 1e-35, 1.0], device="cuda").repeat(rows // 6)
    x = 2 * torch.rand(rows, D, generator=gen, device="cuda") - 1
    x[:, 0::128] = 1   # the largest of every 128
    x[:, 1::128] = -1
    x[:, 5::7] = 0
    x = (x * size[:, None]).to(TYPES[dtype])
    w = torch.ones(D, device="cuda")
    codes, scale = vla.rms_norm(x, w, eps=1e-6, out=out, group=group)
    vr, _ = ref.rms_norm(f64(x), f64(w), np.zeros((rows, D)), 1e-6)
    top = 448.0 if out == "e4m3" else 127.0
    sr = ref.scales(vr, top, group)
    scale, q = f64(scale).reshape(rows, -1), f64(codes)
    c = (D / 2 + 8) * U32
    # a product below the normal range is off by 2^-150, of at least 1e-38
    close(scale, sr, (c + 2 * U32 + 2.0 ** -150 / 1e-38) * sr, "scale")
    assert np.isfinite(q).all() and np.abs(q).max() <= top
    want = vr / np.repeat(sr, group or D, 1)[:, :D]
    step = 0.5 if out == "int8" else np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10)
    close(q, want, step * (1 + 1e-3) + (2 * c + 6 * U32) * np.abs(want) + top * 2.0 ** -150 / 1e-38, "codes")
    assert (q[f64(x) == 0] == 0).all()


# ---------------------------------------------------------------------------------------------
# scan: NaN and infinity

CAUSAL = [  # lens, packed, dtype, H, P, N, gate
    ([300], False, "bf16", 2, 64, 128, False),
    ([300, 300], False, "bf16", 2, 72, 64, True),
    ([200, 333, 20], True, "bf16", 2, 128, 64, True),
    ([3000], False, "bf16", 2, 64, 64, False),
    ([20], False, "bf16", 2, 64, 64, True),
    ([300], False, "f32", 2, 64, 64, False),
]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens,packed,dtype,H,P,N,gate", CAUSAL)
def test_nan_and_infinity_reach_no_earlier_token_and_no_other_row(vla, lens, packed, dtype, H, P, N, gate, bad):  # noqa: F811
    """x of one row p not finite at some tokens: its outputs are not finite from the first of them on, all
    other outputs and states are what they are without."""
    gen = generator(P + N)
    lead = (sum(lens),) if packed else (len(lens), lens[0])
    off = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda") if packed else None
    v = scan_inputs(gen, lead, H, P, 1, N, TYPES[dtype], gate, False)
    starts = list(np.cumsum([0, *lens[:-1]]))
    s0 = rand(gen, len(lens), H, P, N)
    s1 = s0.clone()
    want = vla.ssm_scan(**v, state=s0, offsets=off).flatten(0, -3)
    hit = torch.zeros_like(want, dtype=torch.bool)        # outputs that may not be finite
    rows = torch.zeros(len(lens), H, P, dtype=torch.bool, device="cuda")
    x = v["x"].flatten(0, -3)
    assert x.data_ptr() == v["x"].data_ptr()
    for s, (at, n) in enumerate(zip(starts, lens)):
        if s == 1:
            continue   # a sequence that stays clean
        for head, p, tokens in ((0, 3, (n - 2, n // 2, n // 2 + 1)), (1, P - 1, (n - 1,)), (1, 33, (min(127, n - 1),)),
                                (0, 17, (0, n // 3))):
            for t in tokens:
                x[at + t, head, p] = bad
            hit[at + min(tokens):at + n, head, p] = True
            rows[s, head, p] = True
    got = vla.ssm_scan(**v, state=s1, offsets=off).flatten(0, -3)
    assert torch.equal(got[~hit], want[~hit]) and not got[hit].isfinite().any()
    assert torch.equal(s1[~rows], s0[~rows]) and not s1[rows].isfinite().any()


@pytest.mark.parametrize("name", ["dt", "B", "C", "z"])
@pytest.mark.parametrize("T,dtype", [(300, "bf16"), (20, "bf16"), (300, "f32")])
def test_other_operands_that_are_nan_reach_no_earlier_token(vla, name, T, dtype):  # noqa: F811
    gen = generator(T)
    v = scan_inputs(gen, (1, T), 2, 64, 1, 64, TYPES[dtype], True, False)
    t0 = T // 2 - 3
    want = vla.ssm_scan(**v)[0, :t0].double()
    v[name][:, t0] = float("nan")
    got = vla.ssm_scan(**v)[0]
    assert got[t0].isnan().all()
    # a block of tokens with a NaN step takes its exponentials pair by pair: bfloat16 factors may round otherwise
    assert (got[:t0].double() - want).norm() <= 2 * U16 * want.norm()
