"""The state space layer's operators where their numbers run to the ends of their ranges, against the
float64 references and the bounds of test_gpu_layer.py."""
import math

import pytest

from test_gpu_layer import check_scan, generator, vla  # noqa: F401

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
