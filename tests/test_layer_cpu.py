"""The state space layer's operators, as far as they go without a GPU: the float64 references against
closed forms and independent formulas, and refusals of the C entry points."""
import ctypes
import os

import numpy as np
import pytest

from _util import ROOT, ensure_built
from oracle import layer_ref as ref


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import sherman_morrison_inverse_gb300 as vla
    return vla.load_library()


def test_convolution_against_numpy_convolve():
    rng = np.random.default_rng(1)
    x, w, b, s = rng.normal(size=(20, 3)), rng.normal(size=(3, 4)), rng.normal(size=3), rng.normal(size=(3, 3))
    y, y_abs, state = ref.short_conv(x, w, b, s, False)
    for c in range(3):
        whole = np.concatenate([s[:, c], x[:, c]])
        assert np.allclose(y[:, c], np.convolve(whole, w[c, ::-1], "valid") + b[c], atol=1e-13)
    assert np.array_equal(state, x[-3:]) and (y_abs >= np.abs(y) - 1e-13).all()
    assert np.array_equal(ref.short_conv(x[:1], w, b, s, False)[2], np.concatenate([s[1:], x[:1]]))


def test_scan_with_a_constant_decay_is_a_geometric_sum():
    T, s, A = 9, 0.5, -1.25
    one = np.ones((T, 1, 1))
    y, _, h, _ = ref.ssm_scan(one, np.full((T, 1), s), np.array([A]), one, one, np.zeros((1, 1, 1)), softplus_on=False)
    a = np.exp(A * s)
    want = s * (1 - a ** np.arange(1, T + 1)) / (1 - a)
    assert np.allclose(y[:, 0, 0], want, rtol=1e-14) and np.isclose(h[0, 0, 0], want[-1])


def test_scan_against_its_matrix_form():
    """Y = (C B^T o decays o steps) X + decay C h: the form the prompt kernel computes chunk by chunk."""
    rng = np.random.default_rng(2)
    T, H, P, G, N = 12, 4, 3, 2, 5
    x, dt, z = rng.normal(size=(T, H, P)), rng.normal(size=(T, H)), rng.normal(size=(T, H, P))
    B, C, h0 = rng.normal(size=(T, G, N)), rng.normal(size=(T, G, N)), rng.normal(size=(H, P, N))
    A, D, bias = -rng.uniform(0.5, 3, H), rng.normal(size=H), rng.normal(size=H)
    y, y_abs, h, _ = ref.ssm_scan(x, dt, A, B, C, h0, D, z, bias)
    s = np.log1p(np.exp(dt + bias))
    cum = np.cumsum(A * s, 0)
    for i in range(H):
        b, c = B[:, i // 2], C[:, i // 2]
        decay = np.tril(np.exp(cum[:, None, i] - cum[None, :, i]))
        want = (c @ b.T * decay * s[:, i]) @ x[:, i] + np.exp(cum[:, i])[:, None] * (c @ h0[i].T) + D[i] * x[:, i]
        assert np.allclose(y[:, i], want * z[:, i] / (1 + np.exp(-z[:, i])), atol=1e-12)
        tail = s[:, i] * np.exp(cum[-1, i] - cum[:, i])
        assert np.allclose(h[i], np.exp(cum[-1, i]) * h0[i] + (x[:, i] * tail[:, None]).T @ b, atol=1e-12)
    assert (y_abs >= np.abs(y) - 1e-12).all()


def test_norm_of_a_known_row():
    v, r = ref.rms_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), np.array([[0.0, 0.0]]), 0.0)
    assert np.allclose(v, np.array([[3.0, 8.0]]) / np.sqrt(12.5)) and np.array_equal(r, [[3.0, 4.0]])
    assert np.allclose(ref.scales(np.array([[1.0] * 128 + [-2.0]]), 127.0, 128), [[1 / 127, 2 / 127]])
    assert ref.scales(np.zeros((1, 5)), 448.0, 0) == 1.0


def test_entry_points_reject_a_null_handle(lib):
    n = (None,) * 5
    assert lib.vla_short_conv(None, *n, 1, 4, 4, None, None, 0, 8, 4, None, 0, 0, None) == 1
    assert b"handle" in lib.vla_last_error(None)
    assert lib.vla_ssm_scan(None, *n, *n, 1, 4, 4, None, None, 0, 2, 8, 1, 8, None, 1, 0, None, 0, None) == 1
    size = ctypes.c_size_t()
    assert lib.vla_ssm_workspace(None, 1, 4, 4, 0, 2, 8, 8, 0, ctypes.byref(size)) == 1
    assert lib.vla_rms_norm(None, *n, 1, 8, 8, 0, 8, 1e-6, 0, 0, 0, 0, None) == 1
    assert b"handle" in lib.vla_last_error(None)


def test_binding_refuses_host_tensors(lib):
    """Shapes, types and places are checked before anything is launched."""
    import torch
    import sherman_morrison_inverse_gb300 as vla

    class Detached(vla.Handle):   # a handle's checks without a device behind it
        def __init__(self):
            self.lib, self._h, self._ptr_value, self._device_index = lib, None, 0, 0

        def __del__(self):
            pass

    import sherman_morrison_inverse_gb300.layer as layer
    h = Detached()
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    call = lambda *a: layer._native.conv(h, *a, None, None, None, True, None, None, None, False, 0)   # noqa: E731
    with pytest.raises(ValueError, match="not on a CUDA device"):
        call(x, w)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        call(x.half(), w)
    with pytest.raises(ValueError, match=r"\[S, T, C\]"):
        call(x[0], w)
    with pytest.raises(AttributeError):
        call(3, w)


def test_the_measured_cases_are_well_formed():
    """perf/operators.py lists and draws cases of plain values; work() counts each input once."""
    import importlib.util
    import random
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    cases = m.listed() + [m.draw(random.Random(i)) for i in range(50)]
    most = max(m.work(c)["bytes"] for c in m.listed())
    for c in cases:
        assert all(isinstance(v, (str, int, bool)) for v in c.values())
        assert 0 < m.work(c)["bytes"] <= most
