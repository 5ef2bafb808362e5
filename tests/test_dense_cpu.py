"""Products with an epilogue and layer norm, as far as they go without a GPU: the float64 references against other
formulas, refusals of the C entry points, and the measured cases."""
import ctypes
import importlib.util
import os
import random

import numpy as np
import pytest
import torch

from _util import ROOT, ensure_built
from oracle import dense_ref as ref


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import sherman_morrison_inverse_gb300 as vla
    return vla.load_library()


def test_activations_against_torch():
    v = np.linspace(-9, 9, 400)
    t = torch.tensor(v, requires_grad=True)
    for kind, fn in (("silu", torch.nn.functional.silu), ("gelu", torch.nn.functional.gelu)):
        y = fn(t)
        assert np.allclose(ref.act(v, kind), y.detach().numpy(), atol=1e-14)
        assert np.allclose(ref.slope(v, kind)[0], torch.autograd.grad(y.sum(), t)[0].numpy(), atol=1e-14)


def test_gradients_against_autograd():
    rng = np.random.default_rng(3)
    x, w, b, dy = (rng.normal(size=s) for s in ((5, 7), (4, 7), (4,), (5, 4)))
    tx, tw, tb = (torch.tensor(t, requires_grad=True) for t in (x, w, b))
    v = tx @ tw.t() + tb
    want = torch.autograd.grad(torch.nn.functional.gelu(v), (tx, tw, tb), torch.tensor(dy))
    got, mag = ref.linear_backward(dy, x, w, v.detach().numpy(), "gelu")
    for g, t, m in zip(got, want, mag):
        assert np.allclose(g, t.numpy(), atol=1e-13) and (m >= np.abs(g) - 1e-13).all()
    nw, nb = rng.normal(size=7), rng.normal(size=7)
    dn = rng.normal(size=(5, 7))
    tn, tnb = (torch.tensor(t, requires_grad=True) for t in (nw, nb))
    y = torch.nn.functional.layer_norm(tx, (7,), tn, tnb, 1e-5)
    got_y, r, mean, rstd = ref.layer_norm(x, nw, nb)
    assert np.allclose(got_y, y.detach().numpy(), atol=1e-13)
    want = torch.autograd.grad(y, (tx, tn, tnb), torch.tensor(dn))
    got, mag = ref.layer_norm_backward(dn, x, nw, mean, rstd)
    for g, t, m in zip(got, want, mag):
        assert np.allclose(g, t.numpy(), atol=1e-12) and (m >= np.abs(g) - 1e-12).all()


def test_scales_and_residual_of_the_reference():
    y, v, mag = ref.linear(np.array([[1.0, -2.0]]), np.array([[3.0, 1.0]]), np.array([0.5]), np.array([[10.0]]), "none",
                           np.array([2.0]), np.array([4.0]))
    assert v[0, 0] == 8.5 and y[0, 0] == 18.5 and mag[0, 0] == 40.5


def test_entry_points_reject_a_null_handle(lib):
    rows = (ctypes.c_longlong * 6)()
    size = ctypes.c_size_t()
    assert lib.vla_linear(None, *(None,) * 8, 1, 1, 1, rows, 0, 0, 0, None, 0, None) == 1
    assert b"handle" in lib.vla_last_error(None)
    assert lib.vla_linear_workspace(None, None, None, 1, 1, 1, rows, 0, 0, ctypes.byref(size)) == 1
    assert lib.vla_linear_backward(None, *(None,) * 7, 1, 1, 1, rows, 0, 0, None, 0, None) == 1
    assert lib.vla_linear_backward_workspace(None, *(None,) * 3, 1, 1, 1, 1, 1, 1, rows, 0, 0, ctypes.byref(size)) == 1
    assert lib.vla_layer_norm(None, *(None,) * 6, 1, 8, 8, 0, 8, 1e-5, 0, 0, None) == 1
    assert lib.vla_layer_norm_backward(None, *(None,) * 8, 1, 8, rows, 0, 0, None, 0, None) == 1
    assert lib.vla_layer_norm_backward_workspace(None, 1, 8, ctypes.byref(size)) == 1


def test_binding_refuses_before_anything_is_launched(lib):
    import sherman_morrison_inverse_gb300 as vla

    class Detached(vla.Handle):   # a handle's checks without a device behind it
        def __init__(self):
            self.lib, self._h, self._ptr_value, self._device_index = lib, None, 0, 0

        def __del__(self):
            pass

    h = Detached()
    native = vla.layer._native
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    call = lambda x, w: native.linear(h, x, w, None, None, None, 0, None, None, None, None, 0)   # noqa: E731
    with pytest.raises(ValueError, match="not on a CUDA device"):
        call(x, w)
    with pytest.raises(ValueError, match="float32, bfloat16 or float8_e4m3fn"):
        call(x.half(), w)
    with pytest.raises(ValueError, match=r"\[N, K\]"):
        call(x, w[0])
    with pytest.raises(AttributeError):
        call(3, w)
    with pytest.raises(ValueError, match="act must be one of"):
        h.linear(x, w, act="tanh")
    with pytest.raises(ValueError, match="not on a CUDA device"):
        native.linear_back(h, torch.zeros(4, 6), x, w, None, 0, None, None, None, 0)
    with pytest.raises(ValueError, match="not on a CUDA device"):
        native.layer_norm(h, x, x[0], None, None, None, 1e-5, False, 0)
    with pytest.raises(ValueError, match="not on a CUDA device"):
        native.layer_norm_back(h, x, x, x[0], None, None, None, None, None, 0)


def test_the_measured_cases_are_well_formed():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    cases = m.listed() + [m.draw(random.Random(i)) for i in range(200)]
    most = {k: max(m.work(c)[k] for c in m.listed()) for k in ("bytes", "flops")}
    for c in cases:
        assert all(isinstance(v, (str, int, bool)) for v in c.values())
        assert all(0 < m.work(c)[k] <= most[k] for k in most)
