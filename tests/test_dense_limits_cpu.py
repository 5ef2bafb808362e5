"""What the products' and norms' calls refuse and how they end, as far as that goes without a GPU."""
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

from _util import ROOT, ensure_built


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import sherman_morrison_inverse_gb300 as vla
    return vla.load_library()


def test_the_wait_limit_needs_a_handle(lib):
    assert lib.vla_wait_limit(None, 100) == 1
    assert b"handle" in lib.vla_last_error(None)


@pytest.fixture
def detached(lib):
    """A handle's checks without a device behind it."""
    import sherman_morrison_inverse_gb300 as vla

    class Detached(vla.Handle):
        def __init__(self):
            self.lib, self._h, self._ptr_value, self._device_index = lib, None, 0, 0

        def __del__(self):
            pass

    return Detached()


def test_tensors_that_require_a_gradient_are_refused(detached):
    """The result would silently have none.  Without gradients being recorded the next check speaks."""
    import sherman_morrison_inverse_gb300 as vla
    native, h = vla.layer._native, detached
    z = lambda *s: torch.zeros(*s)   # noqa: E731
    calls = {   # name -> the call's arguments but the handle and the stream
        native.linear: dict(x=z(4, 8), w=z(6, 8), bias=z(6), residual=z(4, 6), y=z(4, 6), act=0, pre=z(4, 6), x_scale=z(4), w_scale=z(6),
                            dtype=None),
        native.linear_back: dict(dy=z(4, 6), x=z(4, 8), w=z(6, 8), pre=z(4, 6), act=1, dx=z(4, 8), dw=z(6, 8), db=z(6)),
        native.layer_norm: dict(x=z(4, 8), w=z(8), b=z(8), residual=z(4, 8), y=z(4, 8), eps=1e-5, stats=z(4, 2)),
        native.layer_norm_back: dict(dy=z(4, 8), x=z(4, 8), w=z(8), stats=z(4, 2), dresidual=z(4, 8), dx=z(4, 8), dw=z(8), db=z(8)),
    }
    for call, args in calls.items():
        for name, value in args.items():
            if not torch.is_tensor(value):
                continue
            value.requires_grad_()
            with pytest.raises(ValueError, match=f"^{name} requires a gradient"):
                call(h, *args.values(), 0)
            with torch.no_grad(), pytest.raises(ValueError, match="not on a CUDA device"):
                call(h, *args.values(), 0)
            value.requires_grad_(False)
        with pytest.raises(ValueError, match="not on a CUDA device"):
            call(h, *args.values(), 0)


@pytest.mark.parametrize("older", ["without setup_dense", "setup_dense of other arguments"])
def test_a_binding_of_older_sources_does_not_keep_the_library_from_loading(lib, tmp_path, older):
    """The scans load without it, and the layer's operators say what to do when they are called."""
    from sherman_morrison_inverse_gb300 import build as b
    with open(os.path.join(b.CSRC, "layer_binding.c")) as f:
        text = f.read()
    if older == "without setup_dense":
        old = text.replace('    {"setup_dense", py_setup_dense, METH_VARARGS, NULL},\n', "")
    else:
        old = text.replace('"KKKKKKKOOOOOO"', '"KKKKKKKOOOOO"')
    assert old != text
    source = tmp_path / "layer_binding.c"
    source.write_text(old)
    made = tmp_path / os.path.basename(b.BINDING)
    subprocess.run(["gcc", "-w", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"], "-I", b.INCLUDE, str(source), "-o",
                    str(made)], check=True)
    code = f"""
import sherman_morrison_inverse_gb300 as vla, torch
vla.layer.BINDING = {str(made)!r}
lib = vla.load_library()
assert lib.vla_scan_fwd.argtypes
class Detached(vla.Handle):
    def __init__(self): self.lib, self._h, self._ptr_value, self._device_index = lib, None, 0, 0
    def __del__(self): pass
x = torch.zeros(2, 8)
for call in (lambda h: h.rms_norm(x, x[0]), lambda h: h.linear(x, x), lambda h: h.layer_norm(x, x[0])):
    try:
        call(Detached())
    except RuntimeError as e:
        print(e)
"""
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    assert p.stdout.count("not from these sources") == 3
