"""The layer operators' argument checks in C: what the library does without them, and with a module that
is stale or of another interpreter."""
import os
import subprocess
import sys

import pytest

from _util import ROOT, ensure_built
from sherman_morrison_inverse_gb300 import build as b


def python(code):
    """What a fresh interpreter prints."""
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    return p.stdout


def test_the_library_loads_without_the_binding():
    """The scans need nothing of it; the layer's operators say what is missing when they are called."""
    ensure_built()
    out = python("""
import sys
sys.modules["sherman_morrison_inverse_gb300._layer_binding"] = None   # not to be had
import sherman_morrison_inverse_gb300 as vla, torch
vla.layer.BINDING = "nowhere"
lib = vla.load_library()
assert lib.vla_scan_fwd.argtypes
class Detached(vla.Handle):
    def __init__(self): self.lib, self._h, self._ptr_value, self._device_index = lib, None, 0, 0
    def __del__(self): pass
x = torch.zeros(2, 8)
for call in (lambda h: h.rms_norm(x, x[0]), lambda h: h.short_conv_step(x, x), lambda h: h.ssm_step(x, x, x, x, x)):
    try:
        call(Detached())
    except RuntimeError as e:
        print(e)
""")
    assert out.count("_layer_binding is not built") == 3


@pytest.mark.parametrize("headers", [True, False])
def test_the_library_is_built_where_the_binding_cannot_be(monkeypatch, tmp_path, headers):
    def run(cmd, **kw):
        ok = headers or "layer_binding.c" not in " ".join(cmd)
        if ok:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0 if ok else 1, "", "" if ok else "Python.h: No such file")

    monkeypatch.setattr(b.subprocess, "run", run)
    for name in ("LIB", "BINDING", "OUT_DIR"):
        monkeypatch.setattr(b, name, str(tmp_path / name))
    if headers:
        assert b.build() == b.LIB and os.path.exists(b.LIB) and os.path.exists(b.BINDING)
    else:
        with pytest.warns(UserWarning, match="Python.h"):
            assert b.build() == b.LIB
        assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)


@pytest.mark.parametrize("state", ["missing", "older than its source", "fresh"])
def test_tests_do_not_run_on_a_stale_binding(monkeypatch, tmp_path, state):
    made = tmp_path / "binding"
    for name, path in (("LIB", tmp_path / "lib"), ("BINDING", made)):
        monkeypatch.setattr(b, name, str(path))
        path.touch()   # as new as can be
    if state == "missing":
        made.unlink()
    elif state != "fresh":
        os.utime(made, (0, 0))
    calls = []
    monkeypatch.setattr(b, "build", lambda: calls.append("library"))
    monkeypatch.setattr(b, "build_binding", lambda: calls.append("binding"))
    ensure_built()
    assert calls == ([] if state == "fresh" else ["binding"])


def test_a_module_of_another_interpreter_is_not_loaded(tmp_path):
    """The file's name carries the interpreter's tag, and an untagged one beside it is not taken for it."""
    import sysconfig
    ensure_built()
    assert os.path.basename(b.BINDING) == "_layer_binding" + sysconfig.get_config_var("EXT_SUFFIX")
    package = tmp_path / "sherman_morrison_inverse_gb300"
    package.mkdir()
    here = os.path.dirname(b.LIB)
    for name in ("__init__.py", "layer.py", "build.py", "libvla.so"):
        os.symlink(os.path.join(here, name), package / name)
    (package / "_layer_binding.so").write_bytes(b"of another interpreter")
    out = python(f"""
import importlib.util, os, sys
sys.path.insert(0, {str(tmp_path)!r})
import sherman_morrison_inverse_gb300 as vla
assert vla.__file__.startswith({str(tmp_path)!r}), vla.__file__
vla.load_library()
try:
    vla.layer._native.norm
except RuntimeError as e:
    print(e)
""")
    assert "not built" in out and "_layer_binding.so" not in out


@pytest.mark.parametrize("call", ["norm", "conv", "scan"])
def test_other_threads_run_during_a_call(call):
    """A launch can wait for the device's queue: it does so without the interpreter's lock.  The entry points
    are replaced by libc's usleep, whose argument is the handle."""
    ensure_built()
    out = python(f"""
import ctypes, threading, time
from sherman_morrison_inverse_gb300 import layer
import importlib.util
loader = importlib.machinery.ExtensionFileLoader("x._layer_binding", layer.BINDING)
native = importlib.util.module_from_spec(importlib.util.spec_from_loader(loader.name, loader))
sleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
nothing = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: 0)
f32, other = object(), object()
native.setup(sleep, sleep, ctypes.cast(nothing, ctypes.c_void_p).value, sleep, f32, other, other, other, other,
             *[lambda *a, **k: 1 / 0] * 5)
class Handle:
    _ptr_value, _device_index = 900000, 0
class Tensor:
    dtype = f32
    def __init__(self, *shape):
        self.shape = shape
        strides = [1]
        for n in shape[:0:-1]:
            strides.insert(0, strides[0] * n)
        self.strides = tuple(strides)
    def stride(self): return self.strides
    def get_device(self): return 0
    def data_ptr(self): return 64
seen, stop = [], False
def watch():
    while not stop:
        seen.append(time.monotonic())
        time.sleep(0.01)
t = threading.Thread(target=watch)
t.start()
T = Tensor
start = time.monotonic()
if {call!r} == "norm":
    native.norm(Handle(), T(2, 8), T(8), None, T(2, 8), 1e-6, 0, 0, None, 0)
elif {call!r} == "conv":
    native.conv(Handle(), T(1, 4, 8), T(8, 2), None, None, T(1, 4, 8), True, None, None, None, False, 0)
else:
    native.scan(Handle(), T(1, 4, 2, 8), T(1, 4, 2), T(2), T(1, 4, 1, 4), T(1, 4, 1, 4), None, T(1, 4, 2, 8), None, None,
                None, True, None, None, None, False, 0)
end = time.monotonic()
stop = True
t.join()
print(end - start, sum(start + 0.1 < s < end - 0.1 for s in seen))
""")
    took, seen = out.split()
    assert float(took) > 0.8 and int(seen) >= 3
