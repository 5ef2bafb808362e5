"""Operators of a state space layer on GB300: short causal convolution, selective scan, norm.

The methods here are part of ``Handle`` (see the package's docstring); like the rest of the
binding they check and marshal arguments, and every step runs in the library's CUDA kernels.

    r  = rms_norm(x, w, residual, out="e4m3")            # codes and scales for an 8-bit projection
    u  = short_conv(u, w, bias, conv_state)              # x | B | C of the layer's input projection
    y  = ssm_scan(x, dt, A, B, C, ssm_state, D=D, z=z, dt_bias=dt_bias)
    y  = ssm_step(...); u = short_conv_step(...)         # the same states, one token a sequence

A batch of prompts is dense, [S, T, ...], or packed, [tokens, ...] with ``offsets`` (int32 [S + 1]
on the device).  States live in pools, [n_slots, ...], and are updated in place; ``slots`` (int32
[S] on the device) names the slot of each sequence, a negative one skips it.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os
import sysconfig

import torch

STATUS_INDEX = 4
# The argument checks in C, for this interpreter and machine: a module of another one has another name.
BINDING = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                       "_layer_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
_OUT = {"io": 0, "e4m3": 1, "int8": 2}


def _dense(x, dtype=None):
    return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)


def _empty(x, shape):
    return x.new_empty(shape, dtype=torch.float32)


def _bytes(x, n):
    return x.new_empty(n, dtype=torch.uint8)


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


class _Missing:
    """Stands in for the argument checks in C where they are not built: the layer's operators say so
    when they are called, and the rest of the library loads without them."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise RuntimeError(f"_layer_binding is not built ({self._why}); run "
                           "`python -m sherman_morrison_inverse_gb300.build`")


_native = None


def declare(lib):
    """Declare the layer's C signatures, and hand the entry points to the argument checks in C."""
    global _native
    vp, ci, cll, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    lib.vla_short_conv.argtypes = [vp] * 6 + [cll] * 3 + [vp] * 2 + [cll] * 2 + [ci, vp, ci, ci, vp]
    lib.vla_ssm_scan.argtypes = [vp] * 11 + [cll] * 3 + [vp] * 2 + [cll] * 5 + [vp, ci, ci, vp, ctypes.c_size_t, vp]
    lib.vla_ssm_workspace.argtypes = [vp, cll, cll, cll, ci, cll, cll, cll, ci, ctypes.POINTER(ctypes.c_size_t)]
    lib.vla_rms_norm.argtypes = [vp] * 6 + [cll] * 5 + [cf, ci, ci, ci, ci, vp]
    for fn in (lib.vla_short_conv, lib.vla_ssm_scan, lib.vla_ssm_workspace, lib.vla_rms_norm):
        fn.restype = ci
    try:
        loader = importlib.machinery.ExtensionFileLoader(f"{__package__}._layer_binding", BINDING)
        native = importlib.util.module_from_spec(importlib.util.spec_from_loader(loader.name, loader))
        loader.exec_module(native)
    except ImportError as e:
        _native = _Missing(e)
        return
    at = [ctypes.cast(fn, ctypes.c_void_p).value
          for fn in (lib.vla_short_conv, lib.vla_ssm_scan, lib.vla_ssm_workspace, lib.vla_rms_norm)]
    # the current stream's handle without a Stream object around it, where torch has that
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
    native.setup(*at, torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn, torch.int8,
                 torch.empty_like, _dense, _empty, _bytes, stream)
    _native = native


_here = contextlib.nullcontext()


def _on(stream):
    """Outputs are allocated from the memory of the stream that writes them."""
    return _here if stream is None else torch.cuda.stream(stream)


def _raw(stream):
    return None if stream is None else stream.cuda_stream


class LayerOps:
    """Methods of Handle: the state space layer's operators."""

    def _layer_fail(self, code):
        from . import VlaError
        msg = self.lib.vla_last_error(self._h)
        raise VlaError(code, msg.decode() if msg else "")

    def short_conv(self, x, w, bias=None, state=None, y=None, *, silu: bool = True, offsets=None, slots=None,
                   max_len: int | None = None, stream=None):
        """y[t, c] = act(bias[c] + sum_j w[c, j] x[t - K + 1 + j, c]) over every sequence.

        x [S, T, C], or [tokens, C] with offsets; float32 or bfloat16, channels adjacent.  w [C, K]
        (2 to 4 taps) and bias [C] float32.  state [n_slots, K - 1, C] in x's dtype holds the
        inputs before the sequence and is updated in place (None: zeros, not kept).  Returns y."""
        with _on(stream):
            return _native.conv(self, x, w, bias, state, y, silu, offsets, slots, max_len, False, _raw(stream))

    def short_conv_step(self, x, w, bias=None, state=None, y=None, *, silu: bool = True, slots=None, stream=None):
        """One token a sequence: x [S, C] -> y [S, C] (see short_conv)."""
        with _on(stream):
            return _native.conv(self, x, w, bias, state, y, silu, None, slots, None, True, _raw(stream))

    def ssm_scan(self, x, dt, A, B, C, state=None, y=None, *, D=None, z=None, dt_bias=None, softplus: bool = True,
                 offsets=None, slots=None, max_len: int | None = None, stream=None):
        """The selective scan: s = softplus(dt + dt_bias), h = exp(A s) h + s x B^T,
        y = (h C + D x) * silu(z), token by token over every sequence.

        x, z [S, T, H, P], dt [S, T, H], B, C [S, T, G, N] (G divides H), or without S and with
        offsets; one dtype, float32 or bfloat16, the values of a token adjacent.  A, D, dt_bias [H]
        float32.  state [n_slots, H, P, N] float32 is updated in place (None: zeros, not kept).
        Returns y in x's shape."""
        with _on(stream):
            return _native.scan(self, x, dt, A, B, C, state, y, D, z, dt_bias, softplus, offsets, slots, max_len,
                                False, _raw(stream))

    def ssm_step(self, x, dt, A, B, C, state=None, y=None, *, D=None, z=None, dt_bias=None, softplus: bool = True,
                 slots=None, stream=None):
        """One token a sequence: x, z [S, H, P], dt [S, H], B, C [S, G, N] (see ssm_scan)."""
        with _on(stream):
            return _native.scan(self, x, dt, A, B, C, state, y, D, z, dt_bias, softplus, None, slots, None, True,
                                _raw(stream))

    def rms_norm(self, x, w, residual=None, y=None, *, eps: float = 1e-6, out: str = "io", group: int = 0,
                 scale=None, stream=None):
        """v = r / sqrt(mean(r^2) + eps) * w over the last dimension, r = x + residual.

        x [..., D] float32 or bfloat16, its rows evenly spaced; w [D] float32; residual (x's shape,
        float32 or bfloat16) is updated in place to r.  out="io" returns v in x's dtype; "e4m3" and
        "int8" return (codes, scale): v ~ codes * scale with one scale a row, or with group=128 one
        for every 128 values ([..., ceil(D / 128)])."""
        kind = _OUT.get(out)
        if kind is None:
            raise ValueError(f"out must be one of {sorted(_OUT)}")
        with _on(stream):
            return _native.norm(self, x, w, residual, y, eps, kind, group, scale, _raw(stream))
