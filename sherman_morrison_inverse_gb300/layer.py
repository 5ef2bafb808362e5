"""Operators of a state space layer on GB300: short causal convolution, selective scan, norms, projections.

The methods here are part of ``Handle`` (see the package's docstring); like the rest of the
binding they check and marshal arguments, and every step runs in the library's CUDA kernels.

    r  = rms_norm(x, w, residual, out="e4m3")            # codes and scales for an 8-bit projection
    u  = short_conv(u, w, bias, conv_state)              # x | B | C of the layer's input projection
    y  = ssm_scan(x, dt, A, B, C, ssm_state, D=D, z=z, dt_bias=dt_bias)
    y  = ssm_step(...); u = short_conv_step(...)         # the same states, one token a sequence

    h, st = layer_norm(x, w, b, residual, stats=True)    # the other norm, and its gradients
    dx, dw, db = layer_norm_backward(dh, residual, w, st, dresidual)
    y  = linear(codes, w, bias, residual, act="silu", x_scale=scale, w_scale=ws)   # bfloat16, float32 or e4m3
    dx, dw, db = linear_backward(dy, x, w, pre, act="silu")

A batch of prompts is dense, [S, T, ...], or packed, [tokens, ...] with ``offsets`` (int32 [S + 1]
on the device).  States live in pools, [n_slots, ...], and are updated in place; ``slots`` (int32
[S] on the device) names the slot of each sequence, a negative one skips it.

Outputs that the caller gives must not overlap an input or each other (but ``linear``'s y, which may be its residual).
With ``stream`` a call runs there and allocates from that stream's memory; as of torch's own operators under
``torch.cuda.stream``, its inputs have to be ready there and to live until the work is done (``Tensor.record_stream``).

No operator here records a gradient.  ``linear``, ``layer_norm`` and their gradients refuse a tensor that
requires one while torch records them: call them under ``torch.no_grad()``, or in the forward and backward
of a ``torch.autograd.Function``.
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
_ACT = {"none": 0, "silu": 1, "gelu": 2}


def _dense(x, dtype=None):
    return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)


def _empty(x, shape):
    return x.new_empty(shape, dtype=torch.float32)


def _bytes(x, n):
    return x.new_empty(n, dtype=torch.uint8)


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


def _there(call, args, stream):
    """A call on a stream other than the current one, its outputs allocated from that stream's memory."""
    with torch.cuda.stream(stream):
        return call(*args, stream.cuda_stream)


class _Missing:
    """Stands in for the argument checks in C where they are not built: the layer's operators say so
    when they are called, and the rest of the library loads without them."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise RuntimeError(f"_layer_binding is not built, or not from these sources ({self._why}); run "
                           "`python -m sherman_morrison_inverse_gb300.build`")


_native = None


def declare(lib):
    """Declare the layer's C signatures, and hand the entry points to the argument checks in C.  Where those are missing or of
    other sources, the layer's operators say so when they are called."""
    global _native
    vp, ci, cll, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    lib.vla_short_conv.argtypes = [vp] * 6 + [cll] * 3 + [vp] * 2 + [cll] * 2 + [ci, vp, ci, ci, vp]
    lib.vla_ssm_scan.argtypes = [vp] * 11 + [cll] * 3 + [vp] * 2 + [cll] * 5 + [vp, ci, ci, vp, ctypes.c_size_t, vp]
    lib.vla_ssm_workspace.argtypes = [vp, cll, cll, cll, ci, cll, cll, cll, ci, ctypes.POINTER(ctypes.c_size_t)]
    lib.vla_rms_norm.argtypes = [vp] * 6 + [cll] * 5 + [cf, ci, ci, ci, ci, vp]
    size = ctypes.POINTER(ctypes.c_size_t)
    lib.vla_linear.argtypes = [vp] * 9 + [cll] * 3 + [vp, ci, ci, ci, vp, ctypes.c_size_t, vp]
    lib.vla_linear_workspace.argtypes = [vp] * 3 + [cll] * 3 + [vp, ci, ci, size]
    lib.vla_linear_backward.argtypes = [vp] * 8 + [cll] * 3 + [vp, ci, ci, vp, ctypes.c_size_t, vp]
    lib.vla_linear_backward_workspace.argtypes = [vp] * 4 + [ci] * 3 + [cll] * 3 + [vp, ci, ci, size]
    lib.vla_layer_norm.argtypes = [vp] * 7 + [cll] * 5 + [cf, ci, ci, vp]
    lib.vla_layer_norm_backward.argtypes = [vp] * 9 + [cll] * 2 + [vp, ci, ci, vp, ctypes.c_size_t, vp]
    lib.vla_layer_norm_backward_workspace.argtypes = [vp, cll, cll, size]
    dense = (lib.vla_linear, lib.vla_linear_workspace, lib.vla_linear_backward, lib.vla_linear_backward_workspace,
             lib.vla_layer_norm, lib.vla_layer_norm_backward, lib.vla_layer_norm_backward_workspace)
    for fn in (lib.vla_short_conv, lib.vla_ssm_scan, lib.vla_ssm_workspace, lib.vla_rms_norm, *dense):
        fn.restype = ci
    try:
        loader = importlib.machinery.ExtensionFileLoader(f"{__package__}._layer_binding", BINDING)
        native = importlib.util.module_from_spec(importlib.util.spec_from_loader(loader.name, loader))
        loader.exec_module(native)
        _hand_over(native, lib, dense)
    except (ImportError, AttributeError, TypeError) as e:   # not there; of older sources, without a function or an argument of it
        _native = _Missing(e)
        return
    _native = native


def _hand_over(native, lib, dense):
    at = [ctypes.cast(fn, ctypes.c_void_p).value
          for fn in (lib.vla_short_conv, lib.vla_ssm_scan, lib.vla_ssm_workspace, lib.vla_rms_norm)]
    # the current stream's handle without a Stream object around it, where torch has that
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
    native.setup(*at, torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn, torch.int8,
                 torch.empty_like, _dense, _empty, _bytes, stream)
    # the caching allocator without the dispatcher around it, the current device, and the number of modes that watch the
    # dispatcher, where torch has all three
    strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)
    here = getattr(torch._C, "_cuda_getDevice", None)
    modes = getattr(torch._C, "_len_torch_dispatch_stack", None)
    if strided is None or here is None or modes is None:
        strided = here = modes = None
    native.setup_dense(*[ctypes.cast(fn, ctypes.c_void_p).value for fn in dense], torch.is_grad_enabled, torch.empty, torch.uint8,
                       strided, here, modes)


_here = contextlib.nullcontext()


def _on(stream):
    """Outputs are allocated from the memory of the stream that writes them."""
    return _here if stream is None else torch.cuda.stream(stream)


def _raw(stream):
    return None if stream is None else stream.cuda_stream


def _activation(act):
    kind = _ACT.get(act)
    if kind is None:
        raise ValueError(f"act must be one of {sorted(_ACT)}")
    return kind


class LayerOps:
    """Methods of Handle: the state space layer's operators, and the products and layer norms around them."""

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

    def linear(self, x, w, bias=None, residual=None, y=None, *, act: str = "none", pre=None, x_scale=None, w_scale=None,
               dtype=None, stream=None):
        """y = act(v) + residual, v = x w^T + bias, the product of a projection with its epilogue.

        x [..., K] and w [N, K] in one type, bfloat16, float32 or e4m3 codes, their rows evenly
        spaced; codes stand for codes * x_scale[..., None] (those of rms_norm with a scale a row) and
        codes * w_scale[:, None], [...] and [N] float32 (None: 1).  bias [N] float32.  act "none", "silu"
        or "gelu" (v Phi(v)).  Returns y [..., N] in `dtype`: x's type, bfloat16 for codes, or
        float32.  residual and pre have y's shape and type; pre receives v, for the gradient; y may
        be the residual itself."""
        kind = _activation(act)
        args = (self, x, w, bias, residual, y, kind, pre, x_scale, w_scale, dtype)
        return _native.linear(*args, None) if stream is None else _there(_native.linear, args, stream)

    def linear_backward(self, dy, x, w, pre=None, dx=None, dw=None, db=None, *, act: str = "none", input: bool = True,
                        weight: bool = True, bias: bool = True, stream=None):
        """Gradients of linear: g = dy * act'(pre); dx = g w, dw = g^T x, db = the sum of g's rows.

        dy [..., N], x [..., K], w [N, K] and pre [..., N] (what linear left there; not needed
        without an activation) in one type, bfloat16 or float32.  Returns (dx, dw, db), dx and dw in
        that type, db float32; None in the place of those that input, weight or bias say not to
        compute.  The residual's gradient is dy."""
        kind = _activation(act)
        args = (self, dy, x, w, pre, kind, dx if input else False, dw if weight else False, db if bias else False)
        return _native.linear_back(*args, None) if stream is None else _there(_native.linear_back, args, stream)

    def layer_norm(self, x, w, b=None, residual=None, y=None, *, eps: float = 1e-5, stats=False, stream=None):
        """y = (r - mean(r)) / sqrt(var(r) + eps) * w + b over the last dimension, r = x + residual.

        x [..., D] float32 or bfloat16, its rows evenly spaced; w, b [D] float32; residual (x's
        shape, float32 or bfloat16) is updated in place to r.  Returns y in x's type; with stats=True
        (y, stats), stats [..., 2] float32 the rows' mean and 1 / sqrt(var + eps) for the gradient."""
        if stats is None:
            stats = False
        args = (self, x, w, b, residual, y, eps, stats)
        return _native.layer_norm(*args, None) if stream is None else _there(_native.layer_norm, args, stream)

    def layer_norm_backward(self, dy, x, w, stats, dresidual=None, dx=None, dw=None, db=None, *, bias: bool = True,
                            stream=None):
        """Gradients of layer_norm: dx = (a - mean(a) - h mean(a h)) rstd + dresidual, a = dy w and h the
        normalised row; dw = the rows' sum of dy h, db = that of dy.

        dy [..., D]; x what was normalised (x, or the residual that the call left), stats as
        layer_norm returned them; dresidual (x's shape and type) the gradient that the residual
        stream already has.  dx has x's type.  Returns (dx, dw, db), dw and db float32; db None without bias."""
        args = (self, dy, x, w, stats, dresidual, dx, dw, db if bias else False)
        return _native.layer_norm_back(*args, None) if stream is None else _there(_native.layer_norm_back, args, stream)
