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

import torch

STATUS_INDEX = 4
OUT_IO, OUT_E4M3, OUT_INT8 = 0, 1, 2
_OUT = {"io": (OUT_IO, None), "e4m3": (OUT_E4M3, torch.float8_e4m3fn), "int8": (OUT_INT8, torch.int8)}
_IO = {torch.float32: 0, torch.bfloat16: 1}
_Four, _Twelve = ctypes.c_longlong * 4, ctypes.c_longlong * 12


def declare(lib):
    """C signatures of the layer's entry points."""
    vp, ci, cll, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    lib.vla_short_conv.argtypes = [vp] * 6 + [cll] * 3 + [vp] * 2 + [cll] * 2 + [ci, vp, ci, ci, vp]
    lib.vla_ssm_scan.argtypes = [vp] * 11 + [cll] * 3 + [vp] * 2 + [cll] * 5 + [vp, ci, ci, vp, ctypes.c_size_t, vp]
    lib.vla_ssm_workspace.argtypes = [vp, cll, cll, cll, ci, cll, cll, cll, ci, ctypes.POINTER(ctypes.c_size_t)]
    lib.vla_rms_norm.argtypes = [vp] * 6 + [cll] * 5 + [cf, ci, ci, ci, ci, vp]
    for fn in (lib.vla_short_conv, lib.vla_ssm_scan, lib.vla_ssm_workspace, lib.vla_rms_norm):
        fn.restype = ci


def _ptr(t):
    return None if t is None else t.data_ptr()


def _allocating(stream):
    """Where outputs are allocated: from the memory of the stream that writes them."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class LayerOps:
    """Methods of Handle: the state space layer's operators."""

    def _layer_check(self, name, t, shape, dtype):
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the handle is on {self.device}")

    def _layer_dense(self, name, t, shape, dtype):
        self._layer_check(name, t, shape, dtype)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")

    def _layer_rows(self, name, t, shape, dtype, lead):
        """(sequence stride, token stride) of token rows whose values within a token are adjacent."""
        self._layer_check(name, t, shape, dtype)
        strides, width = t.stride(), 1
        for i in range(len(shape) - 1, lead - 1, -1):
            if shape[i] != 1 and strides[i] != width:
                raise ValueError(f"{name}: the values of a token must be adjacent (strides {strides})")
            width *= shape[i]
        return (strides[0], strides[1]) if lead == 2 else (0, strides[0])

    def _layer_seqs(self, x, offsets, slots, state, max_len):
        """(leading dimensions, sequences, T, max_len, slots in the pool) of a batch."""
        if offsets is None:
            n_seq, T, lead = x.shape[0], x.shape[1], 2
            max_len = T
        else:
            if offsets.dim() != 1 or offsets.shape[0] < 1:
                raise ValueError("offsets must be [sequences + 1]")
            self._layer_dense("offsets", offsets, offsets.shape, torch.int32)
            n_seq, T, lead = offsets.shape[0] - 1, x.shape[0], 1
            max_len = T if max_len is None else int(max_len)
        if slots is not None:
            if state is None:
                raise ValueError("slots need a state")
            self._layer_dense("slots", slots, (n_seq,), torch.int32)
        return lead, n_seq, T, max_len, 0 if state is None else state.shape[0]

    def short_conv(self, x, w, bias=None, state=None, y=None, *, silu: bool = True, offsets=None, slots=None,
                   max_len: int | None = None, stream=None):
        """y[t, c] = act(bias[c] + sum_j w[c, j] x[t - K + 1 + j, c]) over every sequence.

        x [S, T, C], or [tokens, C] with offsets; float32 or bfloat16, channels adjacent.  w [C, K]
        (2 to 4 taps) and bias [C] float32.  state [n_slots, K - 1, C] in x's dtype holds the
        inputs before the sequence and is updated in place (None: zeros, not kept).  Returns y."""
        if x.dim() != (3 if offsets is None else 2):
            raise ValueError("x must be [S, T, C], or [tokens, C] with offsets")
        io = _IO.get(x.dtype)
        if io is None:
            raise ValueError("x must be float32 or bfloat16")
        if w.dim() != 2 or w.shape[0] != x.shape[-1]:
            raise ValueError("w must be [C, K]")
        C, K = w.shape
        lead, n_seq, T, max_len, n_slots = self._layer_seqs(x, offsets, slots, state, max_len)
        xs = self._layer_rows("x", x, x.shape, x.dtype, lead)
        self._layer_dense("w", w, w.shape, torch.float32)
        if bias is not None:
            self._layer_dense("bias", bias, (C,), torch.float32)
        if state is not None:
            self._layer_dense("state", state, (n_slots, K - 1, C), x.dtype)
        if y is None:
            with _allocating(stream):
                y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        ys = self._layer_rows("y", y, x.shape, x.dtype, lead)
        code = self.lib.vla_short_conv(self._h, x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(state), y.data_ptr(),
                                       n_seq, T, max_len, _ptr(offsets), _ptr(slots), n_slots, C, K,
                                       _Four(*xs, *ys), silu, io, self._layer_stream(stream))
        if code:
            self._layer_fail(code)
        return y

    def short_conv_step(self, x, w, bias=None, state=None, y=None, *, silu: bool = True, slots=None, stream=None):
        """One token a sequence: x [S, C] -> y [S, C] (see short_conv)."""
        if x.dim() != 2:
            raise ValueError("x must be [S, C]")
        out = self.short_conv(x.unsqueeze(1), w, bias, state, None if y is None else y.unsqueeze(1), silu=silu,
                              slots=slots, stream=stream)
        return out.squeeze(1) if y is None else y

    def ssm_scan(self, x, dt, A, B, C, state=None, y=None, *, D=None, z=None, dt_bias=None, softplus: bool = True,
                 offsets=None, slots=None, max_len: int | None = None, stream=None):
        """The selective scan: s = softplus(dt + dt_bias), h = exp(A s) h + s x B^T,
        y = (h C + D x) * silu(z), token by token over every sequence.

        x, z [S, T, H, P], dt [S, T, H], B, C [S, T, G, N] (G divides H), or without S and with
        offsets; one dtype, float32 or bfloat16, the values of a token adjacent.  A, D, dt_bias [H]
        float32.  state [n_slots, H, P, N] float32 is updated in place (None: zeros, not kept).
        Returns y in x's shape."""
        if x.dim() != (4 if offsets is None else 3):
            raise ValueError("x must be [S, T, H, P], or [tokens, H, P] with offsets")
        io = _IO.get(x.dtype)
        if io is None:
            raise ValueError("x must be float32 or bfloat16")
        if B.dim() != x.dim():
            raise ValueError("B must be [S, T, G, N], or [tokens, G, N] with offsets")
        lead, n_seq, T, max_len, n_slots = self._layer_seqs(x, offsets, slots, state, max_len)
        H, P, G, N = x.shape[-2], x.shape[-1], B.shape[-2], B.shape[-1]
        front = x.shape[:lead]
        dtype = x.dtype
        xs = self._layer_rows("x", x, x.shape, dtype, lead)
        ds = self._layer_rows("dt", dt, front + (H,), dtype, lead)
        bs = self._layer_rows("B", B, front + (G, N), dtype, lead)
        cs = self._layer_rows("C", C, front + (G, N), dtype, lead)
        zs = (0, 0) if z is None else self._layer_rows("z", z, x.shape, dtype, lead)
        for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias)):
            if t is not None:
                self._layer_dense(name, t, (H,), torch.float32)
        if state is not None:
            self._layer_dense("state", state, (n_slots, H, P, N), torch.float32)
        need = ctypes.c_size_t()
        code = self.lib.vla_ssm_workspace(self._h, n_seq, T, max_len, lead == 1, H, P, N, io, ctypes.byref(need))
        if code:
            self._layer_fail(code)
        ws = None
        if y is None or need.value:
            with _allocating(stream):
                if y is None:
                    y = torch.empty(x.shape, dtype=dtype, device=x.device)
                if need.value:
                    ws = torch.empty(need.value, dtype=torch.uint8, device=x.device)
        ys = self._layer_rows("y", y, x.shape, dtype, lead)
        code = self.lib.vla_ssm_scan(self._h, x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(),
                                     _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(state), y.data_ptr(), n_seq, T, max_len,
                                     _ptr(offsets), _ptr(slots), n_slots, H, P, G, N,
                                     _Twelve(*xs, *ds, *bs, *cs, *zs, *ys), softplus, io, _ptr(ws), need.value,
                                     self._layer_stream(stream))
        if code:
            self._layer_fail(code)
        return y

    def ssm_step(self, x, dt, A, B, C, state=None, y=None, *, D=None, z=None, dt_bias=None, softplus: bool = True,
                 slots=None, stream=None):
        """One token a sequence: x, z [S, H, P], dt [S, H], B, C [S, G, N] (see ssm_scan)."""
        if x.dim() != 3 or dt.dim() != 2 or B.dim() != 3 or C.dim() != 3:
            raise ValueError("x must be [S, H, P], dt [S, H], B and C [S, G, N]")
        one = lambda t: None if t is None else t.unsqueeze(1)   # noqa: E731
        out = self.ssm_scan(one(x), one(dt), A, one(B), one(C), state, one(y), D=D, z=one(z), dt_bias=dt_bias,
                            softplus=softplus, slots=slots, stream=stream)
        return out.squeeze(1) if y is None else y

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
        io = _IO.get(x.dtype)
        if io is None:
            raise ValueError("x must be float32 or bfloat16")
        if x.dim() < 1:
            raise ValueError("x must be [..., D]")
        if group not in (0, 128):
            raise ValueError("group must be 0 or 128")
        D = x.shape[-1]
        self._layer_dense("w", w, (D,), torch.float32)
        rows, x_row = self._layer_even("x", x, x.shape, x.dtype)
        res_row, res_io = 0, 0
        if residual is not None:
            res_io = _IO.get(residual.dtype)
            if res_io is None:
                raise ValueError("residual must be float32 or bfloat16")
            _, res_row = self._layer_even("residual", residual, x.shape, residual.dtype)
        with _allocating(stream):
            if y is None:
                y = torch.empty(x.shape, dtype=kind[1] or x.dtype, device=x.device)
            if kind[0] and scale is None:
                scale = torch.empty(x.shape[:-1] + ((-(-D // 128),) if group else ()), dtype=torch.float32,
                                    device=x.device)
        _, y_row = self._layer_even("y", y, x.shape, kind[1] or x.dtype)
        if kind[0]:
            self._layer_dense("scale", scale, x.shape[:-1] + ((-(-D // 128),) if group else ()), torch.float32)
        code = self.lib.vla_rms_norm(self._h, x.data_ptr(), w.data_ptr(), _ptr(residual), y.data_ptr(), _ptr(scale),
                                     rows, D, x_row, res_row, y_row, eps, group, kind[0], io, res_io,
                                     self._layer_stream(stream))
        if code:
            self._layer_fail(code)
        return (y, scale) if kind[0] else y

    def _layer_even(self, name, t, shape, dtype):
        """(rows, elements between rows) of a tensor whose rows are evenly spaced."""
        self._layer_check(name, t, shape, dtype)
        if t.is_contiguous():
            D = shape[-1]
            return (t.numel() // D if D else 0), D
        strides = t.stride()
        if shape[-1] > 1 and strides[-1] != 1:
            raise ValueError(f"{name}: the values of a row must be adjacent (strides {strides})")
        step = rows = None
        for i in range(len(shape) - 2, -1, -1):
            if shape[i] == 1:
                continue
            if step is None:
                step, rows = strides[i], shape[i]
            elif strides[i] != step * rows:
                raise ValueError(f"{name}: rows must be evenly spaced (strides {strides})")
            else:
                rows *= shape[i]
        return (1, shape[-1]) if step is None else (rows, step)

    def _layer_stream(self, stream):
        return (torch.cuda.current_stream(self.device) if stream is None else stream).cuda_stream

    def _layer_fail(self, code):
        from . import VlaError
        msg = self.lib.vla_last_error(self._h)
        raise VlaError(code, msg.decode() if msg else "")
