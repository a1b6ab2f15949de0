"""The norms around a block's sublayers with the gate, the residual scale and the
residual sum, over the C ABI (tp_norm_* of include/tpffn.h).

    norm = SublayerNorm(d=4096, kind="rms", before=True, after=True, scale=0.5)
    r, out, stats = norm.forward(x, b, w_after=wa, gate=g, w_before=wb)
    grads = norm.backward(b, r, stats, dr, dout, w_after=wa, gate=g, w_before=wb)

x is the residual stream and b the output of the sublayer (TensorParallelFFN,
TensorParallelAttention) that it is added to; r the stream behind it and out the
input of the next sublayer:

    u = norm(b) * w_after + c_after (after) or b;  r = x + scale * gate * u;
    out = norm(r) * w_before + c_before (before)

PyTorch allocates the device buffers and supplies the stream; every step runs
in libtpffn.so.
"""
from __future__ import annotations

import ctypes

import torch

from . import tpffn as abi
from .weights4 import Scratch, check_tensor, current_device, current_stream, device_index

_KINDS = {"rms": abi.TP_NORM_RMS, "layer": abi.TP_NORM_LAYER}
_DTYPES = {"f32": (abi.TP_F32, torch.float32), "bf16": (abi.TP_BF16, torch.bfloat16)}


def _at(t):
    return None if t is None else t.data_ptr()


class SublayerNorm:
    """What stands between two sublayers of width d (a multiple of 8 up to 8192)."""

    def __init__(self, d, kind="rms", before=True, after=False, eps=1e-5, scale=1.0, dtype="bf16", device="cuda"):
        if kind not in _KINDS or dtype not in _DTYPES:
            raise ValueError(f"kind is one of {tuple(_KINDS)}, dtype of {tuple(_DTYPES)}")
        if not 8 <= d <= 8192 or d % 8:
            raise ValueError("d is a multiple of 8 up to 8192")
        code, self.torch_dtype = _DTYPES[dtype]
        self.d, self.before, self.after = int(d), bool(before), bool(after)
        self.abi = abi.Norm(self.d, _KINDS[kind], code, int(self.before), int(self.after), float(eps), float(scale))
        self._at = ctypes.addressof(self.abi)
        self.device = torch.device(device)
        self._scratch, self._need = Scratch(), {}  # workspace bytes by device, tokens and gates

    def _vectors(self, index, **vectors):
        for name, t in vectors.items():
            if t is None:
                continue
            if not (self.before if name.endswith("before") else self.after):
                raise ValueError(f"{name} belongs to a norm that there is not")
            check_tensor(name, t, self.torch_dtype, (self.d,), index)

    def _gates(self, gate, n, index):
        if gate is None:
            return 0
        if not isinstance(gate, torch.Tensor) or gate.dim() != 2 or gate.shape[0] < 1 or n % gate.shape[0]:
            raise ValueError("gate: [gates, d] with a number of gates that divides the tokens")
        check_tensor("gate", gate, self.torch_dtype, (gate.shape[0], self.d), index)
        return gate.shape[0]

    def forward(self, x, b=None, w_after=None, c_after=None, gate=None, w_before=None, c_before=None, save=True,
                r_out=None):
        """(r, out, stats): the residual stream [n, d] behind the sublayer (in r_out
        if given, which may be x), the next sublayer's input (None without `before`)
        and, if `save`, what backward() needs besides."""
        index = device_index(self.device)
        if current_device() != index:
            with torch.cuda.device(index):
                return self.forward(x, b, w_after, c_after, gate, w_before, c_before, save, r_out)
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x: a matrix [tokens, d] is needed")
        n, t = x.shape[0], self.torch_dtype
        shape = (n, self.d)
        check_tensor("x", x, t, shape, index)
        if b is not None:
            check_tensor("b", b, t, shape, index)
        elif self.after or gate is not None:
            raise ValueError("b, the sublayer's output, is needed for its norm and gate")
        self._vectors(index, w_after=w_after, c_after=c_after, w_before=w_before, c_before=c_before)
        gates = self._gates(gate, n, index)
        if r_out is None:
            r = torch.empty_like(x)
        else:
            check_tensor("r_out", r_out, t, shape, index)
            r = r_out
        out = torch.empty_like(x) if self.before else None
        stats = torch.empty((n, 4), dtype=torch.float32, device=index) if save and (self.before or self.after) else None
        rc = abi._lib.tp_norm_fwd(self._at, n, gates, x.data_ptr(), _at(b), _at(w_after), _at(c_after), _at(gate),
                                  _at(w_before), _at(c_before), r.data_ptr(), _at(out), _at(stats), current_stream(index))
        if rc:
            abi.check(rc, "tp_norm_fwd")
        return r, out, stats

    def backward(self, b, r, stats, dr, dout=None, w_after=None, c_after=None, gate=None, w_before=None,
                 shift_before=False):
        """Gradients from dr [n, d], that of r (None: zeros), and dout, that of out, given
        forward()'s b, r and stats: a dict of dx, db (None where there was no b), dgate,
        dw_after, dc_after, dw_before and dc_before, None for what was not given.
        shift_before: there was a c_before."""
        index = device_index(self.device)
        if current_device() != index:
            with torch.cuda.device(index):
                return self.backward(b, r, stats, dr, dout, w_after, c_after, gate, w_before, shift_before)
        first = dr if dr is not None else dout if dout is not None else b
        if not isinstance(first, torch.Tensor) or first.dim() != 2:
            raise ValueError("dr, dout: matrices [tokens, d] are needed")
        n, t = first.shape[0], self.torch_dtype
        shape = (n, self.d)
        if (dout is None) == self.before:
            raise ValueError("dout belongs to `before`")
        for name, a in (("b", b), ("dr", dr), ("dout", dout)):
            if a is not None:
                check_tensor(name, a, t, shape, index)
        if b is None and (self.after or gate is not None):
            raise ValueError("b, the sublayer's output, is needed for its norm and gate")
        if self.before:
            check_tensor("r", r, t, shape, index)
        if self.before or self.after:
            check_tensor("stats", stats, torch.float32, (n, 4), index)
        self._vectors(index, w_after=w_after, c_after=c_after, w_before=w_before)
        if shift_before and not self.before:
            raise ValueError("c_before belongs to a norm that there is not")
        gates = self._gates(gate, n, index)
        new = torch.empty if n else torch.zeros

        def like(want, shape):
            return new(shape, dtype=t, device=index) if want else None
        one = (self.d,)
        g = dict(dx=like(True, shape), db=like(b is not None, shape), dgate=like(gate is not None, (gates, self.d)),
                 dw_after=like(w_after is not None, one), dc_after=like(c_after is not None, one),
                 dw_before=like(w_before is not None, one), dc_before=like(shift_before, one))
        need = self._need.get((index, n, gates))
        if need is None:
            need = self._need[index, n, gates] = max(16, abi.tp_norm_workspace_bytes(self.abi, n, gates))
        with self._scratch.turn:
            st = current_stream(index)
            ws = self._scratch.take(need, index, st)
            rc = abi._lib.tp_norm_bwd(self._at, n, gates, _at(b), _at(r) if self.before else None,
                                      _at(stats) if self.before or self.after else None, _at(w_after), _at(c_after),
                                      _at(gate), _at(w_before), _at(dr), _at(dout), _at(g["dx"]), _at(g["db"]),
                                      _at(g["dw_after"]), _at(g["dc_after"]), _at(g["dgate"]), _at(g["dw_before"]),
                                      _at(g["dc_before"]), ws.data_ptr(), need, st)
        if rc:
            abi.check(rc, "tp_norm_bwd")
        return g
