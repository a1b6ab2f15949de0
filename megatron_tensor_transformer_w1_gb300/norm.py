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

import torch

from . import tpffn as abi
from .weights4 import Scratch, check_tensor, full_device

_KINDS = {"rms": abi.TP_NORM_RMS, "layer": abi.TP_NORM_LAYER}
_DTYPES = {"f32": (abi.TP_F32, torch.float32), "bf16": (abi.TP_BF16, torch.bfloat16)}


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
        self.device = torch.device(device)
        self._scratch = Scratch(self.device)

    def _rows(self, name, t, n, dev):
        check_tensor(name, t, self.torch_dtype, (n, self.d), dev)

    def _vectors(self, dev, after, before, **vectors):
        for name, t in vectors.items():
            if t is None:
                continue
            if not (before if name.endswith("before") else after):
                raise ValueError(f"{name} belongs to a norm that there is not")
            check_tensor(name, t, self.torch_dtype, (self.d,), dev)

    def _gates(self, gate, n, dev):
        if gate is None:
            return 0
        if not isinstance(gate, torch.Tensor) or gate.dim() != 2 or gate.shape[0] < 1 or n % gate.shape[0]:
            raise ValueError("gate: [gates, d] with a number of gates that divides the tokens")
        check_tensor("gate", gate, self.torch_dtype, gate.shape[:1] + (self.d,), dev)
        return gate.shape[0]

    def forward(self, x, b=None, w_after=None, c_after=None, gate=None, w_before=None, c_before=None, save=True,
                r_out=None):
        """(r, out, stats): the residual stream [n, d] behind the sublayer (in r_out
        if given, which may be x), the next sublayer's input (None without `before`)
        and, if `save`, what backward() needs besides."""
        dev = full_device(self.device)
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x: a matrix [tokens, d] is needed")
        n = x.shape[0]
        self._rows("x", x, n, dev)
        if b is not None:
            self._rows("b", b, n, dev)
        elif self.after or gate is not None:
            raise ValueError("b, the sublayer's output, is needed for its norm and gate")
        self._vectors(dev, self.after, self.before, w_after=w_after, c_after=c_after, w_before=w_before, c_before=c_before)
        gates = self._gates(gate, n, dev)
        if r_out is not None:
            self._rows("r_out", r_out, n, dev)
        with torch.cuda.device(dev):
            r = torch.empty_like(x) if r_out is None else r_out
            out = torch.empty_like(x) if self.before else None
            stats = torch.empty(n, 4, dtype=torch.float32, device=dev) if save and (self.before or self.after) else None
            abi.check(abi.tp_norm_fwd(self.abi, n, gates, x, b, w_after, c_after, gate, w_before, c_before, r, out, stats,
                                      torch.cuda.current_stream()), "tp_norm_fwd")
        return r, out, stats

    def backward(self, b, r, stats, dr, dout=None, w_after=None, c_after=None, gate=None, w_before=None,
                 shift_before=False):
        """Gradients from dr [n, d], that of r (None: zeros), and dout, that of out, given
        forward()'s b, r and stats: a dict of dx, db (None where there was no b), dgate,
        dw_after, dc_after, dw_before and dc_before, None for what was not given.
        shift_before: there was a c_before."""
        dev = full_device(self.device)
        first = next((t for t in (dr, dout, b) if t is not None), None)
        if not isinstance(first, torch.Tensor) or first.dim() != 2:
            raise ValueError("dr, dout: matrices [tokens, d] are needed")
        n = first.shape[0]
        if (dout is None) == self.before:
            raise ValueError("dout belongs to `before`")
        for name, t in (("b", b), ("dr", dr), ("dout", dout)):
            if t is not None:
                self._rows(name, t, n, dev)
        if b is None and (self.after or gate is not None):
            raise ValueError("b, the sublayer's output, is needed for its norm and gate")
        if self.before:
            self._rows("r", r, n, dev)
        if self.before or self.after:
            check_tensor("stats", stats, torch.float32, (n, 4), dev)
        self._vectors(dev, self.after, self.before, w_after=w_after, c_after=c_after, w_before=w_before)
        if shift_before and not self.before:
            raise ValueError("c_before belongs to a norm that there is not")
        gates = self._gates(gate, n, dev)
        with torch.cuda.device(dev), self._scratch.turn:
            st = torch.cuda.current_stream()
            new = torch.empty if n else torch.zeros
            row = lambda want: new(n, self.d, dtype=self.torch_dtype, device=dev) if want else None
            vector = lambda want: new(self.d, dtype=self.torch_dtype, device=dev) if want else None
            g = dict(dx=row(True), db=row(b is not None), dgate=None if gate is None else torch.empty_like(gate),
                     dw_after=vector(w_after is not None), dc_after=vector(c_after is not None),
                     dw_before=vector(w_before is not None), dc_before=vector(shift_before))
            if not n and gate is not None:
                g["dgate"].zero_()
            ws = self._scratch.take(abi.tp_norm_workspace_bytes(self.abi, n, gates), st)
            abi.check(abi.tp_norm_bwd(self.abi, n, gates, b, r if self.before else None,
                                      stats if self.before or self.after else None, w_after, c_after, gate, w_before,
                                      dr, dout, g["dx"], g["db"], g["dw_after"], g["dc_after"], g["dgate"],
                                      g["dw_before"], g["dc_before"], ws, ws.numel(), st), "tp_norm_bwd")
        return g
