"""A thin convenience layer over the C ABI: PyTorch allocates the device
buffers and supplies the stream; every computation is a libtpffn.so call.

    ffn = TensorParallelFFN(d=4096, d_ff=14336, T_p=8, act="swiglu", dtype="bf16")
    w13p, w2p = ffn.pack(W1, W2, W3)
    y, saved = ffn.forward(x, w13p, w2p)
    grads = ffn.backward(x, w13p, w2p, saved, dy)
    w13_4, w2_4 = ffn.pack4(W1, W2, W3)               # serving from 4-bit weights
    y = ffn.forward4(x, w13_4, w2_4)
"""
from __future__ import annotations

import torch

from . import tpffn as abi
from . import weights4 as w4

_ACTS = {"none": abi.TP_ACT_NONE, "gelu_tanh": abi.TP_ACT_GELU_TANH, "swiglu": abi.TP_ACT_SWIGLU}
_DTYPES = {"f32": (abi.TP_F32, torch.float32), "bf16": (abi.TP_BF16, torch.bfloat16)}


class TensorParallelFFN:
    """All T_p shards of one tensor-parallel FFN (or W_O projection) on one GPU."""

    def __init__(self, d, d_ff, T_p, act="gelu_tanh", dtype="bf16", device="cuda", n_heads=None,
                 n_kv_heads=None, head_dim=None):
        self.act_name = act
        self.dtype_code, self.torch_dtype = _DTYPES[dtype]
        self.device = torch.device(device)
        if act == "none" and n_heads is not None:
            rc, h = abi.tp_attn_out_plan_create(d, n_heads, n_kv_heads or n_heads, head_dim, T_p, self.dtype_code)
        else:
            rc, h = abi.tp_ffn_plan_create(d, d_ff, T_p, _ACTS[act], self.dtype_code)
        abi.check(rc, "plan_create")
        self.plan = h
        self.info = abi.tp_ffn_plan_info(h)
        self.d, self.d_ff, self.T_p = self.info["d"], self.info["d_ff"], self.info["T_p"]
        self._ws = None
        self._scratch4 = w4.Scratch()
        self._key4 = ("ffn", act, self.d, self.d_ff, self.T_p)
        self._need4 = {}  # workspace bytes by device and tokens

    def __del__(self):
        plan = getattr(self, "plan", None)
        if plan:
            abi.tp_ffn_plan_destroy(plan)
            self.plan = None

    # ------------------------------------------------------------ buffers
    def _bytes(self, nbytes):
        return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=self.device)

    def workspace(self, n_tokens, flags=0):
        need = abi.tp_ffn_workspace_bytes(self.plan, n_tokens, flags)
        if self._ws is None or self._ws.numel() < need:
            self._ws = self._bytes(need)
        return self._ws

    def _stream(self):
        return torch.cuda.current_stream(self.device)

    # ------------------------------------------------------------ packing
    def pack(self, W1, W2, W3=None):
        st = self._stream()
        w13p = None
        if self.act_name != "none":
            w13p = self._bytes(abi.tp_ffn_packed_bytes(self.plan, abi.TP_PACK_COLUMNS))
            abi.check(abi.tp_ffn_shard_columns(self.plan, W1, W3, w13p, st), "shard_columns")
        w2p = self._bytes(abi.tp_ffn_packed_bytes(self.plan, abi.TP_PACK_ROWS))
        abi.check(abi.tp_ffn_shard_rows(self.plan, W2, w2p, st), "shard_rows")
        return w13p, w2p

    def unpack_columns(self, w13p):
        st = self._stream()
        W1 = torch.empty(self.d_ff, self.d, dtype=self.torch_dtype, device=self.device)
        W3 = torch.empty_like(W1) if self.act_name == "swiglu" else None
        abi.check(abi.tp_ffn_unshard_columns(self.plan, w13p, W1, W3, st), "unshard_columns")
        return W1, W3

    def unpack_rows(self, w2p):
        st = self._stream()
        W2 = torch.empty(self.d, self.d_ff, dtype=self.torch_dtype, device=self.device)
        abi.check(abi.tp_ffn_unshard_rows(self.plan, w2p, W2, st), "unshard_rows")
        return W2

    # ------------------------------------------------------------ 4-bit weights
    def _no_up4(self):
        if self.act_name == "none":
            raise ValueError("this sublayer has no first matrix")

    def pack4(self, W1, W2, W3=None, group=None):
        """4-bit weights for forward4, (w13_4, w2_4).  Each of W1, W2, W3 (W1 and W3
        None where the sublayer has none) is a bfloat16 matrix, which is quantised, or
        a weights4.Codes4, W2's with T_p segments.  group: 32, 64 or 128 (the default,
        or the codes' own)."""
        if self.dtype_code != abi.TP_BF16:
            raise ValueError("4-bit weights need a bf16 sublayer")
        dev = w4.device_index(self.device)
        group = w4.group_of(group, W1, W2, W3)
        gated = self.act_name == "swiglu"
        if (W1 is None) != (self.act_name == "none") or (W3 is None) == gated:
            raise ValueError("W1 belongs to sublayers with an activation, W3 to swiglu")
        with torch.cuda.device(dev):
            st = torch.cuda.current_stream()
            up = None
            if W1 is not None:
                c1 = w4.as_codes("W1", W1, self.d_ff, self.d, group, 1, dev)
                c3 = w4.as_codes("W3", W3, self.d_ff, self.d, group, 1, dev) if gated else None
                up = torch.empty(abi.tp_ffn_packed4_bytes(self.plan, abi.TP_PACK_COLUMNS, group), dtype=torch.uint8, device=dev)
                abi.check(abi.tp_ffn_shard_columns4(self.plan, group, c1.codes, c1.scales, c3 and c3.codes,
                                                    c3 and c3.scales, up, st), "shard_columns4")
                up = w4.Packed4(up, group, abi.TP_PACK_COLUMNS, self._key4)
            c2 = w4.as_codes("W2", W2, self.d, self.d_ff, group, self.T_p, dev)
            down = torch.empty(abi.tp_ffn_packed4_bytes(self.plan, abi.TP_PACK_ROWS, group), dtype=torch.uint8, device=dev)
            abi.check(abi.tp_ffn_shard_rows4(self.plan, group, c2.codes, c2.scales, down, st), "shard_rows4")
        return up, w4.Packed4(down, group, abi.TP_PACK_ROWS, self._key4)

    def unpack4_columns(self, w13_4):
        """The codes of W1 and of W3 (None without it)."""
        self._no_up4()
        dev = w4.device_index(self.device)
        w4.check_packed("w13_4", w13_4, abi.TP_PACK_COLUMNS, self._key4, dev)
        with torch.cuda.device(dev):
            c = [w4.Codes4.empty(self.d_ff, self.d, w13_4.group, 1, dev) for _ in range(2 if self.act_name == "swiglu" else 1)]
            c1, c3 = c[0], (c[1] if len(c) > 1 else None)
            abi.check(abi.tp_ffn_unshard_columns4(self.plan, w13_4.group, w13_4.data, c1.codes, c1.scales,
                                                  c3 and c3.codes, c3 and c3.scales, torch.cuda.current_stream()),
                      "unshard_columns4")
        return c1, c3

    def unpack4_rows(self, w2_4):
        """The codes of W2, with T_p segments."""
        dev = w4.device_index(self.device)
        w4.check_packed("w2_4", w2_4, abi.TP_PACK_ROWS, self._key4, dev)
        with torch.cuda.device(dev):
            c = w4.Codes4.empty(self.d, self.d_ff, w2_4.group, self.T_p, dev)
            abi.check(abi.tp_ffn_unshard_rows4(self.plan, w2_4.group, w2_4.data, c.codes, c.scales,
                                               torch.cuda.current_stream()), "unshard_rows4")
        return c

    def forward4(self, x, w13_4, w2_4, b1=None, b2=None, out=None, flags=0):
        """y [n, d] of forward() for inference, from the 4-bit weights of pack4()
        (w13_4 None where the sublayer has no first matrix)."""
        index = w4.device_index(self.device)
        if w4.current_device() != index:
            with torch.cuda.device(index):
                return self.forward4(x, w13_4, w2_4, b1, b2, out, flags)
        none = self.act_name == "none"
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x: a bfloat16 matrix [tokens, features] is needed")
        n = x.shape[0]
        w4.check_tensor("x", x, w4.BF16, (n, self.d_ff if none else self.d), index)
        w4.check_packed("w2_4", w2_4, abi.TP_PACK_ROWS, self._key4, index)
        if not none:
            w4.check_packed("w13_4", w13_4, abi.TP_PACK_COLUMNS, self._key4, index, w2_4.group)
        elif w13_4 is not None:
            self._no_up4()
        if b1 is not None:
            w4.check_tensor("b1", b1, w4.BF16, (self.d_ff,), index)
        if b2 is not None:
            w4.check_tensor("b2", b2, w4.BF16, (self.d,), index)
        if out is None:
            out = torch.empty((n, self.d), dtype=w4.BF16, device=index)
        else:
            w4.check_tensor("out", out, w4.BF16, (n, self.d), index)
        need = self._need4.get((index, n))
        if need is None:
            need = self._need4[index, n] = max(16, abi.tp_ffn_workspace4_bytes(self.plan, n, flags))
        with self._scratch4.turn:
            st = w4.current_stream(index)
            ws = self._scratch4.take(need, index, st)
            rc = abi._lib.tp_ffn_fwd4(self.plan, w2_4.group, n, x.data_ptr(), None if none else w13_4.data.data_ptr(),
                                      w2_4.data.data_ptr(), None if b1 is None else b1.data_ptr(),
                                      None if b2 is None else b2.data_ptr(), out.data_ptr(), ws.data_ptr(), need, flags, st)
        if rc:
            abi.check(rc, "tp_ffn_fwd4")
        return out

    # ------------------------------------------------------------ passes
    def forward(self, x, w13p, w2p, b1=None, b2=None, save=True, fused=False, want_partials=False, flags=0,
                overlap=False):
        n = x.shape[0]
        flags |= abi.TP_SUM_FUSED if fused else 0
        flags |= abi.TP_SUM_OVERLAP if overlap else 0
        st = self._stream()
        y = torch.empty(n, self.d, dtype=self.torch_dtype, device=self.device)
        saved = self._bytes(abi.tp_ffn_saved_bytes(self.plan, n)) if save and self.act_name != "none" else None
        part = torch.empty(self.T_p, n, self.d, dtype=torch.float32, device=self.device) if want_partials else None
        ws = self.workspace(n, flags)
        abi.check(abi.tp_ffn_fwd(self.plan, n, x, w13p, w2p, b1, b2, y, part, saved, ws, ws.numel(), flags, st),
                  "fwd")
        return y, saved, part

    def backward(self, x, w13p, w2p, saved, dy, fused=False, want_partials=False, bias=False, flags=0,
                 overlap=False):
        n = dy.shape[0]
        flags |= abi.TP_SUM_FUSED if fused else 0
        flags |= abi.TP_SUM_OVERLAP if overlap else 0
        st = self._stream()
        d_in = self.d_ff if self.act_name == "none" else self.d
        dx = torch.empty(n, d_in, dtype=self.torch_dtype, device=self.device)
        part = torch.empty(self.T_p, n, self.d, dtype=torch.float32, device=self.device) if want_partials else None
        dw13p = None
        if self.act_name != "none":
            dw13p = self._bytes(abi.tp_ffn_packed_bytes(self.plan, abi.TP_PACK_COLUMNS))
        dw2p = self._bytes(abi.tp_ffn_packed_bytes(self.plan, abi.TP_PACK_ROWS))
        db1 = torch.empty(self.d_ff, dtype=self.torch_dtype, device=self.device) if bias and self.act_name == "gelu_tanh" else None
        db2 = torch.empty(self.d, dtype=self.torch_dtype, device=self.device) if bias else None
        ws = self.workspace(n, flags)
        abi.check(abi.tp_ffn_bwd(self.plan, n, x, w13p, w2p, saved, dy, dx, part, dw13p, dw2p, db1, db2, ws,
                                 ws.numel(), flags, st), "bwd")
        return dict(dx=dx, dx_partials=part, dw13p=dw13p, dw2p=dw2p, db1=db1, db2=db2)
