"""Head-sharded attention sublayer over the C ABI (tp_attn_* of include/tpffn.h).

PyTorch allocates the device buffers and supplies the stream; every step runs
in libtpffn.so ("7.9 Tensor and pipeline parallelism (TP, PP)", §2.2
"Attention, sharded").

    attn = TensorParallelAttention(d=3072, n_heads=24, n_kv_heads=24, head_dim=128, T_p=8)
    wqkv, wo = attn.pack(Wq, Wk, Wv, Wo)
    y, saved = attn.forward(x, B, S, wqkv, wo)
    g = attn.backward(x, B, S, wqkv, wo, saved, dy)   # dx, dwqkv, dwo
    y = attn.decode(x, cache, batch, wqkv, wo)        # serving, over a kv_cache.PagedKVCache
    y = attn.decode(x, cache, batch, *attn.pack4(Wq, Wk, Wv, Wo))  # the same from 4-bit weights
"""
from __future__ import annotations

import torch

from . import tpffn as abi
from . import weights4 as w4


class TensorParallelAttention:
    """All T_p shards of one attention sublayer on one GPU (bf16, head_dim 128)."""

    def __init__(self, d, n_heads, n_kv_heads, head_dim, T_p, causal=True, device="cuda"):
        rc, h = abi.tp_attn_plan_create(d, n_heads, n_kv_heads, head_dim, T_p, causal, abi.TP_BF16)
        abi.check(rc, "tp_attn_plan_create")
        self.plan = h
        self.d, self.H, self.Hkv, self.hd, self.T_p = d, n_heads, n_kv_heads, head_dim, T_p
        self.causal = bool(causal)
        self.device = torch.device(device)
        self.info = abi.tp_attn_plan_info(h)
        self._ws = None

    def __del__(self):
        plan = getattr(self, "plan", None)
        if plan:
            abi.tp_attn_plan_destroy(plan)
            self.plan = None

    def _bytes(self, nbytes):
        return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=self.device)

    def _stream(self):
        return torch.cuda.current_stream(self.device)

    def workspace(self, B, S, flags=0):
        need = abi.tp_attn_workspace_bytes(self.plan, B, S, flags)
        if self._ws is None or self._ws.numel() < need:
            self._ws = self._bytes(need)
        return self._ws

    # ------------------------------------------------------------ weights
    def pack(self, Wq, Wk, Wv, Wo):
        wqkv = self._bytes(abi.tp_attn_packed_bytes(self.plan, abi.TP_PACK_COLUMNS))
        wo = self._bytes(abi.tp_attn_packed_bytes(self.plan, abi.TP_PACK_ROWS))
        abi.check(abi.tp_attn_shard_weights(self.plan, Wq, Wk, Wv, Wo, wqkv, wo, self._stream()), "shard_weights")
        return wqkv, wo

    def unpack(self, wqkv, wo):
        bf = dict(dtype=torch.bfloat16, device=self.device)
        Wq = torch.empty(self.H * self.hd, self.d, **bf)
        Wk = torch.empty(self.Hkv * self.hd, self.d, **bf)
        Wv = torch.empty_like(Wk)
        Wo = torch.empty(self.d, self.H * self.hd, **bf)
        abi.check(abi.tp_attn_unshard_weights(self.plan, wqkv, wo, Wq, Wk, Wv, Wo, self._stream()),
                  "unshard_weights")
        return Wq, Wk, Wv, Wo

    def _key4(self):
        return ("attention", self.d, self.H, self.Hkv, self.hd, self.T_p)

    def _shapes4(self):
        """(rows, columns, segments) of Wq, Wk, Wv, Wo."""
        nq, nk = self.H * self.hd, self.Hkv * self.hd
        return ((nq, self.d, 1), (nk, self.d, 1), (nk, self.d, 1), (self.d, nq, self.T_p))

    def pack4(self, Wq, Wk, Wv, Wo, group=None):
        """4-bit weights for decode(), (wqkv_4, wo_4).  Each weight is a bfloat16 matrix,
        which is quantised, or a weights4.Codes4, Wo's with T_p segments.  group: 32, 64
        or 128 (the default, or the codes' own)."""
        dev = w4.device_index(self.device)
        weights = (Wq, Wk, Wv, Wo)
        group = w4.group_of(group, *weights)
        with torch.cuda.device(dev):
            c = [w4.as_codes(name, W, rows, cols, group, segments, dev)
                 for name, W, (rows, cols, segments) in zip(("Wq", "Wk", "Wv", "Wo"), weights, self._shapes4())]
            packed = [w4.Packed4(torch.empty(abi.tp_attn_packed4_bytes(self.plan, which, group), dtype=torch.uint8, device=dev),
                                 group, which, self._key4()) for which in (abi.TP_PACK_COLUMNS, abi.TP_PACK_ROWS)]
            abi.check(abi.tp_attn_shard_weights4(self.plan, group, [a.codes for a in c], [a.scales for a in c],
                                                 packed[0].data, packed[1].data, torch.cuda.current_stream()),
                      "shard_weights4")
        return tuple(packed)

    def unpack4(self, wqkv_4, wo_4):
        """The codes of Wq, Wk, Wv and Wo."""
        dev = w4.device_index(self.device)
        w4.check_packed("wqkv_4", wqkv_4, abi.TP_PACK_COLUMNS, self._key4(), dev)
        w4.check_packed("wo_4", wo_4, abi.TP_PACK_ROWS, self._key4(), dev, wqkv_4.group)
        with torch.cuda.device(dev):
            c = [w4.Codes4.empty(rows, cols, wo_4.group, segments, dev) for rows, cols, segments in self._shapes4()]
            abi.check(abi.tp_attn_unshard_weights4(self.plan, wo_4.group, wqkv_4.data, wo_4.data, [a.codes for a in c],
                                                   [a.scales for a in c], torch.cuda.current_stream()),
                      "unshard_weights4")
        return tuple(c)

    # ------------------------------------------------------------ passes
    def saved_views(self, saved, B, S):
        """(qkv [B*S, qkv_width], c [B*S, H*hd], lse [B*H, S_pad]) views of `saved`."""
        off = abi.tp_attn_saved_offsets(self.plan, B, S)
        n, W, nq = B * S, self.info["qkv_width"], self.H * self.hd
        s_pad = (S + 127) // 128 * 128
        qkv = saved[off["qkv"]:off["qkv"] + n * W * 2].view(torch.bfloat16).view(n, W)
        c = saved[off["c"]:off["c"] + n * nq * 2].view(torch.bfloat16).view(n, nq)
        lse = saved[off["lse"]:off["lse"] + B * self.H * s_pad * 4].view(torch.float32).view(B * self.H, s_pad)
        return qkv, c, lse

    def forward(self, x, B, S, wqkv, wo, fused=False, overlap=False, flags=0):
        flags |= (abi.TP_SUM_FUSED if fused else 0) | (abi.TP_SUM_OVERLAP if overlap else 0)
        y = torch.empty(B * S, self.d, dtype=torch.bfloat16, device=self.device)
        saved = self._bytes(abi.tp_attn_saved_bytes(self.plan, B, S))
        ws = self.workspace(B, S, flags)
        abi.check(abi.tp_attn_fwd(self.plan, B, S, x, wqkv, wo, y, saved, ws, ws.numel(), flags, self._stream()),
                  "tp_attn_fwd")
        return y, saved

    def backward(self, x, B, S, wqkv, wo, saved, dy, fused=False, overlap=False, flags=0):
        flags |= (abi.TP_SUM_FUSED if fused else 0) | (abi.TP_SUM_OVERLAP if overlap else 0)
        dx = torch.empty(B * S, self.d, dtype=torch.bfloat16, device=self.device)
        dwqkv = self._bytes(abi.tp_attn_packed_bytes(self.plan, abi.TP_PACK_COLUMNS))
        dwo = self._bytes(abi.tp_attn_packed_bytes(self.plan, abi.TP_PACK_ROWS))
        ws = self.workspace(B, S, flags)
        abi.check(abi.tp_attn_bwd(self.plan, B, S, x, wqkv, wo, saved, dy, dx, dwqkv, dwo, ws, ws.numel(), flags,
                                  self._stream()), "tp_attn_bwd")
        return dict(dx=dx, dwqkv=dwqkv, dwo=dwo)

    def decode(self, x, cache, batch, wqkv, wo, shared_len=0, fused=False, overlap=False, flags=0):
        """Serving pass over a PagedKVCache of this sublayer: projects the new tokens
        x [n_tokens, d] of a batch, appends their keys and values, attends to the
        cache and projects the head outputs: y [n_tokens, d].  wqkv, wo: of pack() or
        both of pack4()."""
        if cache.attn is not self:
            raise ValueError("the cache belongs to another attention sublayer")
        flags |= (abi.TP_SUM_FUSED if fused else 0) | (abi.TP_SUM_OVERLAP if overlap else 0)
        return cache.decode(x, batch, wqkv, wo, shared_len, flags=flags)

    def core_forward(self, qkv, B, S, flags=0):
        o = torch.empty(B * S, self.H * self.hd, dtype=torch.bfloat16, device=self.device)
        lse = torch.empty(B * self.H, (S + 127) // 128 * 128, dtype=torch.float32, device=self.device)
        ws = self.workspace(B, S, flags)
        abi.check(abi.tp_attn_core_fwd(self.plan, B, S, qkv, o, lse, ws, ws.numel(), flags, self._stream()),
                  "tp_attn_core_fwd")
        return o, lse

    def core_backward(self, qkv, o, lse, dO, B, S, flags=0):
        dqkv = torch.empty_like(qkv)
        ws = self.workspace(B, S, flags)
        abi.check(abi.tp_attn_core_bwd(self.plan, B, S, qkv, o, lse, dO, dqkv, ws, ws.numel(), flags,
                                       self._stream()), "tp_attn_core_bwd")
        return dqkv
