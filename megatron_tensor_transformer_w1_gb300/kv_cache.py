"""The attention sublayer's paged key/value cache over the C ABI (tp_attn_kv_*
and tp_attn_paged_fwd of include/tpffn.h).

PyTorch allocates the device buffers and supplies the stream; every step runs
in libtpffn.so.

    attn = TensorParallelAttention(d=4096, n_heads=32, n_kv_heads=8, head_dim=128, T_p=8)
    cache = PagedKVCache(attn, n_pages=4096, page_size=64, inv_freq=inv_freq)
    batch = cache.batch(cu_tokens, kv_len, page_table, n_tokens=n, max_new=1)
    q = cache.append(qkv, batch)                      # keys and values stored, q rotated
    o = cache.attend(q, batch, shared_len=0)          # [n, H * 128]
    y = attn.decode(x, cache, batch, wqkv, wo)        # both, between the projections

The cache keeps a workspace for every stream that it has been used on, and the
status words that an append needs likewise; a call that is being captured into a
graph takes its own (from the graph's memory).  So calls on different streams,
and replays beside them, have nothing in common but the pages.  Host threads on
one stream take turns: the launches of an attention call or a decode pass, which
follow one another in the stream's workspace, are made under the cache's lock.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import tpffn as abi
from . import weights4 as w4

_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing
_REFUSED = (abi.TP_ERR_INVALID, abi.TP_ERR_UNSUPPORTED, abi.TP_ERR_ALIGN)  # without any work


class KVBatch:
    """Device arrays that describe a batch of sequences (see tp_kv_batch).

    The tensors are used where they lie: their contents may change from step to
    step (a replayed graph reads them anew) as long as n_tokens and max_new
    still bound them."""

    def __init__(self, cu_tokens, kv_len, page_table, n_tokens, max_new):
        for name, t, dims in (("cu_tokens", cu_tokens, 1), ("kv_len", kv_len, 1), ("page_table", page_table, 2)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous():
                raise ValueError(f"{name}: a contiguous int32 tensor of {dims} dimension(s) is needed")
        if cu_tokens.numel() != kv_len.numel() + 1 or page_table.shape[0] != kv_len.numel():
            raise ValueError("cu_tokens has one entry more than kv_len, page_table a row for each")
        if len({cu_tokens.device, kv_len.device, page_table.device}) != 1:
            raise ValueError("the batch's tensors lie on different devices")
        n_tokens, max_new = int(n_tokens), int(max_new)
        if n_tokens < 0 or max_new < 0:
            raise ValueError("n_tokens and max_new are not negative")
        self.cu_tokens, self.kv_len, self.page_table = cu_tokens, kv_len, page_table
        self.n_seqs, self.n_tokens, self.max_new = kv_len.numel(), n_tokens, max_new
        self.device = kv_len.device
        self._index = kv_len.get_device()
        self.abi = abi.KvBatch(self.n_seqs, n_tokens, max_new, page_table.shape[1], cu_tokens.data_ptr(),
                               kv_len.data_ptr(), page_table.data_ptr())
        self._at = ctypes.addressof(self.abi)
        self._bytes = {}  # workspace sizes of the calls made with this batch


class PagedKVCache:
    """Pages of keys and values of one attention sublayer, [n_pages, n_kv_heads,
    page_size, 128] each in bf16, and the rotation of its queries and keys.

    inv_freq: float32 [rotary_dim / 2] on the device, or None for no rotation;
    k, v: existing pages (zeros are allocated otherwise)."""

    def __init__(self, attn, n_pages, page_size, k=None, v=None, inv_freq=None, interleaved=False, rotary_scale=1.0):
        shape = (int(n_pages), attn.Hkv, int(page_size), attn.hd)
        self.attn, self.n_pages, self.page_size = attn, shape[0], shape[2]
        self._width, self._q_width = attn.info["qkv_width"], attn.H * attn.hd
        self.device = attn.device if attn.device.index is not None else torch.device(
            attn.device.type, torch.cuda.current_device())
        if n_pages < 1 or page_size < 8 or page_size > 1024 or page_size & (page_size - 1):
            raise ValueError("n_pages is at least 1, page_size a power of two from 8 to 1024")
        self._index = self.device.index
        pages = []
        for name, t in (("k", k), ("v", v)):
            if t is None:
                t = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
            self._check(name, t, torch.bfloat16, shape)
            pages.append(t)
        self.k, self.v = pages
        self.inv_freq = inv_freq
        self._abi = abi.KvCache(self.k.data_ptr(), self.v.data_ptr(), shape[0], shape[2])
        self._rot = None
        if inv_freq is not None:
            if inv_freq.dim() != 1 or inv_freq.numel() % 8 or not 8 <= inv_freq.numel() <= attn.hd // 2:
                raise ValueError("inv_freq has rotary_dim / 2 entries: a multiple of 8 up to half the head width")
            self._check("inv_freq", inv_freq, torch.float32, inv_freq.shape)
            self._rot = abi.KvRotation(inv_freq.data_ptr(), 2 * inv_freq.numel(), int(bool(interleaved)),
                                       float(rotary_scale))
        self._at = ctypes.addressof(self._abi)
        self._rot_at = None if self._rot is None else ctypes.addressof(self._rot)
        self._status_bytes = abi.tp_attn_kv_workspace_bytes(attn.plan, abi.KvBatch(), self.page_size, 0,
                                                            abi.TP_KV_APPEND)
        self._statuses = {}    # of the appends, by stream
        self._workspaces = {}  # by stream
        self._last = None      # workspace of the last call, for last_device_error
        self._turn = threading.Lock()
        self._weight_bytes = [abi.tp_attn_packed_bytes(attn.plan, which)
                              for which in (abi.TP_PACK_COLUMNS, abi.TP_PACK_ROWS)]

    def _check(self, name, t, dtype, shape):
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != self._index:
            raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on {self.device} is "
                             f"needed, not {t.dtype} {tuple(t.shape)} on {t.device}")

    def _check_weights(self, name, t, nbytes):
        if not isinstance(t, torch.Tensor) or t.device != self.k.device or not t.is_contiguous() or t.nbytes < nbytes:
            raise ValueError(f"{name}: the packed weight of this sublayer is needed, {nbytes} bytes on {self.device}")

    def _out(self, name, t, shape):
        if t is None:
            return torch.empty(shape, dtype=torch.bfloat16, device=self.device)
        self._check(name, t, torch.bfloat16, shape)
        return t

    def _buffer(self, kept, need, stream):
        if _capturing():
            return torch.empty(need, dtype=torch.uint8, device=self.device)
        t = kept.get(stream)
        if t is None or t.numel() < need:
            t = kept[stream] = torch.empty(need, dtype=torch.uint8, device=self.device)
        return t

    def _workspace(self, batch, shared_len, call, flags, stream):
        key = (self.attn, self.page_size, shared_len, call, flags)
        need = batch._bytes.get(key)
        if need is None:
            need = max(16, abi.tp_attn_kv_workspace_bytes(self.attn.plan, batch.abi, self.page_size, shared_len, call,
                                                          flags))
            batch._bytes[key] = need
        return self._buffer(self._workspaces, need, stream), need

    def _done(self, rc, where, batch, ws):
        """After a call: what last_device_error reads is the workspace of the last
        one that enqueued work."""
        if rc not in _REFUSED:
            self._last = ws if batch.n_tokens and batch.n_seqs else None
        if rc:
            abi.check(rc, where)

    def _elsewhere(self, batch):
        """Whether the cache's device is not the current one."""
        if batch._index != self._index:
            raise ValueError(f"the batch lies on {batch.device}, the cache on {self.device}")
        return _current_device() != self._index

    def batch(self, cu_tokens, kv_len, page_table, n_tokens, max_new):
        return KVBatch(cu_tokens, kv_len, page_table, n_tokens, max_new)

    def append(self, qkv, batch, q=None, flags=0):
        """Stores the new tokens' keys (rotated) and values; returns the rotated
        queries [n_tokens, H * 128] (in `q` if given)."""
        if self._elsewhere(batch):
            with torch.cuda.device(self.device):
                return self.append(qkv, batch, q, flags)
        n = batch.n_tokens
        self._check("qkv", qkv, torch.bfloat16, (n, self._width))
        q = self._out("q", q, (n, self._q_width))
        st = _current_stream(self._index)
        status = self._buffer(self._statuses, self._status_bytes, st)
        rc = abi._lib.tp_attn_kv_append(self.attn.plan, self._at, batch._at, self._rot_at, qkv.data_ptr(),
                                        q.data_ptr(), status.data_ptr(), self._status_bytes, flags, st)
        self._done(rc, "tp_attn_kv_append", batch, status)
        return q

    def attend(self, q, batch, shared_len=0, lse=False, out=None, flags=0):
        """Attention of q [n_tokens, H * 128] over the cache: o, or (o, lse) with
        the rows' log2-sum-exp [n_tokens, H] if `lse`."""
        if self._elsewhere(batch):
            with torch.cuda.device(self.device):
                return self.attend(q, batch, shared_len, lse, out, flags)
        n = batch.n_tokens
        shape = (n, self._q_width)
        self._check("q", q, torch.bfloat16, shape)
        o = torch.empty_like(q) if out is None else self._out("out", out, shape)
        rows = torch.empty((n, self.attn.H), dtype=torch.float32, device=self.device) if lse else None
        st = _current_stream(self._index)
        with self._turn:
            ws, need = self._workspace(batch, shared_len, abi.TP_KV_ATTEND, 0, st)
            rc = abi._lib.tp_attn_paged_fwd(self.attn.plan, self._at, batch._at, shared_len, q.data_ptr(),
                                            o.data_ptr(), rows.data_ptr() if lse else None, ws.data_ptr(), need,
                                            flags, st)
        self._done(rc, "tp_attn_paged_fwd", batch, ws)
        return (o, rows) if lse else o

    def decode(self, x, batch, wqkv, wo, shared_len=0, out=None, flags=0):
        """The sublayer's serving pass, y [n_tokens, d] (TensorParallelAttention.decode)."""
        if self._elsewhere(batch):
            with torch.cuda.device(self.device):
                return self.decode(x, batch, wqkv, wo, shared_len, out, flags)
        a, n = self.attn, batch.n_tokens
        self._check("x", x, torch.bfloat16, (n, a.d))
        if isinstance(wqkv, w4.Packed4) or isinstance(wo, w4.Packed4):
            w4.check_packed("wqkv", wqkv, abi.TP_PACK_COLUMNS, a._key4(), self._index)
            w4.check_packed("wo", wo, abi.TP_PACK_ROWS, a._key4(), self._index, wqkv.group)
            y = self._out("out", out, (n, a.d))
            st = _current_stream(self._index)
            with self._turn:
                ws, need = self._workspace(batch, shared_len, abi.TP_KV_DECODE4, flags, st)
                rc = abi.tp_attn_decode_fwd4(a.plan, self._abi, batch.abi, self._rot, shared_len, wo.group, x, wqkv.data,
                                             wo.data, y, ws, need, flags, st)
            self._done(rc, "tp_attn_decode_fwd4", batch, ws)
            return y
        self._check_weights("wqkv", wqkv, self._weight_bytes[0])
        self._check_weights("wo", wo, self._weight_bytes[1])
        y = self._out("out", out, (n, a.d))
        st = _current_stream(self._index)
        with self._turn:
            ws, need = self._workspace(batch, shared_len, abi.TP_KV_DECODE, flags, st)
            rc = abi.tp_attn_decode_fwd(a.plan, self._abi, batch.abi, self._rot, shared_len, x, wqkv, wo, y, ws,
                                        need, flags, st)
        self._done(rc, "tp_attn_decode_fwd", batch, ws)
        return y

    def last_device_error(self):
        """Waits for the current stream and returns the status that the last call
        on this cache left on the device (TP_OK, TP_ERR_BATCH, ...): to be called
        on that call's stream, or after a wait for it."""
        if self._last is None:
            return abi.TP_OK
        with torch.cuda.device(self.device):
            return abi.tp_attn_kv_last_device_error(self.attn.plan, self._last,
                                                    torch.cuda.current_stream(self.device))
