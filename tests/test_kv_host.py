"""Host-side checks of the serving entry points (no GPU needed): refusals come
before any device work, and the binding's structures have the ABI's layout."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def abi():
    from megatron_tensor_transformer_w1_gb300 import build
    build.build()
    from megatron_tensor_transformer_w1_gb300 import tpffn
    return tpffn


A = 1 << 20  # a 16-byte-aligned address; never dereferenced on these paths


@pytest.fixture
def plan(abi):
    rc, p = abi.tp_attn_plan_create(256, 8, 2, 128, 2, True, abi.TP_BF16)
    assert rc == abi.TP_OK
    yield p
    abi.tp_attn_plan_destroy(p)


def _cache(abi, **kw):
    f = dict(k=A, v=A, n_pages=10, page_size=16)
    f.update(kw)
    return abi.KvCache(f["k"], f["v"], f["n_pages"], f["page_size"])


def _batch(abi, **kw):
    f = dict(n_seqs=3, n_tokens=4, max_new=2, max_pages=5, cu=A, kv_len=A, table=A)
    f.update(kw)
    return abi.KvBatch(f["n_seqs"], f["n_tokens"], f["max_new"], f["max_pages"], f["cu"], f["kv_len"], f["table"])


def _rot(abi, **kw):
    f = dict(inv_freq=A, rotary_dim=128, interleaved=0, scale=1.0)
    f.update(kw)
    return abi.KvRotation(f["inv_freq"], f["rotary_dim"], f["interleaved"], f["scale"])


def test_structures(abi):
    assert ctypes.sizeof(abi.KvCache) == 32 and ctypes.sizeof(abi.KvBatch) == 56
    assert ctypes.sizeof(abi.KvRotation) == 24 and abi.KvRotation.scale.offset == 16
    assert abi.tp_ffn_status_string(abi.TP_ERR_BATCH).startswith("TP_ERR_BATCH")


SHARED_BAD = [  # what differs from a good call, and the status
    (dict(cache=None), "INVALID"), (dict(batch=None), "INVALID"),
    (dict(cache=dict(k=None)), "INVALID"), (dict(cache=dict(v=None)), "INVALID"),
    (dict(cache=dict(n_pages=0)), "INVALID"), (dict(cache=dict(page_size=0)), "INVALID"),
    (dict(cache=dict(page_size=4)), "UNSUPPORTED"), (dict(cache=dict(page_size=24)), "UNSUPPORTED"),
    (dict(cache=dict(page_size=2048)), "UNSUPPORTED"), (dict(cache=dict(n_pages=2 ** 31)), "UNSUPPORTED"),
    (dict(cache=dict(k=A + 8)), "ALIGN"), (dict(cache=dict(v=A + 2)), "ALIGN"),
    (dict(batch=dict(n_seqs=-1)), "INVALID"), (dict(batch=dict(n_tokens=-1)), "INVALID"),
    (dict(batch=dict(max_new=0)), "INVALID"), (dict(batch=dict(max_pages=0)), "INVALID"),
    (dict(batch=dict(cu=None)), "INVALID"), (dict(batch=dict(kv_len=None)), "INVALID"),
    (dict(batch=dict(table=None)), "INVALID"), (dict(batch=dict(cu=A + 2)), "ALIGN"),
    (dict(batch=dict(n_tokens=2 ** 24 + 1)), "UNSUPPORTED"), (dict(batch=dict(n_seqs=2 ** 24 + 1)), "UNSUPPORTED"),
    (dict(batch=dict(max_pages=2 ** 28)), "UNSUPPORTED"),
    (dict(ws=None), "INVALID"), (dict(ws=A + 8), "ALIGN"), (dict(short=1), "INVALID"),
]


def _parts(abi, kw):
    make = lambda f, d: None if d is None else f(abi, **d)
    return make(_cache, kw.get("cache", {})), make(_batch, kw.get("batch", {}))


@pytest.mark.parametrize("kw,status", SHARED_BAD + [
    (dict(qkv=None), "INVALID"), (dict(q=None), "INVALID"), (dict(qkv=A + 4), "ALIGN"), (dict(q=A + 4), "ALIGN"),
    (dict(rot=dict(rotary_dim=24)), "INVALID"), (dict(rot=dict(rotary_dim=144)), "INVALID"),
    (dict(rot=dict(rotary_dim=-16)), "INVALID"), (dict(rot=dict(inv_freq=None)), "INVALID"),
    (dict(rot=dict(inv_freq=A + 2)), "ALIGN")])
def test_append_refusals(abi, plan, kw, status):
    cache, batch = _parts(abi, kw)
    need = abi.tp_attn_kv_workspace_bytes(plan, _batch(abi), 16, 0, abi.TP_KV_APPEND)
    rc = abi.tp_attn_kv_append(plan, cache, batch, _rot(abi, **kw.get("rot", {})), kw.get("qkv", A), kw.get("q", A),
                               kw.get("ws", A), need - kw.get("short", 0))
    assert rc == getattr(abi, "TP_ERR_" + status)


@pytest.mark.parametrize("kw,status", SHARED_BAD + [
    (dict(q=None), "INVALID"), (dict(o=None), "INVALID"), (dict(q=A + 4), "ALIGN"), (dict(o=A + 4), "ALIGN"),
    (dict(lse=A + 2), "ALIGN"), (dict(shared=-1), "INVALID"), (dict(shared=5 * 16 + 1), "INVALID")])
def test_attend_refusals(abi, plan, kw, status):
    cache, batch = _parts(abi, kw)
    need = abi.tp_attn_kv_workspace_bytes(plan, _batch(abi), 16, 0, abi.TP_KV_ATTEND)
    rc = abi.tp_attn_paged_fwd(plan, cache, batch, kw.get("shared", 0), kw.get("q", A), kw.get("o", A),
                               kw.get("lse"), kw.get("ws", A), need - kw.get("short", 0))
    assert rc == getattr(abi, "TP_ERR_" + status)


@pytest.mark.parametrize("kw,status", SHARED_BAD + [
    (dict(x=None), "INVALID"), (dict(y=None), "INVALID"), (dict(wqkv=None), "INVALID"), (dict(wo=None), "INVALID"),
    (dict(x=A + 4), "ALIGN"), (dict(shared=5 * 16 + 1), "INVALID"), (dict(flags=1 | 8), "INVALID"),
    (dict(rot=dict(rotary_dim=24)), "INVALID")])
def test_decode_refusals(abi, plan, kw, status):
    cache, batch = _parts(abi, kw)
    need = abi.tp_attn_kv_workspace_bytes(plan, _batch(abi), 16, 0, abi.TP_KV_DECODE)
    rc = abi.tp_attn_decode_fwd(plan, cache, batch, _rot(abi, **kw.get("rot", {})), kw.get("shared", 0),
                                kw.get("x", A), kw.get("wqkv", A), kw.get("wo", A), kw.get("y", A), kw.get("ws", A),
                                need - kw.get("short", 0), kw.get("flags", 0))
    assert rc == getattr(abi, "TP_ERR_" + status)


def test_null_plan_and_empty_batches(abi, plan):
    c, b = _cache(abi), _batch(abi)
    assert abi.tp_attn_kv_append(None, c, b, None, A, A, A, 1 << 30) == abi.TP_ERR_INVALID
    assert abi.tp_attn_paged_fwd(None, c, b, 0, A, A, None, A, 1 << 30) == abi.TP_ERR_INVALID
    assert abi.tp_attn_decode_fwd(None, c, b, None, 0, A, A, A, A, A, 1 << 30) == abi.TP_ERR_INVALID
    assert abi.tp_attn_kv_last_device_error(None, A) == abi.TP_ERR_INVALID
    assert abi.tp_attn_kv_last_device_error(plan, None) == abi.TP_ERR_INVALID
    assert abi.tp_attn_kv_workspace_bytes(None, b, 16, 0, abi.TP_KV_ATTEND) == 0
    assert abi.tp_attn_kv_workspace_bytes(plan, b, 24, 0, abi.TP_KV_ATTEND) == 0
    assert abi.tp_attn_kv_workspace_bytes(plan, b, 16, 0, 9) == 0
    for empty in (dict(n_seqs=0, cu=None, kv_len=None, table=None), dict(n_tokens=0, cu=None, max_new=0)):
        b = _batch(abi, **empty)
        assert abi.tp_attn_kv_append(plan, c, b, None, None, None, None, 0) == abi.TP_OK
        assert abi.tp_attn_paged_fwd(plan, c, b, 0, None, None, None, None, 0) == abi.TP_OK
        assert abi.tp_attn_decode_fwd(plan, c, b, None, 0, None, None, None, None, None, 0) == abi.TP_OK
        assert abi.tp_attn_last_launch_count(plan) == 0


def test_batch_tensors_are_checked(abi):
    from megatron_tensor_transformer_w1_gb300.kv_cache import KVBatch
    i32 = lambda *sh: torch.zeros(*sh, dtype=torch.int32)
    KVBatch(i32(4), i32(3), i32(3, 5), 7, 2)
    for cu, kv, table, n, new in ((i32(3), i32(3), i32(3, 5), 7, 2), (i32(4), i32(3), i32(2, 5), 7, 2),
                                  (i32(4).long(), i32(3), i32(3, 5), 7, 2), (i32(4), i32(3).float(), i32(3, 5), 7, 2),
                                  (i32(4), i32(3), i32(3, 10)[:, ::2], 7, 2), (i32(4), i32(3), i32(15), 7, 2),
                                  (i32(8)[::2], i32(3), i32(3, 5), 7, 2), (i32(4), i32(3), i32(3, 5), -1, 2),
                                  ([0, 1, 2, 3], i32(3), i32(3, 5), 7, 2)):
        with pytest.raises(ValueError):
            KVBatch(cu, kv, table, n, new)
