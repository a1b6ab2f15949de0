"""How PagedKVCache hands buffers to the library, on the CPU: the library's calls
are replaced by recorders, the device's streams by numbers."""
import threading
import time
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture
def host(monkeypatch):
    from megatron_tensor_transformer_w1_gb300 import build
    build.build()
    from megatron_tensor_transformer_w1_gb300 import kv_cache, tpffn as abi

    class HostCache(kv_cache.PagedKVCache):
        def _elsewhere(self, batch):
            return False

        def _check(self, name, t, dtype, shape):
            assert t.dtype is dtype and t.shape == shape and t.is_contiguous()

    rc, plan = abi.tp_attn_plan_create(256, 8, 2, 128, 2, True, abi.TP_BF16)
    assert rc == abi.TP_OK
    attn = type("Sublayer", (), dict(plan=plan, H=8, Hkv=2, hd=128, d=256, info=abi.tp_attn_plan_info(plan),
                                     device=torch.device("cpu", 0)))()
    weights = [torch.zeros(abi.tp_attn_packed_bytes(plan, which), dtype=torch.uint8) for which in (0, 1)]
    env = SimpleNamespace(abi=abi, stream=1, capturing=False, status=abi.TP_OK, calls=[], attn=attn, weights=weights,
                          during=lambda at: None)
    monkeypatch.setattr(kv_cache, "_current_stream", lambda index: env.stream)
    monkeypatch.setattr(kv_cache, "_capturing", lambda: env.capturing)

    def append(plan, cache, batch, rot, qkv, q, ws, ws_bytes, flags, stream):
        env.calls.append((stream, ws, ws_bytes))
        env.during(ws)
        return env.status

    def attend(plan, cache, batch, shared, q, o, lse, ws, ws_bytes, flags, stream):
        return append(plan, cache, batch, None, q, o, ws, ws_bytes, flags, stream)

    def decode(plan, cache, batch, rot, shared, x, wqkv, wo, y, ws, ws_bytes, flags, stream):
        return append(plan, cache, batch, None, x, y, ws.data_ptr(), ws_bytes, flags, stream)
    monkeypatch.setattr(abi, "_lib", SimpleNamespace(
        tp_attn_kv_append=append, tp_attn_paged_fwd=attend, tp_attn_packed_bytes=abi._lib.tp_attn_packed_bytes,
        tp_attn_kv_workspace_bytes=abi._lib.tp_attn_kv_workspace_bytes,
        tp_ffn_status_string=abi._lib.tp_ffn_status_string))
    monkeypatch.setattr(abi, "tp_attn_decode_fwd", decode)
    env.cache = HostCache(attn, 10, 16)
    i32 = lambda *sh: torch.zeros(*sh, dtype=torch.int32)
    env.batch = env.cache.batch(i32(4), i32(3), i32(3, 5), 4, 2)
    env.rows = lambda width: torch.zeros(4, width, dtype=torch.bfloat16)
    yield env
    monkeypatch.undo()
    abi.tp_attn_plan_destroy(plan)


def test_append_has_a_status_buffer_of_its_stream_and_of_its_capture(host):
    qkv = host.rows(12 * 128)
    kept = []  # what a captured call was given stays with its graph

    def call(stream, capturing=False):
        host.stream, host.capturing = stream, capturing
        host.cache.append(qkv, host.batch)
        kept.append(host.cache._last)
        assert host.calls[-1][0] == stream
        return host.calls[-1][1]
    a, b = call(1), call(2)
    assert a != b and call(1) == a and call(2) == b
    c, d = call(1, True), call(1, True)
    assert len({a, b, c, d}) == 4 and call(1) == a
    need = host.abi.tp_attn_kv_workspace_bytes(host.attn.plan, host.batch.abi, 16, 0, host.abi.TP_KV_APPEND)
    assert all(size == need for _, _, size in host.calls)


@pytest.mark.parametrize("what", ["attend", "decode", "both"])
def test_two_threads_on_one_stream_take_turns(host, what):
    """A call is several launches: in one workspace, those of two calls must not mix."""
    inside, met = [], []

    def during(ws):
        inside.append(ws)
        time.sleep(0.002)  # the other thread's turn, as where a call into the library lets go of the interpreter
        met.append(inside.count(ws) > 1)
        inside.remove(ws)
    host.during = during
    q, x = host.rows(8 * 128), host.rows(256)

    def work(decode):
        for _ in range(20):
            if decode:
                host.cache.decode(x, host.batch, *host.weights)
            else:
                host.cache.attend(q, host.batch)
    threads = [threading.Thread(target=work, args=(what == "decode" or (what == "both" and i),)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(met) == 40 and not any(met)


def test_decode_checks_its_weights(host):
    """Packed weights of another sublayer, layout or place do not reach the kernels."""
    x = host.rows(256)
    wqkv, wo = host.weights
    y = host.cache.decode(x, host.batch, wqkv, wo)
    assert y.shape == (4, 256) and len(host.calls) == 1
    for t in (None, wqkv[:-16], torch.zeros(2 * wqkv.numel(), dtype=torch.uint8)[::2], wqkv.to("meta"),
              wqkv.data_ptr()):
        with pytest.raises(ValueError, match="wqkv"):
            host.cache.decode(x, host.batch, t, wo)
    for t in (None, wo[:-16], wo.to("meta")):
        with pytest.raises(ValueError, match="wo"):
            host.cache.decode(x, host.batch, wqkv, t)
    assert len(host.calls) == 1
    host.cache.decode(x, host.batch, wqkv.view(torch.bfloat16), wo)  # their bytes count, not their type
    assert len(host.calls) == 2


def test_workspace_of_a_batch_without_work():
    """A batch without sequences or tokens needs no sizes: whatever its bounds say,
    the call is made and its workspace is that of no work."""
    from megatron_tensor_transformer_w1_gb300 import build
    build.build()
    from megatron_tensor_transformer_w1_gb300 import tpffn as abi
    rc, plan = abi.tp_attn_plan_create(256, 8, 2, 128, 2, True, abi.TP_BF16)
    assert rc == abi.TP_OK
    cache = abi.KvCache(1 << 20, 1 << 20, 10, 16)
    try:
        for n_seqs, n_tokens in ((0, 4), (3, 0), (0, 0)):
            sizes = []
            for max_new, max_pages in ((0, 5), (-1, 5), (-(2 ** 40), 5), (0, -1), (0, -(2 ** 40)), (2 ** 40, 5)):
                b = abi.KvBatch(n_seqs, n_tokens, max_new, max_pages, None, None, None)
                assert abi.tp_attn_paged_fwd(plan, cache, b, 0, None, None, None, None, 0) == abi.TP_OK
                sizes.append([abi.tp_attn_kv_workspace_bytes(plan, b, 16, 0, call)
                              for call in (abi.TP_KV_APPEND, abi.TP_KV_ATTEND, abi.TP_KV_DECODE)])
            assert all(s == sizes[0] for s in sizes), sizes
            assert max(max(s) for s in sizes) < 1 << 26
    finally:
        abi.tp_attn_plan_destroy(plan)


@pytest.mark.parametrize("what", ["append", "attend", "decode"])
def test_a_refused_call_leaves_the_last_status_alone(host, what):
    """last_device_error reads what the last call wrote: one that was refused wrote nothing,
    one that ran and failed did."""
    def call():
        if what == "append":
            host.cache.append(host.rows(12 * 128), host.batch)
        elif what == "attend":
            host.cache.attend(host.rows(8 * 128), host.batch)
        else:
            host.cache.decode(host.rows(256), host.batch, *host.weights)
        return host.cache._last
    for status in ("INVALID", "UNSUPPORTED", "ALIGN"):
        host.status = getattr(host.abi, "TP_ERR_" + status)
        with pytest.raises(host.abi.TPFFNError):
            call()
        assert host.cache._last is None
    host.status = host.abi.TP_OK
    host.stream = 5
    good = call()
    assert good.data_ptr() == host.calls[-1][1]
    host.stream, host.status = 6, host.abi.TP_ERR_INVALID
    with pytest.raises(host.abi.TPFFNError):
        call()
    assert host.cache._last is good
    for status in ("BATCH", "TIMEOUT"):
        host.status = getattr(host.abi, "TP_ERR_" + status)
        with pytest.raises(host.abi.TPFFNError):
            call()
        assert host.cache._last.data_ptr() == host.calls[-1][1]
