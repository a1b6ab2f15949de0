"""Calls on one cache at the same time: each reports its own status."""
import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_kv_cache import HD, _cache, _modules

pytestmark = pytest.mark.gpu


def _two_appends():
    """A cache, a large batch with a page outside it, and a good one of other sequences."""
    s = ref.make_batch([40] * 30, [8] * 30, 2, 16, seed=61, junk=0.0)
    cache, _ = _cache(s, 4, 2)
    table = s["table"].clone()
    table[14, 0] = 1  # (its first new token's page)
    table[14, 1] = s["n_pages"]
    i32 = dict(dtype=torch.int32, device="cuda")
    bad = cache.batch(torch.arange(0, 29 * 40 + 1, 40, **i32), s["kv_len"][:29].clone(), table[:29].contiguous(), 1160, 40)
    good = cache.batch(torch.tensor([0, 1], **i32), s["kv_len"][29:].clone(), s["table"][29:].contiguous(), 1, 1)
    qkv = torch.ones(1160, 8 * HD, dtype=torch.bfloat16, device="cuda")
    return _modules()[0], cache, bad, good, qkv


@pytest.mark.parametrize("bad_last", [True, False])
def test_appends_on_two_streams_report_their_own_status(bad_last):
    """The call that is made last runs first: the other stream is busy meanwhile."""
    abi, cache, bad, good, qkv = _two_appends()
    calls = [(good, qkv[:1]), (bad, qkv)] if bad_last else [(bad, qkv), (good, qkv[:1])]
    torch.cuda.synchronize()
    busy, free = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(20_000_000)  # some ten milliseconds
        cache.append(calls[0][1], calls[0][0])
    with torch.cuda.stream(free):
        cache.append(calls[1][1], calls[1][0])
        torch.cuda.synchronize()
        assert cache.last_device_error() == (abi.TP_ERR_BATCH if bad_last else abi.TP_OK)


def test_a_replayed_append_leaves_an_eager_one_its_status():
    abi, cache, bad, good, qkv = _two_appends()
    cache.append(qkv[:1], good)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = cache.append(qkv, bad)
    graph.replay()
    assert cache.last_device_error() == abi.TP_ERR_BATCH  # of the captured call, the last one
    cache.append(qkv[:1], good)
    graph.replay()
    assert cache.last_device_error() == abi.TP_OK
    assert held.shape == (1160, 4 * HD)
