"""Calls on one cache as a server makes them: from threads, in place, replayed on
two streams at once.  Results are compared bit for bit with calls made singly."""
import math
import threading

import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_kv_cache import HD, _cache, _modules, _q

pytestmark = pytest.mark.gpu

BATCHES = [  # new, ctx, H, Hkv, T, page, shared: every attention kernel and the join of each
    ([1, 4, 2], [500, 3000, 7], 8, 2, 2, 16, 0),
    ([70, 1, 200], [500, 3000, 7], 8, 2, 2, 64, 0),
    ([1] * 64, [(i * 29) % 200 for i in range(64)], 32, 8, 8, 16, 700),
    ([1] * 4, [3, 0, 200, 65], 32, 8, 8, 32, 11000),
    ([9 + i % 8 for i in range(30)], [(61 * i) % 300 for i in range(30)], 32, 8, 8, 16, 1900),
]


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared", BATCHES)
def test_attend_in_place(new, ctx, H, Hkv, T, page, shared):
    s = ref.make_batch(new, ctx, Hkv, page, shared, seed=91)
    cache, batch = _cache(s, H, T)
    q = _q(s["n"], H, 4)
    want = cache.attend(q, batch, shared_len=shared)
    for _ in range(3):
        x = q.clone()
        assert cache.attend(x, batch, shared_len=shared, out=x) is x
        assert torch.equal(x, want)


@pytest.mark.parametrize("own_streams", [False, True])
def test_threads(own_streams):
    """Four threads, each with a batch and shared keys of its own, on one stream and on four."""
    new, ctx, H, Hkv, T, page, shared = BATCHES[2]
    s = ref.make_batch(new, ctx, Hkv, page, shared, seed=92)
    cache, batch = _cache(s, H, T)
    qs = [_q(s["n"], H, 20 + i) for i in range(4)]
    shares = [shared, 0, shared, 600]
    want = [cache.attend(q, batch, shared_len=n) for q, n in zip(qs, shares)]
    torch.cuda.synchronize()
    wrong, main = [], torch.cuda.current_stream()

    def work(i):
        st = torch.cuda.Stream() if own_streams else main
        with torch.cuda.stream(st):
            got = [cache.attend(qs[i], batch, shared_len=shares[i]) for _ in range(40)]
            st.synchronize()
            wrong.extend(i for o in got if not torch.equal(o, want[i]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong


def test_two_captured_passes_at_once():
    """Replayed on two streams, each with its own rows and pages, beside eager calls."""
    abi, Attention, _, Cache = _modules()
    H, Hkv, T, d, page = 8, 2, 2, 512, 16
    s = ref.make_batch([1, 3, 2, 40, 5], [100, 0, 30, 7, 300], Hkv, page, seed=93, junk=0.0)
    attn = Attention(d, H, Hkv, HD, T)
    g = torch.Generator(device="cuda").manual_seed(5)
    w = lambda *sh: (torch.randn(*sh, generator=g, device="cuda") / math.sqrt(sh[1])).to(torch.bfloat16)
    wqkv, wo = attn.pack(w(H * HD, d), w(Hkv * HD, d), w(Hkv * HD, d), w(d, H * HD))
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = Cache(attn, s["n_pages"], page, k=s["k"], v=s["v"])
    parts = []
    for seqs in ([0, 1], [2, 3], [4]):  # the last for the eager calls
        cu = torch.tensor([sum(s["new"][b] for b in seqs[:i]) for i in range(len(seqs) + 1)], **i32)
        at = torch.tensor(seqs, device="cuda")
        n = cu[-1].item()
        x = torch.randn(n, d, generator=g, device="cuda").to(torch.bfloat16)
        parts.append((cache.batch(cu, s["kv_len"][at].contiguous(), s["table"][at].contiguous(), n, 40), x))
    want = [attn.decode(x, cache, b, wqkv, wo) for b, x in parts]
    graphs = []
    for b, x in parts[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = attn.decode(x, cache, b, wqkv, wo)
        graphs.append((graph, y, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, y, st in graphs:
            with torch.cuda.stream(st):
                y.fill_(3)
                graph.replay()
        eager = attn.decode(parts[2][1], cache, parts[2][0], wqkv, wo)
        torch.cuda.synchronize()
        for (graph, y, _), z in zip(graphs, want):
            assert torch.equal(y, z)
        assert torch.equal(eager, want[2])
    assert cache.last_device_error() == abi.TP_OK
