"""The decode pass (q/k/v projection, append, attention, W_O) through each of its
attention kernels, behind shared keys that are taken together and without,
against 64-bit forms, and replayed from a graph.

Tolerance: relative in root mean square, 2 x 2^-8, as in
test_gpu_kv_cache.test_decode_is_the_composition: the pass rounds the
probabilities, the head outputs and y to bf16, each at most 2^-8 of the value
and less than half of that in root mean square (a rounding is spread evenly over
its interval: 2^-8 / sqrt(3)), so the three together stay below 2^-8; q, k and v
are rounded alike on both sides but where the 32-bit product falls on the other
side of a border, which is less than another 2^-8."""
import math

import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_kv_cache import HD, U, _modules
from tests.test_gpu_kv_dispatch import FEW, MANY, S_FEW, S_MANY

pytestmark = pytest.mark.gpu

CASES = [  # new, ctx, H, Hkv, T, page, shared, kernels
    ([1] * 4, [3, 0, 200, 65], 32, 8, 8, 32, 11000, [S_FEW, FEW]),
    ([2] * 4, [3, 0, 200, 65], 32, 8, 4, 32, 11000, [S_FEW, FEW]),
    ([1] * 64, [(i * 29) % 200 for i in range(64)], 32, 8, 8, 64, 700, [S_MANY, FEW]),
    ([9 + i % 8 for i in range(30)], [(61 * i) % 300 for i in range(30)], 32, 8, 8, 16, 1900, [S_MANY, MANY]),
    ([40, 3, 90, 0, 260], [7, 500, 0, 129, 30], 8, 2, 2, 16, 0, [MANY]),
    ([50, 60], [0, 900], 8, 2, 2, 64, 300, [MANY]),   # shared keys that are not worth it
    ([1] * 40, [50 * i for i in range(40)], 8, 2, 2, 16, 0, [FEW]),
]


def _make(new, ctx, H, Hkv, T, page, shared, d=512):
    abi, Attention, _, Cache = _modules()
    s = ref.make_batch(new, ctx, Hkv, page, shared, seed=81)
    attn = Attention(d, H, Hkv, HD, T)
    g = torch.Generator(device="cuda").manual_seed(14)
    w = lambda *sh: (torch.randn(*sh, generator=g, device="cuda") / math.sqrt(sh[1])).to(torch.bfloat16)
    Ws = w(H * HD, d), w(Hkv * HD, d), w(Hkv * HD, d), w(d, H * HD)
    x = torch.randn(s["n"], d, generator=g, device="cuda").to(torch.bfloat16)
    freq = 10000.0 ** (-torch.arange(64, device="cuda") / 64)

    def cache():
        c = Cache(attn, s["n_pages"], page, k=s["k"].clone(), v=s["v"].clone(), inv_freq=freq)
        return c, c.batch(s["cu"], s["kv_len"], s["table"], s["n"], s["max_new"])
    return abi, s, attn, Ws, attn.pack(*Ws), x, cache


def _want(s, Ws, x, cache, batch, H, Hkv, T):
    """y in 64 bits from q, k, v rounded to bf16 (the cache is left with them)."""
    z = torch.cat([x.double() @ W.double().T for W in Ws[:3]], 1)
    order = []
    for t in range(T):
        for first, heads in ((0, H), (H, Hkv), (H + Hkv, Hkv)):
            order += range((first + t * heads // T) * HD, (first + (t + 1) * heads // T) * HD)
    q = cache.append(z[:, order].to(torch.bfloat16).contiguous(), batch)
    o = ref.attend(dict(s, k=cache.k, v=cache.v), q, H)[0]
    return o @ Ws[3].double().T


def _rel(y, want):
    return ((y.double() - want).square().mean() / want.square().mean()).sqrt().item()


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared,kernels", CASES)
def test_decode(new, ctx, H, Hkv, T, page, shared, kernels):
    abi, s, attn, Ws, (wqkv, wo), x, cache = _make(new, ctx, H, Hkv, T, page, shared)
    c0, b0 = cache()
    c1, b1 = cache()
    want = _want(s, Ws, x, c1, b1, H, Hkv, T)
    y = attn.decode(x, c0, b0, wqkv, wo, shared_len=shared, flags=abi.TP_FLAG_TIMING)
    names = [name for name, _ in abi.tp_attn_kernel_times(attn.plan)]
    assert c0.last_device_error() == abi.TP_OK
    assert [n for n in names if n.startswith("kv_")] == ["kv_append"] + kernels + ["kv_combine"]
    assert torch.isfinite(y).all() and _rel(y, want) <= 2 * U, _rel(y, want)
    # the timed launches do not overlap; these do
    for flags in (dict(), dict(fused=True), dict(overlap=True)):
        got = attn.decode(x, c0, b0, wqkv, wo, shared_len=shared, **flags)
        assert _rel(got, want) <= 2 * U, (flags, _rel(got, want))
        if "fused" not in flags:
            assert torch.equal(got, y)
    assert c0.last_device_error() == abi.TP_OK


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared,kernels", CASES[:5])
def test_decode_replayed(new, ctx, H, Hkv, T, page, shared, kernels):
    """Two captured passes on changing inputs, each between calls of the other and eager ones."""
    abi, s, attn, Ws, (wqkv, wo), x, cache = _make(new, ctx, H, Hkv, T, page, shared)
    c, b = cache()
    xs = [x, (2 * x.float()).to(torch.bfloat16), x.flip(0).contiguous()]
    eager = [attn.decode(v, c, b, wqkv, wo, shared_len=shared).clone() for v in xs]
    at = x.clone()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = attn.decode(at, c, b, wqkv, wo, shared_len=shared)
        graphs.append((graph, y))
    for i in (1, 0, 2, 1):
        at.copy_(xs[i])
        for graph, y in graphs:
            y.fill_(9)
            graph.replay()
            assert torch.equal(attn.decode(xs[i], c, b, wqkv, wo, shared_len=shared), eager[i])
            assert torch.equal(y, eager[i])
    assert c.last_device_error() == abi.TP_OK
