"""4-bit weights in use: scales far apart, many and large tokens, what is not finite,
waits that run out, side streams, threads and replays, refusals, and a block's decode
step with the norms around its sublayers.

Tolerances are those of weights4_reference.forward, test_gpu_weights4.test_decode and
test_gpu_norm.close; what runs twice the same way gives the same bits."""
import threading

import pytest
import torch

from tests import test_gpu_norm as norms
from tests import weights4_reference as ref
from tests.test_gpu_weights4 import _check, _ffn, _gen, _lib, _pack, _weights

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -8


def _abi():
    from megatron_tensor_transformer_w1_gb300 import tpffn
    return tpffn


def _matrices(codes, group):
    return [ref.matrix(c.codes, c.scales, c.cols, c.segments, group) for c in codes]


@pytest.mark.parametrize("n", [5, 40, 150])
@pytest.mark.parametrize("act,d,d_ff,T", [("swiglu", 640, 384, 1), ("none", 256, 1024, 4), ("gelu_tanh", 384, 512, 2)])
def test_scales_of_a_row_far_apart(act, d, d_ff, T, n):
    """Scales over 2^24 within a row, and a row whose scales are the smallest there are."""
    ffn, codes = _ffn(act, d, d_ff, T), _weights(act, d, d_ff, T, 32, 21)
    g = _gen(22)
    for c in codes:
        far = torch.randint(-18, 6, c.scales.shape, generator=g, device="cuda").float()
        c.scales.copy_(c.scales.float() * torch.exp2(far))
        c.scales[3] = 2.0 ** -133
        c.scales[5] = 0
    up, down = _pack(ffn, codes)
    x = torch.randn(n, d_ff if act == "none" else d, generator=g, device="cuda").to(BF)
    _check(ffn.forward4(x, up, down), *ref.forward(x, act, _matrices(codes, 32), None, None))


@pytest.mark.parametrize("n", [5, 40])
def test_the_largest_and_smallest_scales(n):
    """Rows whose scales are all as large or as small as a bf16 weight's can be."""
    ffn, codes = _ffn("none", 256, 512, 2), _weights("none", 256, 512, 2, 64, 30)
    sizes = torch.tensor([2.0 ** 125, 2.0 ** 120, 2.0 ** -126, 2.0 ** -60], device="cuda").repeat(64)
    g = _gen(33)
    codes[0].scales.copy_((0.5 + 0.5 * torch.rand(codes[0].scales.shape, generator=g, device="cuda")) * sizes[:, None])
    x = (torch.randn(n, 512, generator=g, device="cuda") * 2.0 ** -30).to(BF)
    want, tol = ref.forward(x, "none", _matrices(codes, 64), None, None)
    # what is below 2^-126 may be lost, a product's and the result's
    _check(ffn.forward4(x, *_pack(ffn, codes)), want, tol + 2.0 ** -116)


@pytest.mark.parametrize("act,d,d_ff,T,n", [("swiglu", 256, 384, 2, 513), ("gelu_tanh", 264, 640, 4, 1030), ("none", 128, 512, 2, 1537)])
def test_many_tokens(act, d, d_ff, T, n):
    """More tokens than go through the products at once."""
    ffn, codes = _ffn(act, d, d_ff, T), _weights(act, d, d_ff, T, 64, 23)
    up, down = _pack(ffn, codes)
    g = _gen(n)
    x = torch.randn(n, d_ff if act == "none" else d, generator=g, device="cuda").to(BF)
    b1 = torch.randn(d_ff, generator=g, device="cuda").to(BF) if act == "gelu_tanh" else None
    b2 = torch.randn(d, generator=g, device="cuda").to(BF)
    _check(ffn.forward4(x, up, down, b1=b1, b2=b2), *ref.forward(x, act, _matrices(codes, 64), b1, b2))


@pytest.mark.parametrize("n", [16, 48])
def test_sizes_of_tokens_and_shifts(n):
    """Tokens from 2^-110 to 2^40 in size beside shifts of ordinary size, and without them."""
    ffn, codes = _ffn("gelu_tanh", 256, 384, 2), _weights("gelu_tanh", 256, 384, 2, 64, 24)
    up, down = _pack(ffn, codes)
    g = _gen(n)
    x = torch.randn(n, 256, generator=g, device="cuda") * torch.exp2(torch.linspace(-110, 40, n, device="cuda").round())[:, None]
    x = x.to(BF)
    b1 = torch.randn(384, generator=g, device="cuda").to(BF)
    for shift in (b1, (b1.float() * 2.0 ** 30).to(BF), None):
        y = ffn.forward4(x, up, down, b1=shift)
        want, tol = ref.forward(x, "gelu_tanh", _matrices(codes, 64), shift, None)
        # a product of numbers below 2^-126 may be lost: at most 2^-126 for each of its terms
        _check(y, want, tol + 2.0 ** -116)


@pytest.mark.parametrize("n", [5, 40])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_scale_that_is_not_finite_stays_in_its_row(value, n):
    ffn, codes = _ffn("none", 256, 512, 2), _weights("none", 256, 512, 2, 128, 25)
    x = torch.randn(n, 512, generator=_gen(n), device="cuda").to(BF)
    clean = ffn.forward4(x, *_pack(ffn, codes))
    codes[0].scales[130, 2] = value
    y = ffn.forward4(x, *_pack(ffn, codes))
    rest = torch.arange(256, device="cuda") != 130
    assert torch.equal(y[:, rest], clean[:, rest])
    assert not torch.isfinite(y[:, 130]).any()


@pytest.mark.parametrize("n", [4, 12, 40, 130])
def test_bounded_wait_expires_and_context_survives(n):
    """A copy that is never issued: its waits run out, the call reports it, and the next call is as ever."""
    abi = _abi()
    ffn, codes = _ffn("swiglu", 512, 640, 2), _weights("swiglu", 512, 640, 2, 64, 26)
    up, down = _pack(ffn, codes)
    x = torch.randn(n, 512, generator=_gen(n), device="cuda").to(BF)
    good = ffn.forward4(x, up, down)
    with pytest.raises(Exception, match="TP_ERR_TIMEOUT"):
        ffn.forward4(x, up, down, flags=abi.TP_FLAG_DEBUG_SKIP_LOAD | abi.TP_FLAG_SYNC)
    assert torch.equal(ffn.forward4(x, up, down, flags=abi.TP_FLAG_SYNC), good)


@pytest.mark.parametrize("n", [3, 70])
def test_streams_threads_and_replays(n):
    ffn, codes = _ffn("swiglu", 512, 1280, 2), _weights("swiglu", 512, 1280, 2, 128, 27)
    up, down = _pack(ffn, codes)
    xs = [torch.randn(n, 512, generator=_gen(i), device="cuda").to(BF) for i in range(4)]
    want = [ffn.forward4(x, up, down) for x in xs]
    torch.cuda.synchronize()
    # two graphs of the object, replayed beside one another and beside eager calls
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs, ins, outs = [], [x.clone() for x in xs[:2]], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(ffn.forward4(ins[i], up, down))
    for turn in range(3):
        for i in range(2):
            ins[i].copy_(xs[(i + turn) % 4])
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        with torch.cuda.stream(streams[2]):
            eager = ffn.forward4(xs[3], up, down)
        torch.cuda.synchronize()
        assert torch.equal(eager, want[3])
        for i in range(2):
            assert torch.equal(outs[i], want[(i + turn) % 4])
    # threads on one stream and on streams of their own
    got, failed = {}, []

    def work(i):
        try:
            with torch.cuda.stream(streams[i % 3]):
                for turn in range(20):
                    got[i] = ffn.forward4(xs[i], up, down)
            streams[i % 3].synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for i in range(4):
        assert torch.equal(got[i], want[i])


def test_refusals():
    w4 = _lib()
    ffn, codes = _ffn("swiglu", 256, 384, 2), _weights("swiglu", 256, 384, 2, 64, 28)
    up, down = _pack(ffn, codes)
    other = _ffn("swiglu", 256, 512, 2)
    up2, _ = _pack(other, _weights("swiglu", 256, 512, 2, 64, 28))
    up128, _ = _pack(ffn, _weights("swiglu", 256, 384, 2, 128, 28))
    x = torch.zeros(5, 256, dtype=BF, device="cuda")
    wide = torch.zeros(5, 512, dtype=BF, device="cuda")
    for bad in (None, x.float(), x.cpu(), x[0], x[:, :128], wide[:, :256], x.t().contiguous().t()):
        with pytest.raises(ValueError):
            ffn.forward4(bad, up, down)
    for bad in (x.float(), x[:4], x.cpu(), wide[:, :256]):
        with pytest.raises(ValueError):
            ffn.forward4(x, up, down, out=bad)
    for weights in ((None, down), (up, None), (up2, down), (up128, down), (down, up), (up.data, down)):
        with pytest.raises(ValueError):
            ffn.forward4(x, *weights)
    with pytest.raises(ValueError):
        ffn.forward4(x, up, down, b2=torch.zeros(255, dtype=BF, device="cuda"))
    with pytest.raises(Exception, match="TP_ERR_UNSUPPORTED"):  # a gated sublayer has no first bias
        ffn.forward4(x, up, down, b1=torch.zeros(384, dtype=BF, device="cuda"))
    for bad in (codes[0].codes.float(), x.t(), x[0], x.cpu()):
        with pytest.raises(ValueError):
            w4.quantize4(bad)
    for group in (0, 16, 48, 256):
        with pytest.raises(ValueError):
            w4.quantize4(x, group=group)
    with pytest.raises(ValueError):
        w4.quantize4(x, segments=3)


def test_a_blocks_decode_step():
    """Norm, attention, norm with gate and residual sum, feed-forward, norm: every step against its plain form on
    the tensors that it got, and the whole captured and replayed."""
    from megatron_tensor_transformer_w1_gb300.attention import TensorParallelAttention
    from megatron_tensor_transformer_w1_gb300.kv_cache import PagedKVCache
    from megatron_tensor_transformer_w1_gb300.norm import SublayerNorm
    w4 = _lib()
    d, d_ff, H, Hkv, T, group = 512, 1280, 4, 2, 2, 64
    g = _gen(31)
    attn, ffn = TensorParallelAttention(d, H, Hkv, 128, T), _ffn("swiglu", d, d_ff, T)
    acodes = [w4.Codes4(*ref.random_codes(r, c, s, group, g, True), c, group, s) for r, c, s in attn._shapes4()]
    fcodes = _weights("swiglu", d, d_ff, T, group, 29)
    wqkv, wo = attn.pack4(*acodes)
    plain_attn = attn.pack(*[w4.dequantize4(c) for c in acodes])
    up, down = _pack(ffn, fcodes)
    first, mid = SublayerNorm(d), SublayerNorm(d, after=True, scale=0.5)
    last = SublayerNorm(d, before=False, after=True)
    w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(BF) for _ in range(5)]
    gate = (0.5 + 0.5 * torch.randn(1, d, generator=g, device="cuda")).to(BF)
    i32 = dict(dtype=torch.int32, device="cuda")
    n, ctx = 6, [40, 0, 5, 70, 33, 17]
    cu, table = torch.arange(n + 1, **i32), torch.arange(n * 6, **i32).view(n, 6)
    kv_len = torch.tensor([c + 1 for c in ctx], **i32)
    k0, v0 = (torch.randn(n * 6, Hkv, 16, 128, generator=g, device="cuda").to(BF) for _ in range(2))
    freq = torch.rand(64, generator=g, device="cuda")
    cache = PagedKVCache(attn, n * 6, 16, k=k0.clone(), v=v0.clone(), inv_freq=freq)
    batch = cache.batch(cu, kv_len, table, n, 1)
    x = torch.randn(n, d, generator=g, device="cuda").to(BF)

    def step():
        r0, a, _ = first.forward(x, w_before=w[0], save=False)
        b = attn.decode(a, cache, batch, wqkv, wo)
        r1, c, _ = mid.forward(r0, b, w_after=w[1], gate=gate, w_before=w[2], save=False)
        y = ffn.forward4(c, up, down)
        r2, _, _ = last.forward(r1, y, w_after=w[3], save=False)
        return r0, a, b, r1, c, y, r2
    r0, a, b, r1, c, y, r2 = step()
    assert cache.last_device_error() == 0

    def norm_check(m, got, x, b, kind=(True, False), **given):
        s = dict(x=x, b=b, w_after=None, c_after=None, gate=None, w_before=None, c_before=None)
        s.update(given)
        before, after = kind
        want = norms.ref_forward(s, "rms", before, after, m.abi.scale, m.abi.eps)
        for name, t in got.items():
            norms.close(name, t, want[name], "bf16")
    assert torch.equal(r0, x)
    norm_check(first, dict(out=a), x, torch.zeros_like(x), w_before=w[0])
    norm_check(mid, dict(r=r1, out=c), r0, b, (True, True), w_after=w[1], gate=gate, w_before=w[2])
    norm_check(last, dict(r=r2), r1, y, (False, True), w_after=w[3])
    _check(y, *ref.forward(c, "swiglu", _matrices(fcodes, group), None, None))
    plain = PagedKVCache(attn, n * 6, 16, k=k0.clone(), v=v0.clone(), inv_freq=freq)
    want = attn.decode(a, plain, plain.batch(cu, kv_len, table, n, 1), *plain_attn)
    rel = ((b.double() - want.double()).square().mean() / want.double().square().mean()).sqrt().item()
    assert rel <= 2 * U, rel
    # the same step again, captured and replayed on other tokens
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    x.copy_(torch.randn(n, d, generator=g, device="cuda").to(BF))
    graph.replay()
    torch.cuda.synchronize()
    for got, want in zip(captured, step()):
        assert torch.equal(got, want)


def test_decode_of_more_tokens_than_go_through_at_once():
    """Prompts of 650 tokens beside the bf16 pass from the same weights (scales that are powers of two), and rows
    behind the last sequence, whose numbers reach nobody."""
    from megatron_tensor_transformer_w1_gb300.attention import TensorParallelAttention
    from megatron_tensor_transformer_w1_gb300.kv_cache import PagedKVCache
    w4 = _lib()
    d, H, Hkv, T, group = 264, 4, 2, 2, 32
    attn = TensorParallelAttention(d, H, Hkv, 128, T)
    g = _gen(41)
    codes = [w4.Codes4(*ref.random_codes(r, c, s, group, g, True), c, group, s) for r, c, s in attn._shapes4()]
    plain, packed = attn.pack(*[w4.dequantize4(c) for c in codes]), attn.pack4(*codes)
    new, ctx, page = [300, 1, 349], [0, 70, 33], 16
    n, spare = sum(new), 5
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 300, 301, 650], **i32)
    kv_len = torch.tensor([a + b for a, b in zip(new, ctx)], **i32)
    table = torch.arange(3 * 24, **i32).view(3, 24)
    k, v = (torch.randn(72, Hkv, page, 128, generator=g, device="cuda").to(BF) for _ in range(2))
    x = torch.randn(n + spare, d, generator=g, device="cuda").to(BF)
    got = []
    for weights in (plain, packed):
        cache = PagedKVCache(attn, 72, page, k=k.clone(), v=v.clone(), inv_freq=torch.rand(64, generator=_gen(0), device="cuda"))
        for last in (0.0, float("nan")):
            x[n:] = last
            y = attn.decode(x, cache, cache.batch(cu, kv_len, table, n + spare, 349), *weights)[:n]
            assert cache.last_device_error() == 0
            got.append(y.double())
    assert torch.equal(got[0], got[1]) and torch.equal(got[2], got[3])
    rel = ((got[2] - got[0]).square().mean() / got[0].square().mean()).sqrt().item()
    assert rel <= 2 * U, rel


def test_kernel_times_name_the_launches():
    abi = _abi()
    ffn, codes = _ffn("swiglu", 256, 384, 2), _weights("swiglu", 256, 384, 2, 64, 42)
    up, down = _pack(ffn, codes)
    for n, names in ((3, ["prepare4", "up_swiglu4", "down4"]), (20, ["prepare4", "up_swiglu4", "finish4", "down4", "finish4"])):
        x = torch.randn(n, 256, generator=_gen(n), device="cuda").to(BF)
        ffn.forward4(x, up, down, flags=abi.TP_FLAG_TIMING | abi.TP_FLAG_SYNC)
        assert [name for name, _ in abi.tp_ffn_kernel_times(ffn.plan)] == names
