"""4-bit weights against plain 64-bit forms: quantising and reading back (equal),
the packed layout there and back (equal), the feed-forward and output-projection
passes from such weights, the attention sublayer's decode pass.

Tolerances of the passes: element by element as derived in
weights4_reference.forward; and in root mean square 2^-8 of the result: h and y
are rounded to bf16, each by at most 2^-8 of the value, evenly spread over the
interval (2^-8 / sqrt(3) at most), together below 2^-8."""
import pytest
import torch

from tests import weights4_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -8


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lib():
    from megatron_tensor_transformer_w1_gb300 import weights4
    return weights4


SHAPES = [(1, 16, 1), (1, 1, 1), (5, 48, 1), (3, 219, 3), (64, 1280, 4), (130, 2730, 3), (2, 40, 5), (7, 1000, 1),
          (257, 8192, 1), (33, 15, 3), (1000, 33, 1), (9, 336, 2)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,cols,segments", SHAPES)
def test_quantize(rows, cols, segments, group):
    w4 = _lib()
    W = torch.randn(rows, cols, generator=_gen(rows + cols), device="cuda").to(BF)
    c = w4.quantize4(W, group=group, segments=segments)
    q, scales = ref.quantize(W, segments, group)
    assert torch.equal(c.scales, scales)
    assert torch.equal(c.codes, ref.bytes_of(q))
    want = ref.matrix(c.codes, c.scales, cols, segments, group).to(BF)
    assert torch.equal(w4.dequantize4(c), want)


@pytest.mark.parametrize("cols,segments", [(128, 1), (99, 3)])
def test_quantize_ties_and_borders(cols, segments):
    """Ties go to the even code; groups of zeros, of one value, of the largest and smallest values."""
    w4 = _lib()
    g = _gen(4)
    rows = []
    for e in (-133, -126, -100, -20, 0, 60, 120):  # scales 2^e: quotients are multiples of a half, ties among them
        steps = torch.randint(-14, 15, (cols,), generator=g, device="cuda").double() / 2
        steps[:: 32] = 7.0
        rows.append((steps * 2.0 ** e).to(BF))
    for b in (129, 150, 199, 255):  # scales of eight bits: ties at odd multiples of half the scale
        steps = torch.randint(-7, 8, (cols,), generator=g, device="cuda").double()
        steps[:: 32] = 7.0
        rows.append((steps * b * 2.0 ** -9).to(BF))
    rows += [torch.zeros(cols, device="cuda", dtype=BF), torch.full((cols,), 3.3895e38, device="cuda", dtype=BF),
             torch.full((cols,), 1e-40, device="cuda", dtype=BF), torch.full((cols,), -0.0, device="cuda", dtype=BF)]
    W = torch.stack(rows)
    for group in (32, 64, 128):
        c = w4.quantize4(W, group=group, segments=segments)
        q, scales = ref.quantize(W, segments, group)
        assert torch.equal(c.scales, scales)
        assert torch.equal(ref.nibbles(c.codes, cols), q)


@pytest.mark.parametrize("cols", [256, 250])
def test_quantize_keeps_what_is_not_finite_in_its_group(cols):
    w4 = _lib()
    W = torch.randn(4, cols, generator=_gen(6), device="cuda").to(BF)
    V = W.clone()
    V[1, 70], V[2, 5], V[3, 200] = float("nan"), float("inf"), -float("inf")
    a, b = w4.quantize4(W, group=64), w4.quantize4(V, group=64)
    bad = torch.zeros_like(a.scales, dtype=torch.bool)
    bad[1, 1] = bad[2, 0] = bad[3, 3] = True
    assert torch.equal(torch.isfinite(b.scales), ~bad)
    assert torch.equal(a.scales[~bad], b.scales[~bad])
    at = ref.group_columns(cols, 1, 64)
    x, y = w4.dequantize4(a), w4.dequantize4(b)
    assert torch.equal(x[~bad[:, at]], y[~bad[:, at]]) and not torch.isfinite(y[bad[:, at]]).any()


def test_quantize_wide_and_empty():
    w4 = _lib()
    for shape in ((0, 64), (3, 0), (0, 0)):
        c = w4.quantize4(torch.empty(shape, dtype=BF, device="cuda"), group=64)
        assert w4.dequantize4(c).shape == shape
    W = torch.randn(70000, 32, generator=_gen(1), device="cuda").to(BF)
    assert torch.equal(w4.quantize4(W, group=32).scales, ref.quantize(W, 1, 32)[1])


# ------------------------------------------------------------ passes
def _ffn(act, d, d_ff, T):
    from megatron_tensor_transformer_w1_gb300.ffn import TensorParallelFFN
    return TensorParallelFFN(d, d_ff, T, act=act)


def _weights(act, d, d_ff, T, group, seed, pow2=False):
    g = _gen(seed)
    shapes = [(d_ff, d, 1)] * {"swiglu": 2, "gelu_tanh": 1, "none": 0}[act] + [(d, d_ff, T)]
    w4 = _lib()
    return [w4.Codes4(*ref.random_codes(r, c, s, group, g, pow2), c, group, s) for r, c, s in shapes]


def _pack(ffn, codes):
    up = codes[:-1] + [None] * (3 - len(codes))
    return ffn.pack4(up[0], codes[-1], up[1])


FFN = [  # act, d, d_ff, T
    ("swiglu", 64, 128, 1), ("swiglu", 1000, 2730, 3), ("swiglu", 264, 33, 3), ("swiglu", 512, 1024, 8),
    ("gelu_tanh", 8, 1, 1), ("gelu_tanh", 200, 300, 4), ("gelu_tanh", 768, 1280, 4), ("gelu_tanh", 136, 777, 7),
    ("none", 256, 512, 4), ("none", 72, 88, 11), ("none", 1032, 1000, 5),
]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("act,d,d_ff,T", FFN)
def test_packed_layout_there_and_back(act, d, d_ff, T, group):
    ffn, codes = _ffn(act, d, d_ff, T), _weights(act, d, d_ff, T, group, 7)
    up, down = _pack(ffn, codes)
    odd = lambda c: c.codes & 15 if c.cols == 1 else c.codes
    back = [ffn.unpack4_rows(down)]
    if act != "none":
        back = [c for c in ffn.unpack4_columns(up) if c is not None] + back
    for a, b in zip(codes, back):
        assert torch.equal(a.scales, b.scales) and torch.equal(a.codes, b.codes)
        assert (a.cols, a.group, a.segments) == (b.cols, b.group, b.segments)


TOKENS = [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 130, 257]


def _check(y, want, tol):
    err = (y.double() - want).abs()
    assert torch.isfinite(y).all()
    assert (err <= tol).all(), (err / tol).max().item()
    rel = (err.square().mean() / want.square().mean()).sqrt().item()
    assert rel <= U, rel


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("act,d,d_ff,T", FFN)
def test_forward(act, d, d_ff, T, group):
    ffn, codes = _ffn(act, d, d_ff, T), _weights(act, d, d_ff, T, group, 8)
    up, down = _pack(ffn, codes)
    Ws = [ref.matrix(c.codes, c.scales, c.cols, c.segments, group) for c in codes]
    g = _gen(d + d_ff)
    for n in TOKENS if group == 64 else (1, 5, 40, 70):
        x = torch.randn(n, d_ff if act == "none" else d, generator=g, device="cuda").to(BF)
        b1 = torch.randn(d_ff, generator=g, device="cuda").to(BF) if act == "gelu_tanh" and n % 2 else None
        b2 = torch.randn(d, generator=g, device="cuda").to(BF) if n % 3 else None
        y = ffn.forward4(x, up, down, b1=b1, b2=b2, flags=2)
        _check(y, *ref.forward(x, act, Ws, b1, b2))


@pytest.mark.parametrize("act,d,d_ff,T,n", [("swiglu", 4096, 14336, 8, 3), ("swiglu", 2048, 5632, 4, 48),
                                            ("gelu_tanh", 1024, 4096, 4, 1), ("none", 4096, 4096, 8, 20),
                                            ("swiglu", 8192, 3584, 1, 16), ("gelu_tanh", 1600, 6400, 5, 129)])
def test_forward_of_many_units(act, d, d_ff, T, n):
    """Matrices whose units are shared by many blocks, each of which may begin and end inside a unit."""
    ffn, codes = _ffn(act, d, d_ff, T), _weights(act, d, d_ff, T, 128, 9)
    up, down = _pack(ffn, codes)
    Ws = [ref.matrix(c.codes, c.scales, c.cols, c.segments, 128) for c in codes]
    x = torch.randn(n, d_ff if act == "none" else d, generator=_gen(3), device="cuda").to(BF)
    y = ffn.forward4(x, up, down)
    _check(y, *ref.forward(x, act, Ws, None, None))
    for _ in range(3):
        assert torch.equal(ffn.forward4(x, up, down), y)


@pytest.mark.parametrize("n", [3, 12, 40])
@pytest.mark.parametrize("act,d,d_ff,T", [("swiglu", 512, 640, 2), ("none", 256, 1024, 4)])
def test_forward_of_wide_ranges(act, d, d_ff, T, n):
    """Tokens of very different sizes, and elements of very different sizes within a block."""
    ffn, codes = _ffn(act, d, d_ff, T), _weights(act, d, d_ff, T, 64, 10)
    up, down = _pack(ffn, codes)
    Ws = [ref.matrix(c.codes, c.scales, c.cols, c.segments, 64) for c in codes]
    g = _gen(n)
    x = torch.randn(n, d_ff if act == "none" else d, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-12, 3, x.shape, generator=g, device="cuda").float())
    size = torch.linspace(-60, 60, n, device="cuda") if act == "none" else torch.linspace(-20, 4, n, device="cuda")
    x = (x * torch.exp2(size.round())[:, None]).to(BF)
    x[1] = 0
    y = ffn.forward4(x, up, down).double()
    want, tol = ref.forward(x, act, Ws, None, None)
    assert torch.isfinite(y).all() and ((y - want).abs() <= tol).all(), ((y - want).abs() / tol).max().item()
    rel = (y - want).norm(dim=1) / want.norm(dim=1).clamp(min=1e-30)
    assert (rel <= U).all(), rel


def test_forward_of_quantised_weights_and_output_in_place():
    ffn = _ffn("swiglu", 256, 512, 2)
    g = _gen(2)
    W1, W3 = (torch.randn(512, 256, generator=g, device="cuda").to(BF) for _ in range(2))
    W2 = torch.randn(256, 512, generator=g, device="cuda").to(BF)
    w4 = _lib()
    up, down = ffn.pack4(W1, W2, W3, group=32)
    Ws = [w4.dequantize4(w4.quantize4(W, 32, s)).double() for W, s in ((W1, 1), (W3, 1), (W2, 2))]
    codes = [w4.quantize4(W, 32, s) for W, s in ((W1, 1), (W3, 1), (W2, 2))]
    Ws = [ref.matrix(c.codes, c.scales, c.cols, c.segments, 32) for c in codes]
    x = torch.randn(21, 256, generator=g, device="cuda").to(BF)
    want = ref.forward(x, "swiglu", Ws, None, None)
    out = torch.full((21, 256), 7, dtype=BF, device="cuda")
    assert ffn.forward4(x, up, down, out=out) is out
    _check(out, *want)
    assert ffn.forward4(x[:0], up, down).shape == (0, 256)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_token(value):
    """... whose outputs are infinities or NaN: also behind a shard's last column, where the next shard's lies beside it."""
    for act, d, d_ff, T in (("none", 72, 88, 11), ("swiglu", 136, 99, 3)):
        ffn, codes = _ffn(act, d, d_ff, T), _weights(act, d, d_ff, T, 32, 12)
        up, down = _pack(ffn, codes)
        x = torch.randn(20, d_ff if act == "none" else d, generator=_gen(1), device="cuda").to(BF)
        clean = ffn.forward4(x, up, down)
        x[7, 8] = value
        y = ffn.forward4(x, up, down)
        rest = torch.arange(20, device="cuda") != 7
        assert torch.equal(y[rest], clean[rest])
        assert not torch.isfinite(y[7]).any()


# ------------------------------------------------------------ the attention sublayer
@pytest.mark.parametrize("H,Hkv,T,d,group", [(2, 1, 1, 256, 64), (8, 2, 2, 520, 128), (8, 8, 4, 264, 32)])
def test_decode(H, Hkv, T, d, group):
    """With scales that are powers of two the weights are bf16 numbers, and the pass is the bf16 one up to the
    order of 32-bit sums: q, k, v, the head outputs and y are rounded to bf16 on both sides."""
    from megatron_tensor_transformer_w1_gb300.attention import TensorParallelAttention
    from megatron_tensor_transformer_w1_gb300.kv_cache import PagedKVCache
    w4 = _lib()
    attn = TensorParallelAttention(d, H, Hkv, 128, T)
    g = _gen(H)
    codes = [w4.Codes4(*ref.random_codes(r, c, s, group, g, True), c, group, s) for r, c, s in attn._shapes4()]
    Ws = [w4.dequantize4(c) for c in codes]
    wqkv, wo = attn.pack(*Ws)
    packed = attn.pack4(*codes)
    for a, b in zip(codes, attn.unpack4(*packed)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    new, ctx = [1, 3, 0, 12], [40, 0, 5, 70]
    n = sum(new)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1, 4, 4, 16], **i32)
    table = torch.arange(4 * 6, **i32).view(4, 6)
    kv_len = torch.tensor([a + b for a, b in zip(new, ctx)], **i32)
    k, v = (torch.randn(24, Hkv, 16, 128, generator=g, device="cuda").to(BF) for _ in range(2))
    x = torch.randn(n, d, generator=g, device="cuda").to(BF)
    got = []
    for weights in ((wqkv, wo), packed):
        cache = PagedKVCache(attn, 24, 16, k=k.clone(), v=v.clone(), inv_freq=torch.rand(64, generator=_gen(0), device="cuda"))
        batch = cache.batch(cu, kv_len, table, n, 12)
        y = attn.decode(x, cache, batch, *weights)
        assert cache.last_device_error() == 0
        got.append((y, cache.k, cache.v))
    for a, b in zip(*got):
        rel = ((a.double() - b.double()).square().mean() / a.double().square().mean()).sqrt().item()
        assert rel <= 2 * U, rel
