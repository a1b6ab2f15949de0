"""What the passes from 4-bit weights keep: tokens and hidden activations as fp16 numbers
times a power of two of their own, 11 bits, the rest in 32 bits; the same to within
that for few and for many tokens, however far one number stands above the others."""
import pytest
import torch

from tests import weights4_reference as ref
from tests.test_gpu_weights4 import _ffn, _gen, _lib, _pack, _weights

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
R16 = 2.0 ** -11  # a rounding to fp16: half a step, relative
LEAST = 2.0 ** -39  # of a token's largest: half of fp16's least, 2^-25, where the largest is in 2^14..2^15


def _weight_error(c):
    """[rows, 1], how far each weight of a row may be from its value: 2^-19 of the row's
    largest scale in rows with scales below 2^-12 of it, else nothing."""
    s = c.scales.double().abs()
    top = s.amax(1, keepdim=True)
    least = torch.where(s > 0, s, top).amin(1, keepdim=True)
    return torch.where(least < 2.0 ** -12 * top, 2.0 ** -19 * top, 0.0)


def _forward(x, act, codes, group):
    """y in 64 bits, and how far a result may be from it.

    Tokens are bf16 numbers, whose eight bits fp16 has: only what is below 2^-25 of the
    token's largest is rounded, to half of the least number there is.  A product of K
    columns is off by e(K) sum |x w| besides, e(K) = (K + 8) 2^-22: four times the 2^-24 of
    each rounding of its sums, for the shortened sums of the matrix unit.  |silu'| <= 1.1,
    |gelu'| <= 1.13; the functions are within 2^-18 of their argument.  A hidden activation is rounded to fp16 (R16 and LEAST), y to bf16."""
    Ws = [ref.matrix(c.codes, c.scales, c.cols, c.segments, group) for c in codes]

    def product(v, ev, at):
        W = Ws[at]
        ev = ev + LEAST * v.abs().amax(1, keepdim=True)
        e = (v.shape[1] + 8) * 2.0 ** -22 * (v.abs() @ W.abs().T)
        return v @ W.T, e + ev @ W.abs().T + v.abs().sum(1, keepdim=True) * _weight_error(codes[at]).T
    v = x.double()
    ev = torch.zeros_like(v)
    if act == "swiglu":
        (a, ea), (b, eb) = product(v, ev, 0), product(v, ev, 1)
        s = torch.nn.functional.silu(a)
        v = s * b
        ev = 1.1 * ea * b.abs() + (s.abs() + 1.1 * ea) * eb + 2.0 ** -18 * (a * b).abs()
    elif act == "gelu_tanh":
        z, ez = product(v, ev, 0)
        v = ref.gelu(z)
        ev = 1.13 * ez + 2.0 ** -18 * z.abs()
    if act != "none":
        ev = ev + R16 * (v.abs() + ev)
    y, ey = product(v, ev, -1)
    return y, (1 + 2.0 ** -8) * ey + 2.0 ** -8 * y.abs() + 1e-30


def _rms(a, dim=None):
    return a.square().mean(dim).sqrt()


def _check(y, want, tol, dim=None):
    """Element by element, and in root mean square (of the whole, or of each token): the
    rounding of y to bf16, found from the 64-bit result itself, and that of the hidden
    activations, R16 at most (the other errors are below 2^-14 together), with a
    twentieth for chance.  Hidden activations in bf16 would add about as much as y's rounding."""
    err = (y.double() - want).abs()
    assert torch.isfinite(y).all()
    assert (err <= tol).all(), (err / tol).max().item()
    size = _rms(want, dim)
    rounding = _rms(want.to(BF).double() - want, dim) / size
    rel, limit = _rms(err, dim) / size, 1.05 * (rounding.square() + R16 ** 2).sqrt()
    assert (rel <= limit).all(), ((rel / limit).max().item(), rounding.max().item())


@pytest.mark.parametrize("n", [1, 8, 9, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("far", [10, 12, 14])
def test_one_large_element_of_a_token(far, group, n):
    """An element 2^10 to 2^14 above a token's others, in front of weights that are zero (code 8): it adds nothing,
    and the others' sums come out as they would without it."""
    ffn, codes = _ffn("none", 256, 1024, 2), _weights("none", 256, 1024, 2, group, 58)
    q = ref.nibbles(codes[0].codes, 1024)
    q[:, 17::100] = 8
    codes[0].codes.copy_(ref.bytes_of(q))
    x = torch.randn(n, 1024, generator=_gen(59), device="cuda")
    x[:, 17::100] = 1.37 * 2.0 ** far
    x = x.to(BF)
    _check(ffn.forward4(x, *_pack(ffn, codes)), *_forward(x, "none", codes, group))


@pytest.mark.parametrize("n", [4, 12])
def test_an_infinity_gives_what_its_weights_say(n):
    """Infinities where the weights of their column are not zero, of the weights' signs, NaN where they are or where
    two differ; NaN gives NaN."""
    group, d_ff = 32, 512
    ffn, codes = _ffn("none", 256, d_ff, 2), _weights("none", 256, d_ff, 2, group, 60)
    W = ref.matrix(codes[0].codes, codes[0].scales, d_ff, 2, group)
    assert (W == 0).any(0).all()
    x = torch.randn(n, d_ff, generator=_gen(61), device="cuda").to(BF)
    inf = float("inf")
    x[0, 5], x[1, 300], x[2, 7], x[2, 200], x[3, 100] = inf, -inf, inf, inf, float("nan")
    y = ffn.forward4(x, *_pack(ffn, codes)).double()
    want = x.double() @ W.T
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.isinf(), want.isinf())
    assert torch.equal(y[y.isinf()], want[want.isinf()])
    assert y[0].isinf().any() and y[0].isnan().any() and y[2].isinf().any() and y[3].isnan().all()


@pytest.mark.parametrize("n", [1, 8, 9, 40, 130])
@pytest.mark.parametrize("act,d,d_ff,T", [("swiglu", 1024, 1536, 4), ("gelu_tanh", 768, 2048, 2), ("none", 1024, 1000, 5)])
def test_only_the_result_is_rounded_to_bf16(act, d, d_ff, T, n):
    ffn, codes = _ffn(act, d, d_ff, T), _weights(act, d, d_ff, T, 64, 51)
    x = torch.randn(n, d_ff if act == "none" else d, generator=_gen(52), device="cuda").to(BF)
    _check(ffn.forward4(x, *_pack(ffn, codes)), *_forward(x, act, codes, 64))


@pytest.mark.parametrize("n", [8, 9, 64, 130])
@pytest.mark.parametrize("rows", [(5, 900), (5, 5)])
@pytest.mark.parametrize("far", [8, 10, 12, 20])
def test_one_large_group_in_either_matrix(far, rows, n):
    """A group of one hidden unit in each of W1 and W3 with a scale far above the others, in different units
    (whose hidden values stay near the others') and in the same (one unit above all others, where it is not
    shut): each token's error stays what it is without them."""
    d, d_ff, T = 1024, 1024, 2
    ffn, codes = _ffn("swiglu", d, d_ff, T), _weights("swiglu", d, d_ff, T, 128, 53)
    for c, row in zip(codes, rows):
        c.scales[row, 3] *= 2.0 ** far
    x = torch.randn(n, d, generator=_gen(54), device="cuda").to(BF)
    _check(ffn.forward4(x, *_pack(ffn, codes)), *_forward(x, "swiglu", codes, 128), dim=1)


@pytest.mark.parametrize("n", [8, 9, 40])
def test_one_large_group_before_gelu(n):
    d, d_ff, T = 512, 1024, 2
    ffn, codes = _ffn("gelu_tanh", d, d_ff, T), _weights("gelu_tanh", d, d_ff, T, 64, 55)
    codes[0].scales[700, 1] *= 2.0 ** 20
    x = torch.randn(n, d, generator=_gen(56), device="cuda").to(BF)
    _check(ffn.forward4(x, *_pack(ffn, codes)), *_forward(x, "gelu_tanh", codes, 64), dim=1)


@pytest.mark.parametrize("n", [3, 8, 9, 40, 150])
@pytest.mark.parametrize("act", ["swiglu", "gelu_tanh"])
def test_hidden_activations_keep_eleven_bits(act, n):
    """Hidden activations that are whole numbers of 1024..2047, times a power of two that the token has: y, the
    difference of two of them, is a bf16 number and comes out as it is (of eight bits, they would be off by up to
    four).  silu(64) and gelu of such numbers are their argument in 32 bits."""
    d, d_ff, T, group = 64, 256, 2, 32
    g = _gen(57)
    base = torch.randint(1024, 1793, (d_ff // 2, 1), generator=g, device="cuda")
    h = (base + torch.randint(0, 256, (d_ff // 2, 2), generator=g, device="cuda")).flatten()

    def codes_of(q, segments):
        groups = segments * -(-(q.shape[1] // segments) // group)
        return _lib().Codes4(ref.bytes_of(q + 8), torch.ones(q.shape[0], groups, dtype=BF, device="cuda"), q.shape[1], group, segments)
    digits, left = torch.zeros(d_ff, d, dtype=torch.long, device="cuda"), h.clone()
    for k in range(3):  # h = sum digit 8^k with digits -4..3, the last up to 4
        digits[:, k] = (left + 4) % 8 - 4
        left = (left - digits[:, k]) // 8
    digits[:, 3] = left
    gate = torch.zeros(d_ff, d, dtype=torch.long, device="cuda")
    gate[:, 4] = 1
    down = torch.zeros(d, d_ff, dtype=torch.long, device="cuda")
    at = torch.arange(d, device="cuda")
    down[at, 4 * at], down[at, 4 * at + 1] = 1, -1  # of both shards
    up = [codes_of(gate, 1), codes_of(digits, 1)] if act == "swiglu" else [codes_of(digits, 1)]
    size = torch.exp2((torch.arange(n, device="cuda") % 4).float())[:, None]
    x = torch.zeros(n, d, device="cuda")
    x[:, :4] = 8.0 ** torch.arange(4, device="cuda")
    x[:, 4] = 64
    x = (x * size).to(BF)
    want = (h[0::4] - h[1::4]) * (64 * size.square() if act == "swiglu" else size)
    ffn = _ffn(act, d, d_ff, T)
    y = ffn.forward4(x, *_pack(ffn, up + [codes_of(down, T)]))
    assert torch.equal(y.double(), want.double())
