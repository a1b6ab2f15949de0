"""4-bit weights and their products in plain 64-bit forms."""
import math

import torch


def group_columns(cols, segments, group):
    """Group number of each column of a row."""
    width = cols // segments
    j = torch.arange(cols, device="cuda")
    return (j // width) * -(-width // group) + (j % width) // group


def quantize(W, segments, group):
    """codes [rows, cols] (whole numbers) and scales bf16 of a bf16 matrix with finite elements."""
    rows, cols = W.shape
    at = group_columns(cols, segments, group)
    n = segments * -(-(cols // segments) // group)
    w = W.double()
    top = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    top.scatter_reduce_(1, at.expand(rows, cols), w.abs(), "amax")
    scales = (top / 7).to(torch.bfloat16)
    s = scales.double()[:, at]
    q = torch.where(s > 0, torch.round(w / torch.where(s > 0, s, 1.0)), 0.0)
    return q.long() + 8, scales


def nibbles(codes, cols):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(1)[:, :cols].long()


def bytes_of(q):
    """Natural layout of codes [rows, cols]; a last odd column stands alone with code 8 behind it."""
    if q.shape[1] % 2:
        q = torch.nn.functional.pad(q, (0, 1), value=8)
    return (q[:, 0::2] + 16 * q[:, 1::2]).to(torch.uint8).contiguous()


def matrix(codes, scales, cols, segments, group):
    return (nibbles(codes, cols) - 8).double() * scales.double()[:, group_columns(cols, segments, group)]


def random_codes(rows, cols, segments, group, g, pow2=False):
    q = torch.randint(0, 16, (rows, cols), generator=g, device="cuda")
    n = segments * -(-(cols // segments) // group)
    e = torch.randn(rows, n, generator=g, device="cuda").mul(0.7)
    if pow2:
        e = e.round()
    scales = (torch.exp2(e) * 2.0 ** round(math.log2(0.2 / math.sqrt(cols)))).to(torch.bfloat16)
    return bytes_of(q), scales


def gelu(z):
    return torch.nn.functional.gelu(z, approximate="tanh")


def forward(x, act, Ws, b1, b2):
    """y in 64 bits, and how far a result may be from it.

    A product takes its tokens as fp16 numbers times a power of two, of 128 columns or
    of the whole token: bf16's eight bits are kept down to 2^-25 of the largest, and what
    is smaller is rounded to 2^-40 of it.  Hidden activations that are kept under a bound
    instead of their largest are rounded to half of fp16's least, 2^-25, where the bound
    is 2^15: below 2^-21 of the largest for bounds up to 2^19 too high, which
    sum |x| 8 max s is for K of some thousand and random codes.
    z is off by at most e(K) sum |x w| besides: 32-bit sums of K products with their
    scales, e(K) = (K + 8) 2^-22 (four times the 2^-24 of each rounding, for the
    shortened sums of the matrix unit).  (The codes are multiplied as 0..15 and the
    offset of 8 taken off as a sum; for codes spread over 0..15 sum |code x| is below
    twice sum |(code - 8) x|, which the factor of four covers.)
    |gelu'| <= 1.13, |silu'| <= 1.1; the functions are within 2^-19 of the value for
    |value| >= 1e-3 and 2^-18 |z| absolutely.  h is rounded to fp16: 2^-8
    relative covers it.  Then the same for y and its rounding."""
    def product(v, ev, W):
        ev = ev + 2.0 ** -21 * v.abs().amax(1, keepdim=True)
        e = (v.shape[1] + 8) * 2.0 ** -22 * (v.abs() @ W.abs().T)
        return v @ W.T, e + ev @ W.abs().T
    h = x.double()
    eh = torch.zeros_like(h)
    if act == "swiglu":
        (a, ea), (g, eg) = product(h, eh, Ws[0]), product(h, eh, Ws[1])
        s = torch.nn.functional.silu(a)
        h = s * g
        eh = 1.1 * ea * g.abs() + (s.abs() + 1.1 * ea) * eg + 2.0 ** -18 * (a.abs() * g.abs())
    elif act == "gelu_tanh":
        z, ez = product(h, eh, Ws[0])
        if b1 is not None:
            z = z + b1.double()
        h = gelu(z)
        eh = 1.13 * (ez + 2.0 ** -23 * z.abs()) + 2.0 ** -18 * z.abs()
    if act != "none":
        eh = eh + 2.0 ** -8 * h.abs()
    y, ey = product(h, eh, Ws[-1])
    if b2 is not None:
        y = y + b2.double()
    return y, (1 + 2.0 ** -8) * ey + 2.0 ** -8 * y.abs() + 1e-30
