"""The norms around a block's sublayers against plain 64-bit forms, forward and
backward, and against autograd and differences in 64 bits.

Tolerances.  An output is rounded to its type: 2^-8 of the value (bf16), 2^-24 (32
bits).  What is computed in 32 bits is off by at most E = 2^-16 times the sum of the
absolute values of its terms, formed alongside: a row's sum is 8 additions in a
thread, 5 + 5 in trees and at most 32 more, below 2^6 roundings of 2^-24, with as
many for its factor; a column's sum over n tokens adds at most n / 128 + 200 of them
(n <= 5000 here: below 2^8), after the roundings of its terms."""
import pytest
import torch

pytestmark = pytest.mark.gpu
E = 2.0 ** -16
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _norm(d, **kw):
    from megatron_tensor_transformer_w1_gb300.norm import SublayerNorm
    return SublayerNorm(d, **kw)


def _inputs(n, d, dtype, before, after, shift, gates, seed=0, mean=0.4):
    g = torch.Generator(device="cuda").manual_seed(seed + n * 31 + d)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    t = TYPES[dtype]
    s = dict(x=(3 * r(n, d) + mean).to(t), b=(2 * r(n, d) - mean).to(t), dr=r(n, d).to(t))
    s["dout"] = r(n, d).to(t) if before else None
    for name, there in (("after", after), ("before", before)):
        s["w_" + name] = (1 + 0.3 * r(d)).to(t) if there else None
        s["c_" + name] = (0.3 * r(d)).to(t) if there and shift else None
    s["gate"] = (0.5 + 0.5 * r(gates, d)).to(t) if gates else None
    return s


D = lambda v: None if v is None else v.double()


def unit(v, kind, eps):
    """(y, mean, factor, absolute error of y in units of E)."""
    m = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    f = ((v - m).square().mean(1, keepdim=True) + eps).rsqrt()
    y = (v - m) * f
    return y, m, f, f * (v.abs() + v.abs().mean(1, keepdim=True)) + y.abs() * (1 + (f * m).abs())


def wide(gate, n):
    return 1.0 if gate is None else gate.double().repeat_interleave(n // gate.shape[0], 0)


def ref_forward(s, kind, before, after, scale, eps):
    """{name: (value, absolute sums)} of r, out and the stats."""
    n = s["x"].shape[0]
    u, eu = D(s["b"]), D(s["b"]).abs()
    out = {}
    if after:
        y, m, f, e = unit(u, kind, eps)
        out["stats_after"] = torch.cat((m, f), 1)
        w = D(s["w_after"])
        u, eu = y * w, e * w.abs()
        if s["c_after"] is not None:
            u, eu = u + D(s["c_after"]), eu + D(s["c_after"]).abs()
    k = scale * wide(s["gate"], n)
    r = D(s["x"]) + k * u
    er = D(s["x"]).abs() + abs(scale) * (k / scale if not torch.is_tensor(k) else (k / scale).abs()) * eu
    out["r"] = r, er
    if before:
        y, m, f, e = unit(r, kind, eps)
        out["stats_before"] = torch.cat((m, f), 1)
        e = e + f * (er + er.mean(1, keepdim=True)) + y.abs() * f * er.square().mean(1, keepdim=True).sqrt()
        w = D(s["w_before"])
        o, eo = y * w, e * w.abs()
        if s["c_before"] is not None:
            o, eo = o + D(s["c_before"]), eo + D(s["c_before"]).abs()
        out["out"] = o, eo
    return out


def ref_backward(s, r, stats, kind, before, after, scale):
    """Gradients from the formulas, with the stored r and statistics: {name: (value, absolute sums)}."""
    n, d = r.shape
    st = D(stats) if stats is not None else None
    mean = lambda v: v.mean(1, keepdim=True)
    layer = kind == "layer"

    def back(dy, edy, y, f):
        a = mean(dy * y)
        g, eg = dy - y * a, edy + y.abs() * mean(edy * y.abs())
        if layer:
            g, eg = g - mean(dy), eg + mean(edy)
        return f * g, f * eg
    out = {}
    g, eg = (D(s["dr"]), D(s["dr"]).abs()) if s["dr"] is not None else (torch.zeros(n, d, device="cuda", dtype=torch.float64),) * 2
    if before:
        y, do, w = (D(r) - st[:, 2:3]) * st[:, 3:4], D(s["dout"]), D(s["w_before"])
        ey = y.abs() + 2 * (st[:, 3:4] * D(r)).abs()
        out["dw_before"] = (do * y).sum(0), (do.abs() * ey).sum(0)
        out["dc_before"] = do.sum(0), do.abs().sum(0)
        dg, e = back(do * w, (do * w).abs(), y, st[:, 3:4])
        g, eg = g + dg, eg + e + st[:, 3:4] * (do * w).abs() * ey
    out["dx"] = g, eg
    u = y = D(s["b"])
    ey = y.abs()
    if after:
        y = (y - st[:, 0:1]) * st[:, 1:2]
        ey = y.abs() + 2 * (st[:, 1:2] * D(s["b"])).abs()
        u = y * D(s["w_after"]) + (0 if s["c_after"] is None else D(s["c_after"]))
    eu = ey * (D(s["w_after"]).abs() if after else 1) + (0 if s["c_after"] is None else D(s["c_after"]).abs())
    if s["gate"] is not None:
        G = s["gate"].shape[0]
        out["dgate"] = tuple(v.view(G, -1, d).sum(1) for v in (scale * g * u, abs(scale) * eg * eu))
    k = scale * wide(s["gate"], n)
    ak = abs(k) if not torch.is_tensor(k) else k.abs()
    du, edu = k * g, ak * eg
    if after:
        out["dw_after"] = (du * y).sum(0), (edu * ey).sum(0)
        out["dc_after"] = du.sum(0), edu.sum(0)
        w = D(s["w_after"])
        du, edu = back(du * w, edu * w.abs() * (1 + ey / (y.abs() + 1)), y, st[:, 1:2])
    out["db"] = du, edu
    return out


def close(name, got, want, dtype):
    value, sums = want
    tol = (1 + 2.0 ** -7) * (HALF_STEP[dtype] * value.abs() + E * sums) + 1e-30
    err = (got.double() - value).abs()
    assert torch.isfinite(got).all() and (err <= tol).all(), (name, (err / tol).max().item())


CASES = [  # n, d, gates
    (1, 8, 0), (1, 8192, 1), (3, 64, 3), (5, 256, 5), (7, 264, 1), (33, 1160, 0), (64, 1024, 4), (300, 768, 3),
    (2000, 128, 2), (4096, 40, 1024), (1201, 512, 1201), (700, 2048, 7), (160, 4096, 1), (320, 5000, 2), (35, 8192, 5), (4097, 1600, 1)]
FORMS = [("rms", True, False, False), ("rms", True, True, False), ("layer", True, True, True), ("layer", False, True, True),
         ("rms", False, False, False), ("layer", True, False, False), ("rms", True, True, True)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,before,after,shift", FORMS)
def test_norm(kind, before, after, shift, dtype):
    for n, d, gates in CASES:
        scale = 0.5 if n % 2 else 1.0
        s = _inputs(n, d, dtype, before, after, shift, gates)
        norm = _norm(d, kind=kind, before=before, after=after, eps=1e-5, scale=scale, dtype=dtype)
        w = dict(w_after=s["w_after"], c_after=s["c_after"], gate=s["gate"], w_before=s["w_before"])
        r, out, stats = norm.forward(s["x"], s["b"], c_before=s["c_before"], **w)
        want = ref_forward(s, kind, before, after, scale, 1e-5)
        close("r", r, want["r"], dtype)
        assert (out is None) == (not before)
        if before:
            close("out", out, want["out"], dtype)
        for at, name in ((0, "stats_after"), (2, "stats_before")):
            if name in want:
                m, f = want[name][:, 0], want[name][:, 1]
                size = (s["b"] if at == 0 else want["r"][0]).double().abs().mean(1)
                assert ((stats[:, at].double() - m).abs() <= 4 * E * size).all()
                assert ((stats[:, at + 1].double() / f - 1).abs() <= 4 * E * (1 + (f * m).square())).all()
        g = norm.backward(s["b"], r, stats, s["dr"], s["dout"], shift_before=s["c_before"] is not None, **w)
        back = ref_backward(s, r, stats, kind, before, after, scale)
        expected = {"dx", "db"} | ({"dgate"} if gates else set()) | ({"dw_after"} if after else set()) | (
            {"dw_before"} if before else set()) | ({"dc_after"} if after and shift else set()) | (
            {"dc_before"} if before and shift else set())
        assert {k for k, v in g.items() if v is not None} == expected
        for name in expected:
            close((name, n, d, gates), g[name], back[name], dtype)
        again = norm.backward(s["b"], r, stats, s["dr"], s["dout"], shift_before=s["c_before"] is not None, **w)
        assert all(v is None or torch.equal(v, again[k]) for k, v in g.items())


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradients_are_those_of_autograd_and_of_differences(kind):
    n, d, gates, scale = 12, 48, 3, 0.7
    s = _inputs(n, d, "f32", True, True, True, gates, seed=5)
    norm = _norm(d, kind=kind, after=True, eps=1e-3, scale=scale, dtype="f32")
    leaves = {k: s[k].double().requires_grad_() for k in ("x", "b", "w_after", "c_after", "gate", "w_before", "c_before")}

    def loss(v):
        q = dict(s, **v)
        f = ref_forward(q, kind, True, True, scale, 1e-3)
        return (f["r"][0] * D(s["dr"])).sum() + (f["out"][0] * D(s["dout"])).sum()
    value = loss(leaves)
    auto = dict(zip(leaves, torch.autograd.grad(value, list(leaves.values()))))
    w = dict(w_after=s["w_after"], c_after=s["c_after"], gate=s["gate"], w_before=s["w_before"])
    r, _, stats = norm.forward(s["x"], s["b"], c_before=s["c_before"], **w)
    g = norm.backward(s["b"], r, stats, s["dr"], s["dout"], shift_before=True, **w)
    back = ref_backward(s, r, stats, kind, True, True, scale)
    generator = torch.Generator(device="cuda").manual_seed(1)
    for leaf, name in (("x", "dx"), ("b", "db"), ("gate", "dgate"), ("w_after", "dw_after"), ("c_after", "dc_after"),
                       ("w_before", "dw_before"), ("c_before", "dc_before")):
        # r is stored in 32 bits here: the formulas' error and r's rounding, 2^-24 of a factor of order one
        tol = 2 * E * back[name][1] + 1e-30
        assert ((g[name].double() - auto[leaf]).abs() <= tol).all(), name
        v = torch.randn(leaves[leaf].shape, generator=generator, device="cuda", dtype=torch.float64)
        h = 1e-4
        with torch.no_grad():
            slope = (loss(dict(leaves, **{leaf: leaves[leaf] + h * v})) - loss(dict(leaves, **{leaf: leaves[leaf] - h * v}))) / (2 * h)
        # central differences: h^2 / 6 of a third derivative, below 1e-5 of the gradient's size here
        assert abs(slope - (g[name].double() * v).sum()) <= 1e-4 * g[name].double().norm() * v.norm() / v.numel() ** 0.5 + (tol * v.abs()).sum()


def test_first_norm_without_a_sublayer_and_unweighted():
    s = _inputs(9, 520, "bf16", True, False, False, 0)
    norm = _norm(520, eps=1e-6)
    r, out, stats = norm.forward(s["x"])
    assert torch.equal(r, s["x"])
    x = s["x"].double()
    want = x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    close("out", out, (want, 2 * want.abs()), "bf16")
    g = norm.backward(None, r, stats, None, s["dout"])
    q = dict(s, w_before=torch.ones(520, device="cuda"), dr=None)
    close("dx", g["dx"], ref_backward(q, r, stats, "rms", True, False, 1.0)["dx"], "bf16")
    assert all(g[k] is None for k in ("db", "dgate", "dw_after", "dc_after", "dw_before", "dc_before"))


def test_rows_of_zeros_of_one_value_and_with_what_is_not_finite():
    """A row without spread has the factor 1 / sqrt(eps); a bad row spoils itself alone."""
    n, d = 40, 768
    for kind in ("rms", "layer"):
        s = _inputs(n, d, "bf16", True, True, True, 1)
        s["b"][3] = 0
        s["x"][3] = 0
        s["b"][4] = 2.5
        norm = _norm(d, kind=kind, after=True)
        w = dict(w_after=s["w_after"], c_after=s["c_after"], gate=s["gate"], w_before=s["w_before"], c_before=s["c_before"])
        r, out, stats = norm.forward(s["x"], s["b"], **w)
        want = ref_forward(s, kind, True, True, 1.0, 1e-5)
        close("r", r, want["r"], "bf16")
        close("out", out, want["out"], "bf16")
        clean = r.clone(), out.clone()
        s["b"][7, 5], s["x"][9, 700], s["b"][11, 0] = float("nan"), float("inf"), -float("inf")
        r, out, stats = norm.forward(s["x"], s["b"], **w)
        rest = torch.ones(n, dtype=torch.bool, device="cuda")
        rest[[7, 9, 11]] = False
        assert torch.equal(r[rest], clean[0][rest]) and torch.equal(out[rest], clean[1][rest])
        assert torch.isnan(out[[7, 9, 11]]).all(1).any() and not torch.isfinite(out[7]).any()


def test_in_place_streams_and_replays():
    n, d = 70, 1024
    s = _inputs(n, d, "bf16", True, True, False, 1)
    norm = _norm(d, after=True, scale=0.5)
    w = dict(w_after=s["w_after"], gate=s["gate"], w_before=s["w_before"])
    r, out, stats = norm.forward(s["x"], s["b"], **w)
    g = norm.backward(s["b"], r, stats, s["dr"], s["dout"], **w)
    x = s["x"].clone()
    r2, out2, _ = norm.forward(x, s["b"], r_out=x, save=False, **w)
    assert r2 is x and torch.equal(x, r) and torch.equal(out2, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g2 = norm.backward(s["b"], r, stats, s["dr"], s["dout"], **w)
    torch.cuda.current_stream().wait_stream(side)
    assert all(v is None or torch.equal(v, g2[k]) for k, v in g.items())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r3, out3, stats3 = norm.forward(s["x"], s["b"], **w)
        g3 = norm.backward(s["b"], r3, stats3, s["dr"], s["dout"], **w)
    for _ in range(2):
        for v in (r3, out3, *(v for v in g3.values() if v is not None)):
            v.fill_(9)
        graph.replay()
        norm.backward(s["b"], r, stats, s["dout"], s["dr"], **w)  # an eager call between
        assert torch.equal(r3, r) and torch.equal(out3, out)
        assert all(v is None or torch.equal(v, g3[k]) for k, v in g.items())


def test_empty():
    norm = _norm(64, after=True)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    r, out, stats = norm.forward(e, e, w_after=w, w_before=w)
    assert r.shape == out.shape == (0, 64)
    g = norm.backward(e, r, stats, e, e, w_after=w, w_before=w)
    assert (g["dw_after"] == 0).all() and (g["dw_before"] == 0).all()


@pytest.mark.parametrize("kind,dtype,d", [("layer", "bf16", 3000), ("rms", "bf16", 1400), ("layer", "f32", 1504), ("rms", "f32", 3000)])
def test_slots_of_48_kib(monkeypatch, kind, dtype, d):
    """Rows whose slots take all of the shared memory that a kernel may have unasked."""
    monkeypatch.setitem(globals(), "CASES", [(n, d, gates) for n, gates in ((451, 451), (800, 1), (200, 0))])
    test_norm(kind, True, True, kind == "layer", dtype)
