"""Cases of a block's serving pass with 4-bit weights and of the norms around its
sublayers: quantising a weight to 4-bit codes with a scale for each group of
inputs, the feed-forward sublayer (or the output projection alone) from such
weights, and the norm after a sublayer with its gate and residual scale and the
norm before the next one, forward and backward.

A case gives the sizes; values come from the seed."""
import math

import torch

own = False

DEV = "cuda"


def listed():
    quantize = dict(op="quantize")
    ffn = dict(op="ffn", bias=False)
    norm = dict(op="norm", kind="rms", dtype="bf16", before=True, after=False, shift=False, gates=0, scale=1.0)
    return [
        # one projection of a small model, row-sharded in four
        dict(quantize, name="quantize_small", rows=1024, cols=1280, group=32, segments=4),
        # the gate projection of the 70B feed-forward: what loading a large model quantises again and again
        dict(quantize, name="quantize_70b_up", rows=28672, cols=8192, group=128, segments=1),
        # one token of a small model with biases: the latency of a call
        dict(ffn, name="ffn_one_token_small", act="gelu_tanh", d=1024, d_ff=4096, shards=4, group=64, tokens=1, bias=True),
        # one token of one conversation with the 70B feed-forward: the weights' bytes
        dict(ffn, name="ffn_one_token_70b", act="swiglu", d=8192, d_ff=28672, shards=8, group=128, tokens=1),
        # a decode step of a serving batch
        dict(ffn, name="ffn_decode_70b", act="swiglu", d=8192, d_ff=28672, shards=8, group=128, tokens=32),
        # widths that fill no tile, small groups, shards whose last group is short
        dict(ffn, name="ffn_odd", act="swiglu", d=1000, d_ff=2730, shards=3, group=32, tokens=19),
        # the attention sublayer's output projection, 16 sequences with four proposed tokens each
        dict(ffn, name="out_proj_verify", act="none", d=4096, d_ff=4096, shards=8, group=128, tokens=64),
        # a prompt's tokens through the 8B feed-forward
        dict(ffn, name="ffn_prompt_8b", act="swiglu", d=4096, d_ff=14336, shards=8, group=64, tokens=389),
        # between two sublayers of a decode step: the residual sum and the next norm
        dict(norm, name="norm_decode_70b", n=32, d=8192),
        # a training pass: norms on both sides of the sublayer, a learned gate for each channel
        dict(norm, name="norm_train_8b", n=8192, d=4096, after=True, gates=1, scale=0.5),
        # its backward pass
        dict(norm, name="norm_backward_8b", op="norm_backward", n=8192, d=4096, after=True, gates=1, scale=0.5),
        # layer norms with shifts, a gate for each of 8 sequences of odd length, in 32 bits
        dict(norm, name="norm_backward_layer", op="norm_backward", kind="layer", dtype="f32", n=8 * 513, d=1160, after=True,
             shift=True, gates=8),
    ]


def _between(rng, lo, hi):
    """A whole number of lo..hi, spread over the logarithm where that is a wide range."""
    if hi > 10 * max(lo, 1):
        return int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))
    return rng.randint(lo, hi)


def draw(rng):
    op = rng.choice(["quantize", "ffn", "ffn", "norm", "norm_backward"])
    if op == "quantize":
        segments = rng.choice([1, 2, 3, 8])
        while True:
            c = dict(op=op, rows=_between(rng, 64, 32768), cols=segments * _between(rng, 64, 28672 // segments),
                     group=rng.choice([32, 64, 128]), segments=segments)
            if c["rows"] * c["cols"] <= 28672 * 8192:
                return c
    if op == "ffn":
        act = rng.choice(["swiglu", "swiglu", "gelu_tanh", "none"])
        shards = rng.choice([1, 2, 3, 4, 8])
        while True:
            s = _between(rng, 64, 28672 // shards)
            if act == "none":
                s = max(s // 8, 8) * 8
            c = dict(op=op, act=act, d=8 * _between(rng, 32, 1024), d_ff=shards * s, shards=shards,
                     group=rng.choice([32, 64, 128]), tokens=_between(rng, 1, 400), bias=act != "swiglu" and rng.random() < 0.5)
            if c["d"] * c["d_ff"] <= 28672 * 8192 and c["tokens"] * c["d"] * c["d_ff"] <= 389 * 4096 * 14336:
                return c
    c = dict(op=op, kind=rng.choice(["rms", "layer"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
             before=rng.random() < 0.8, after=rng.random() < 0.6, shift=rng.random() < 0.5,
             scale=rng.choice([1.0, 0.5, 0.125]))
    c["before"] = c["before"] or not c["after"]
    gates = rng.choice(["none", "one", "sequence", "token"])
    while True:
        n, d = _between(rng, 1, 16384), 8 * _between(rng, 8, 1024)
        if n * d <= (8192 * 4096 if c["dtype"] == "bf16" else 4096 * 4096):
            break
    if gates == "sequence":
        c["gates"] = rng.choice([2, 3, 16])
        n = max(n // c["gates"], 1) * c["gates"]
    else:
        c["gates"] = dict(none=0, one=1, token=n)[gates]
    return dict(c, n=n, d=d)


def _weights(case):
    """(rows, columns, segments) of the sublayer's matrices."""
    d, d_ff, T = case["d"], case["d_ff"], case["shards"]
    up = {"swiglu": 2, "gelu_tanh": 1, "none": 0}[case["act"]]
    return [(d_ff, d, 1)] * up + [(d, d_ff, T)]


def _groups(cols, segments, group):
    return segments * -(-(cols // segments) // group)


def work(case):
    op = case["op"]
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        codes = rows * ((cols + 1) // 2 + 2 * _groups(cols, case["segments"], case["group"]))
        # the weight read, the codes written and read again, the values that they stand for written
        return {"bytes": 4 * rows * cols + 2 * codes, "flops": 4 * rows * cols}
    if op == "ffn":
        n = case["tokens"]
        params = sum(r * c for r, c, _ in _weights(case))
        held = sum(r * ((c + 1) // 2 + 2 * _groups(c, s, case["group"])) for r, c, s in _weights(case))
        acts = n * (case["d"] + (case["d_ff"] if case["act"] == "none" else case["d"]))
        return {"bytes": held + 2 * acts, "flops": 2 * n * params}
    n, d, size = case["n"], case["d"], 2 if case["dtype"] == "bf16" else 4
    if op == "norm":
        rows = 3 + case["before"]  # x, b, r; n
    else:
        rows = 3 + 2 * case["before"] + (case["after"] or case["gates"] > 0)  # dr, dx, db; dn, r; b
    return {"bytes": size * d * (rows * n + case["gates"] * (1 if op == "norm" else 2)), "flops": 12 * n * d}


def prepare(case, seed):
    """A weight; quantised weights and the tokens' activations; the residual stream, a sublayer's output and gradients."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)
    s = dict(case=dict(case))
    op = case["op"]
    if op == "quantize":
        s["w"] = (normal(case["rows"], case["cols"]) / math.sqrt(case["cols"])).to(torch.bfloat16)
    elif op == "ffn":
        n, d, d_ff, T, group = (case[k] for k in ("tokens", "d", "d_ff", "shards", "group"))
        held = []
        for rows, cols, segments in _weights(case):
            even = normal(rows, (cols + 1) // 2).mul_(3).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
            odd = normal(rows, (cols + 1) // 2).mul_(3).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
            scale = normal(rows, _groups(cols, segments, group)).mul_(0.2).exp_() / (3 * math.sqrt(cols))
            held.append((even + 16 * odd, scale.to(torch.bfloat16)))
        s["held"] = held
        s["x"] = normal(n, d_ff if case["act"] == "none" else d).to(torch.bfloat16)
        s["b1"] = (0.1 * normal(d_ff)).to(torch.bfloat16) if case["bias"] and case["act"] == "gelu_tanh" else None
        s["b2"] = (0.1 * normal(d)).to(torch.bfloat16) if case["bias"] else None
        if own:
            from megatron_tensor_transformer_w1_gb300.ffn import TensorParallelFFN
            from megatron_tensor_transformer_w1_gb300.weights4 import Codes4
            ffn = TensorParallelFFN(d, d_ff, T, act=case["act"], device=DEV)
            codes = [Codes4(c, v, cols, group, segments)
                     for (c, v), (_, cols, segments) in zip(held, _weights(case))]
            up = codes[:-1] + [None] * (3 - len(codes))
            s["ffn"], (s["w13"], s["w2"]) = ffn, ffn.pack4(up[0], codes[-1], up[1])
    else:
        n, d = case["n"], case["d"]
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        layer = case["kind"] == "layer"
        s["x"] = (4 * normal(n, d) + (0.5 if layer else 0)).to(t)
        s["b"] = (2 * normal(n, d) + (0.25 if layer else 0)).to(t)
        for side in ("before", "after"):
            there = case[side]
            s["w_" + side] = (1 + 0.2 * normal(d)).to(t) if there else None
            s["c_" + side] = (0.2 * normal(d)).to(t) if there and case["shift"] else None
        s["gate"] = (0.5 + 0.3 * normal(case["gates"], d)).to(t) if case["gates"] else None
        if op == "norm_backward":
            # what the forward pass left: the residual stream behind the sublayer, and each row's statistics
            s["dr"] = normal(n, d).to(t)
            s["dn"] = normal(n, d).to(t) if case["before"] else None
            s["r"], _, s["stats"] = _norm(s)
        if own:
            from megatron_tensor_transformer_w1_gb300.norm import SublayerNorm
            s["norm"] = SublayerNorm(d, kind=case["kind"], before=case["before"], after=case["after"], eps=EPS,
                                     scale=case["scale"], dtype=case["dtype"], device=DEV)
    return s


EPS = 1e-5


def run(state):
    s = state
    op = s["case"]["op"]
    if op == "quantize":
        c = s["case"]
        if own:
            from megatron_tensor_transformer_w1_gb300.weights4 import dequantize4, quantize4
            codes = quantize4(s["w"], group=c["group"], segments=c["segments"])
            return {"values": dequantize4(codes), "scales": codes.scales}
        return _quantize(s["w"], c)
    if op == "ffn":
        if own:
            return s["ffn"].forward4(s["x"], s["w13"], s["w2"], b1=s["b1"], b2=s["b2"])
        return _ffn(s)
    weights = dict(w_after=s["w_after"], c_after=s["c_after"], gate=s["gate"], w_before=s["w_before"])
    if op == "norm":
        if own:
            r, n, _ = s["norm"].forward(s["x"], s["b"], c_before=s["c_before"], save=False, **weights)
        else:
            r, n, _ = _norm(s)
        return {"r": r} if n is None else {"r": r, "n": n}
    if own:
        g = s["norm"].backward(s["b"], s["r"], s["stats"], s["dr"], s["dn"],
                               shift_before=s["c_before"] is not None, **weights)
    else:
        g = _norm_backward(s)
    return {k: v for k, v in g.items() if v is not None}


# ------------------------------------------------------------ plain forms
def _by_group(a, segments, group):
    """[rows, cols] as [rows, segments, groups, group], zeros behind each segment's last column."""
    rows, cols = a.shape
    a = a.reshape(rows, segments, cols // segments)
    a = torch.nn.functional.pad(a, (0, -(cols // segments) % group))
    return a.reshape(rows, segments, -1, group)


def _quantize(w, c):
    v = _by_group(w.float(), c["segments"], c["group"])
    scale = (v.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16).float()
    code = torch.where(scale > 0, v / scale, 0).round().clamp(-8, 7)
    back = (code * scale).reshape(c["rows"], c["segments"], -1)[:, :, :c["cols"] // c["segments"]]
    return {"values": back.reshape(c["rows"], c["cols"]).to(torch.bfloat16),
            "scales": scale.reshape(c["rows"], -1).to(torch.bfloat16)}


def _values(held, cols, segments, group):
    """The matrix that codes and scales stand for, in 32 bits."""
    code, scale = held
    rows = code.shape[0]
    q = torch.stack((code & 15, code >> 4), -1).reshape(rows, -1)[:, :cols].float() - 8
    v = _by_group(q, segments, group) * scale.float().reshape(rows, segments, -1, 1)
    return v.reshape(rows, segments, -1)[:, :, :cols // segments].reshape(rows, cols)


def _ffn(s):
    c = s["case"]
    x, group = s["x"].float(), c["group"]
    if c["act"] == "swiglu":
        a = x @ _values(s["held"][0], c["d"], 1, group).T
        x = a / (1 + (-a).exp()) * (x @ _values(s["held"][1], c["d"], 1, group).T)
    elif c["act"] == "gelu_tanh":
        z = x @ _values(s["held"][0], c["d"], 1, group).T
        if s["b1"] is not None:
            z = z + s["b1"].float()
        x = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    y = x @ _values(s["held"][-1], c["d_ff"], c["shards"], group).T
    if s["b2"] is not None:
        y = y + s["b2"].float()
    return y.to(torch.bfloat16)


def _unit(x, kind):
    """x with mean 0 (layer) and mean square 1 in each row, the mean and the factor."""
    mean = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    factor = 1 / (((x - mean) * (x - mean)).mean(-1, keepdim=True) + EPS).sqrt()
    return (x - mean) * factor, mean, factor


def _gates(s, rows):
    """The gate of every token, times the residual scale."""
    if s["gate"] is None:
        return torch.full_like(rows, s["case"]["scale"])
    return s["gate"].float().repeat_interleave(rows.shape[0] // s["gate"].shape[0], 0) * s["case"]["scale"]


def _affine(x, w, c):
    x = x if w is None else x * w.float()
    return x if c is None else x + c.float()


def _norm(s):
    case = s["case"]
    t = s["x"].dtype
    u = s["b"].float()
    stats = torch.zeros(u.shape[0], 4, device=DEV)
    if case["after"]:
        u, stats[:, 0:1], stats[:, 1:2] = _unit(u, case["kind"])
        u = _affine(u, s["w_after"], s["c_after"])
    r = s["x"].float() + _gates(s, u) * u
    if not case["before"]:
        return r.to(t), None, stats
    n, stats[:, 2:3], stats[:, 3:4] = _unit(r, case["kind"])
    return r.to(t), _affine(n, s["w_before"], s["c_before"]).to(t), stats


def _unit_backward(dy, y, factor, kind):
    """Gradient of x where y = _unit(x)."""
    dx = dy - y * (dy * y).mean(-1, keepdim=True)
    if kind == "layer":
        dx = dx - dy.mean(-1, keepdim=True)
    return dx * factor


def _norm_backward(s):
    case = s["case"]
    t, kind, st = s["r"].dtype, case["kind"], s["stats"]
    out = dict(dx=None, db=None, dgate=None, dw_after=None, dc_after=None, dw_before=None, dc_before=None)
    g = s["dr"].float()
    if case["before"]:
        y, dn = (s["r"].float() - st[:, 2:3]) * st[:, 3:4], s["dn"].float()
        out["dw_before"] = (dn * y).sum(0)
        if s["c_before"] is not None:
            out["dc_before"] = dn.sum(0)
        g = g + _unit_backward(dn * s["w_before"].float(), y, st[:, 3:4], kind)
    out["dx"] = g
    u = b = s["b"].float()
    if case["after"]:
        b = (b - st[:, 0:1]) * st[:, 1:2]
        u = _affine(b, s["w_after"], s["c_after"])
    if s["gate"] is not None:
        out["dgate"] = (g * u).reshape(case["gates"], -1, case["d"]).sum(1) * case["scale"]
    du = g * _gates(s, g)
    if case["after"]:
        out["dw_after"] = (du * b).sum(0)
        if s["c_after"] is not None:
            out["dc_after"] = du.sum(0)
        du = _unit_backward(du * s["w_after"].float(), b, st[:, 1:2], kind)
    out["db"] = du
    return {k: None if v is None else v.to(t) for k, v in out.items()}


# ------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        rows, cols, T, group = case["rows"], case["cols"], case["segments"], case["group"]
        w, width = s["w"], cols // case["segments"]
        values = torch.empty(rows, cols, dtype=torch.float64, device=DEV)
        scales = []
        for t in range(T):
            for first in range(t * width, (t + 1) * width, group):
                part = w[:, first:min(first + group, (t + 1) * width)].double()
                unit = (part.abs().max(1).values / 7).to(torch.bfloat16).double()
                steps = torch.round(part / unit[:, None].clamp(min=1e-300)).clamp(-8, 7)
                values[:, first:first + part.shape[1]] = steps * unit[:, None]
                scales.append(unit)
        return {"values": values, "scales": torch.stack(scales, 1)}
    if case["op"] == "ffn":
        T, group = case["shards"], case["group"]

        def matrix(at):
            rows, cols, segments = _weights(case)[at]
            code, scale = s["held"][at]
            j = torch.arange(cols, device=DEV)
            nibble = (code[:, j // 2].int() >> (4 * (j % 2)).int()) & 15
            width = cols // segments
            column = (j // width) * -(-width // group) + (j % width) // group
            return (nibble.double() - 8).mul_(scale.double()[:, column])
        h = s["x"].double()
        if case["act"] == "gelu_tanh":
            z = h @ matrix(0).T + (0 if s["b1"] is None else s["b1"].double())
            h = torch.nn.functional.gelu(z, approximate="tanh")
        elif case["act"] == "swiglu":
            h = torch.nn.functional.silu(h @ matrix(0).T) * (h @ matrix(1).T)
        return h @ matrix(-1).T + (0 if s["b2"] is None else s["b2"].double())
    n, d = case["n"], case["d"]
    leaves = {k: s[k].double().requires_grad_() for k in ("x", "b", "gate", "w_after", "c_after", "w_before", "c_before")
              if s[k] is not None}

    def normed(v, side):
        if case["kind"] == "layer":
            return torch.nn.functional.layer_norm(v, (d,), leaves["w_" + side], leaves.get("c_" + side), EPS)
        v = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * leaves["w_" + side]
        return v + leaves["c_" + side] if "c_" + side in leaves else v
    u = normed(leaves["b"], "after") if case["after"] else leaves["b"]
    if "gate" in leaves:
        per = n // case["gates"]
        u = (u.view(case["gates"], per, d) * leaves["gate"][:, None]).view(n, d)
    if case["op"] == "norm":
        r = leaves["x"] + case["scale"] * u
        out = {"r": r.detach()}
        if case["before"]:
            out["n"] = normed(r, "before").detach()
        return out
    # the gradients at the residual stream that was stored
    r = s["r"].double().requires_grad_()
    g = s["dr"].double()
    found = {}
    if case["before"]:
        wanted = [k for k in ("w_before", "c_before") if k in leaves]
        got = torch.autograd.grad(normed(r, "before"), [r] + [leaves[k] for k in wanted], s["dn"].double())
        g = g + got[0]
        found.update(zip(wanted, got[1:]))
    wanted = [k for k in ("b", "gate", "w_after", "c_after") if k in leaves]
    found.update(zip(wanted, torch.autograd.grad(case["scale"] * u, [leaves[k] for k in wanted], g)))
    names = dict(b="db", gate="dgate", w_after="dw_after", c_after="dc_after", w_before="dw_before", c_before="dc_before")
    return {"dx": g, **{v: found[k] for k, v in names.items() if k in found}}
