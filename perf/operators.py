"""Cases of the serving operators of the attention sublayer: appending keys and
values to the paged cache (with the rotation by position), and attention over
that cache, with a prefix that all sequences of the batch share.

A case gives head counts, page size and how many sequences, new tokens and
context tokens there are; the lengths of single sequences are spread over the
case's ranges by a fixed rule, the values and the pages' order come from the
seed."""
import math

import torch

own = False

HD = 128  # head width
DEV = "cuda"


def listed():
    append = dict(op="append", rotary=128, interleaved=False)
    attend = dict(op="attend", lse=False)
    return [
        # one new token of one conversation: the latency of a call
        dict(append, name="append_one_token", heads=32, kv_heads=8, shards=8, page=16, seqs=1, new_lo=1, new_hi=1,
             ctx_lo=1000, ctx_hi=1000, shared=0),
        # a decode step of a serving batch
        dict(append, name="append_decode_batch", heads=64, kv_heads=8, shards=8, page=64, seqs=128, new_lo=1,
             new_hi=1, ctx_lo=16, ctx_hi=4096, shared=0),
        # prompts of several requests in one pass
        dict(append, name="append_prompts", heads=32, kv_heads=8, shards=8, page=64, seqs=8, new_lo=301,
             new_hi=4096, ctx_lo=0, ctx_hi=2000, shared=0),
        # adjacent pairs, half the width rotated, far positions, groups of four query heads, odd lengths
        dict(append, name="append_far_interleaved", heads=20, kv_heads=5, shards=5, page=32, seqs=3, new_lo=33,
             new_hi=777, ctx_lo=9999, ctx_hi=131071, shared=0, rotary=64, interleaved=True),
        # one new token of one short conversation: the latency of a call
        dict(attend, name="decode_one_short", heads=32, kv_heads=8, shards=8, page=16, seqs=1, new_lo=1, new_hi=1,
             ctx_lo=511, ctx_hi=511, shared=0),
        # a decode step of a batch with very different context lengths
        dict(attend, name="decode_ragged_batch", heads=64, kv_heads=8, shards=8, page=64, seqs=32, new_lo=1,
             new_hi=1, ctx_lo=64, ctx_hi=16384, shared=0, lse=True),
        # one conversation with a very long context
        dict(attend, name="decode_long", heads=32, kv_heads=8, shards=8, page=128, seqs=1, new_lo=1, new_hi=1,
             ctx_lo=131071, ctx_hi=131071, shared=0),
        # a few proposed tokens per sequence are verified; a key head per query head
        dict(attend, name="verify_odd", heads=16, kv_heads=16, shards=4, page=16, seqs=7, new_lo=1, new_hi=5,
             ctx_lo=100, ctx_hi=5000, shared=0, lse=True),
        # a decode step of a batch behind one long system prompt
        dict(attend, name="shared_decode_batch", heads=32, kv_heads=8, shards=8, page=64, seqs=64, new_lo=1,
             new_hi=1, ctx_lo=16, ctx_hi=1024, shared=8192),
        # a few continuations of one long document
        dict(attend, name="shared_few", heads=8, kv_heads=2, shards=2, page=32, seqs=4, new_lo=4, new_hi=4,
             ctx_lo=1, ctx_hi=300, shared=32768, lse=True),
        # chunks of long prompts
        dict(attend, name="prompt_chunks", heads=32, kv_heads=8, shards=8, page=64, seqs=4, new_lo=300,
             new_hi=2048, ctx_lo=1000, ctx_hi=16384, shared=0),
        # the requests' own prompts behind one system prompt
        dict(attend, name="shared_prompts", heads=32, kv_heads=8, shards=8, page=128, seqs=16, new_lo=50,
             new_hi=512, ctx_lo=0, ctx_hi=0, shared=4096),
    ]


def _between(rng, lo, hi):
    """A whole number of lo..hi, spread over the logarithm where that is a wide range."""
    if hi > 10 * max(lo, 1):
        return int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))
    return rng.randint(lo, hi)


def draw(rng):
    kv = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 4, 5, 8])
    c = dict(op=rng.choice(["append", "attend", "attend"]), heads=kv * group, kv_heads=kv,
             shards=rng.choice([t for t in (1, 2, 4, 5, 8) if kv % t == 0]), page=rng.choice([8, 16, 32, 64, 128, 256]),
             seqs=_between(rng, 1, 128))
    kind = rng.choice(["one", "one", "few", "many"])
    c["new_lo"] = {"one": 1, "few": rng.randint(1, 3), "many": _between(rng, 1, 300)}[kind]
    c["new_hi"] = {"one": 1, "few": rng.randint(3, 8), "many": _between(rng, 300, 2048)}[kind]
    c["ctx_lo"] = rng.choice([0, _between(rng, 1, 1000)])
    c["ctx_hi"] = _between(rng, 1000, 65536)
    c["shared"] = 0
    if c["op"] == "append":
        c["rotary"] = rng.choice([0, 32, 64, 96, 128])
        c["interleaved"] = rng.random() < 0.4
        c["ctx_hi"] = min(c["ctx_hi"], 8192)
    else:
        c["lse"] = rng.random() < 0.4
        if rng.random() < 0.5:
            c["shared"] = max(1, _between(rng, 64, 16384) // c["page"]) * c["page"]
    # no dearer than the largest listed cases
    while True:
        new, ctx = _lengths(c)
        longest = max(ctx) + max(new)
        w = work(c)
        scores = c["seqs"] * c["heads"] * max(new) * longest + sum(new) * c["heads"] * c["shared"]
        gathered = (c["seqs"] * longest + c["shared"]) * c["kv_heads"] * HD
        held = (sum(new) + sum(ctx)) * c["kv_heads"] * HD
        if (w["bytes"] <= 5e8 and w["flops"] <= 1.5e11 and scores <= 6e8 and gathered <= 5e8 and held <= 1.2e8):
            return c
        if c["seqs"] > 1 and rng.random() < 0.5:
            c["seqs"] = c["seqs"] // 2
        elif c["new_hi"] > 64 and rng.random() < 0.5:
            c["new_hi"] = c["new_hi"] * 2 // 3
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
        else:
            c["ctx_hi"] = max(c["ctx_hi"] * 2 // 3, 1)
            c["ctx_lo"] = min(c["ctx_lo"], c["ctx_hi"])


def _lengths(case):
    """New tokens and own context tokens of each sequence: multiples of the golden ratio spread over the case's ranges."""
    def spread(lo, hi, shift):
        out = []
        for i in range(case["seqs"]):
            u = ((i + 1) * 0.6180339887498949 + shift) % 1.0
            if hi > 10 * max(lo, 1):
                a = max(lo, 1)
                out.append(min(hi, int(a * (hi / a) ** u)))
            else:
                out.append(min(hi, lo + int(u * (hi - lo + 1))))
        return out
    return spread(case["new_lo"], case["new_hi"], 0.25), spread(case["ctx_lo"], case["ctx_hi"], 0.0)


def work(case):
    new, ctx = _lengths(case)
    n, H, Hkv, shared = sum(new), case["heads"], case["kv_heads"], case["shared"]
    if case["op"] == "append":
        elems = n * (H + 2 * Hkv) * HD
        return {"bytes": 4 * elems, "flops": 3 * n * (H + Hkv) * case["rotary"]}
    keys = shared + sum(a + b for a, b in zip(new, ctx))
    seen = sum(q * (shared + c) + q * (q + 1) // 2 for q, c in zip(new, ctx))
    return {"bytes": keys * Hkv * HD * 4 + n * H * HD * 4 + (4 * n * H if case["lse"] else 0),
            "flops": 4 * HD * H * seen}


def prepare(case, seed):
    """A cache that already holds the contexts, the page table of the batch and the new tokens' projections."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    H, Hkv, page, B, shared = case["heads"], case["kv_heads"], case["page"], case["seqs"], case["shared"]
    new, ctx = _lengths(case)
    n = sum(new)
    first = shared // page  # pages that all sequences share
    own_pages = [-(-(a + b) // page) for a, b in zip(new, ctx)]
    n_pages = first + sum(own_pages) + 3  # a few are free
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    width = first + max(own_pages)
    col = torch.arange(width, device=DEV)[None, :]
    start = torch.tensor([first + sum(own_pages[:b]) for b in range(B)], device=DEV)[:, None]
    length = torch.tensor(own_pages, device=DEV)[:, None]
    at = torch.where(col < first, col, start + col - first)
    table = torch.where(col < first + length, order[at.clamp(max=n_pages - 1)], 0).to(torch.int32).contiguous()
    cu = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    kv_len = torch.tensor([shared + a + b for a, b in zip(new, ctx)], dtype=torch.int32, device=DEV)

    def values(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    s = dict(case=dict(case), cu=cu, kv_len=kv_len, table=table, n=n, most=max(new),
             k=values(n_pages, Hkv, page, HD), v=values(n_pages, Hkv, page, HD), inv_freq=None)
    if case["op"] == "append":
        s["qkv"] = values(n, (H + 2 * Hkv) * HD)
        if case["rotary"]:
            j = torch.arange(case["rotary"] // 2, device=DEV, dtype=torch.float64)
            s["inv_freq"] = (500000.0 ** (-2 * j / case["rotary"])).to(torch.float32)
    else:
        s["q"] = (1.5 * values(n, H * HD).float()).to(torch.bfloat16)
    if own:
        from megatron_tensor_transformer_w1_gb300.attention import TensorParallelAttention
        from megatron_tensor_transformer_w1_gb300.kv_cache import PagedKVCache
        attn = TensorParallelAttention(H * HD, H, Hkv, HD, case["shards"], causal=True, device=DEV)
        s["cache"] = PagedKVCache(attn, n_pages, page, k=s["k"], v=s["v"], inv_freq=s["inv_freq"],
                                  interleaved=case.get("interleaved", False))
        s["batch"] = s["cache"].batch(cu, kv_len, table, n_tokens=n, max_new=max(new))
    return s


def run(state):
    case = state["case"]
    if case["op"] == "append":
        if own:
            q = state["cache"].append(state["qkv"], state["batch"])
        else:
            q = _append(state)
        return {"q": q, "k": state["k"], "v": state["v"]}
    if own:
        return state["cache"].attend(state["q"], state["batch"], shared_len=case["shared"], lse=case["lse"])
    return _attend(state)


# ------------------------------------------------------------ plain forms
def _tokens(state):
    """Sequence and position of every new token."""
    cu, kv_len = state["cu"].long(), state["kv_len"].long()
    row = torch.arange(state["n"], device=DEV)
    seq = torch.bucketize(row, cu[1:], right=True)
    return seq, kv_len[seq] - cu[seq + 1] + row


def _rotate(x, pos, inv_freq, interleaved):
    """x [n, heads, 128], in 32 bits; the angles in 64."""
    r = 2 * inv_freq.numel()
    angle = pos.double()[:, None] * inv_freq.double()[None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _append(state):
    case = state["case"]
    H, Hkv, T, page, n = case["heads"], case["kv_heads"], case["shards"], case["page"], state["n"]
    x = state["qkv"].float().view(n, T, (H + 2 * Hkv) // T, HD)
    q = x[:, :, :H // T].reshape(n, H, HD)
    k = x[:, :, H // T:(H + Hkv) // T].reshape(n, Hkv, HD)
    v = x[:, :, (H + Hkv) // T:].reshape(n, Hkv, HD)
    seq, pos = _tokens(state)
    if state["inv_freq"] is not None:
        q = _rotate(q, pos, state["inv_freq"], case["interleaved"])
        k = _rotate(k, pos, state["inv_freq"], case["interleaved"])
    pages = state["table"][seq, pos // page].long()
    state["k"][pages, :, pos % page] = k.to(torch.bfloat16)
    state["v"][pages, :, pos % page] = v.to(torch.bfloat16)
    return q.reshape(n, H * HD).to(torch.bfloat16)


def _attend(state):
    """Scores against the shared keys for all rows at once, and against each
    sequence's own keys, padded to the longest; one softmax over both."""
    case = state["case"]
    H, Hkv, page, B, n, shared = case["heads"], case["kv_heads"], case["page"], case["seqs"], state["n"], case["shared"]
    G, most = H // Hkv, state["most"]
    cu, kv_len, table = state["cu"].long(), state["kv_len"].long(), state["table"].long()
    seq, pos = _tokens(state)
    row = torch.arange(n, device=DEV) - cu[seq]
    q = state["q"].float().view(n, Hkv, G, HD) * HD ** -0.5
    # own keys and values [B, Hkv, L, 128]
    pages = table[:, shared // page:]
    L = pages.shape[1] * page
    k = state["k"][pages].float().transpose(1, 2).reshape(B, Hkv, L, HD)
    v = state["v"][pages].float().transpose(1, 2).reshape(B, Hkv, L, HD)
    padded = torch.zeros(B, most, Hkv, G, HD, device=DEV)
    padded[seq, row] = q
    s = torch.matmul(padded.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * most, HD), k.transpose(-1, -2))
    s = s.view(B, Hkv, G, most, L).permute(0, 3, 1, 2, 4)
    last = kv_len[:, None] - (cu[1:] - cu[:-1])[:, None] + torch.arange(most, device=DEV)[None, :] - shared
    s = s.masked_fill((torch.arange(L, device=DEV) > last[:, :, None])[:, :, None, None, :], -math.inf)
    m = s.amax(-1)
    if shared:
        first = table[0, :shared // page]
        k0 = state["k"][first].float().transpose(0, 1).reshape(Hkv, shared, HD)
        v0 = state["v"][first].float().transpose(0, 1).reshape(Hkv, shared, HD)
        s0 = torch.matmul(q.permute(1, 2, 0, 3).reshape(Hkv, G * n, HD), k0.transpose(-1, -2)).view(Hkv, G, n, shared)
        m0 = s0.amax(-1).permute(2, 0, 1)
        top = torch.maximum(m[seq, row], m0)
        m = m.index_put((seq, row), top)
    e = (s - m[..., None]).exp()
    total = e.sum(-1)
    o = torch.matmul(e.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * most, L), v)
    o = o.view(B, Hkv, G, most, HD).permute(0, 3, 1, 2, 4)[seq, row]
    m, total = m[seq, row], total[seq, row]
    if shared:
        e0 = (s0 - m.permute(1, 2, 0)[..., None]).exp()
        total = total + e0.sum(-1).permute(2, 0, 1)
        o0 = torch.matmul(e0.view(Hkv, G * n, shared), v0).view(Hkv, G, n, HD)
        o = o + o0.permute(2, 0, 1, 3)
    o = (o / total[..., None]).reshape(n, H * HD).to(torch.bfloat16)
    if not case["lse"]:
        return o
    return o, ((m + total.log()) * math.log2(math.e)).reshape(n, H)


# ------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    H, Hkv, page, T, n = case["heads"], case["kv_heads"], case["page"], case["shards"], s["n"]
    G = H // Hkv
    cu, lens = s["cu"].tolist(), s["kv_len"].tolist()
    if case["op"] == "append":
        k, v = s["k"].double(), s["v"].double()
        q = torch.empty(n, H, HD, dtype=torch.float64, device=DEV)
        x = s["qkv"].double().view(n, -1, HD)
        per, hq, hk = (H + 2 * Hkv) // T, H // T, Hkv // T
        r = case["rotary"]
        # where each column's partner is and the sign of its sine: y_c = x_c cos + sign_c x_partner sin
        c = torch.arange(HD, device=DEV)
        if case["interleaved"]:
            partner, freq, sign = c ^ 1, c // 2, (c % 2) * 2 - 1
        else:
            low = c < r // 2
            partner, freq, sign = torch.where(low, c + r // 2, c - r // 2), torch.where(low, c, c - r // 2), 1 - 2 * low.long()
        partner, freq = torch.where(c < r, partner, c), torch.where(c < r, freq, 0)

        def turn(y, pos):
            if not r:
                return y
            angle = pos.double()[:, None] * s["inv_freq"].double()[freq][None, :]
            rotated = y * angle.cos()[:, None] + sign * y[..., partner] * angle.sin()[:, None]
            return torch.where(c < r, rotated, y)
        for b in range(case["seqs"]):
            rows = torch.arange(cu[b], cu[b + 1], device=DEV)
            pos = lens[b] - (cu[b + 1] - rows)
            where = s["table"][b].long()[pos // page]
            for t in range(T):
                for h in range(hq):
                    q[rows, t * hq + h] = turn(x[rows, t * per + h][:, None], pos)[:, 0]
                for h in range(hk):
                    k[where, t * hk + h, pos % page] = turn(x[rows, t * per + hq + h][:, None], pos)[:, 0]
                    v[where, t * hk + h, pos % page] = x[rows, t * per + hq + hk + h]
        return {"q": q.view(n, H * HD), "k": k, "v": v}
    o = torch.empty(n, H, HD, dtype=torch.float64, device=DEV)
    lse = torch.empty(n, H, dtype=torch.float64, device=DEV)
    for b in range(case["seqs"]):
        where = s["table"][b, : -(-lens[b] // page)].long()
        rows = slice(cu[b], cu[b + 1])
        new = cu[b + 1] - cu[b]
        hidden = torch.ones(new, lens[b], dtype=torch.bool, device=DEV).triu(lens[b] - new + 1)
        for h in range(Hkv):
            k = s["k"][where, h].reshape(-1, HD)[: lens[b]].double()
            v = s["v"][where, h].reshape(-1, HD)[: lens[b]].double()
            for j in range(h * G, (h + 1) * G):
                z = s["q"][rows, j * HD:(j + 1) * HD].double() @ k.T / math.sqrt(HD)
                z = z.masked_fill(hidden, -math.inf)
                lse[rows, j] = torch.logsumexp(z, 1) / math.log(2.0)
                o[rows, j] = torch.softmax(z, 1) @ v
    o = o.view(n, H * HD)
    return (o, lse) if case["lse"] else o
