"""Plain 64-bit forms of the serving operators over the paged cache, one
sequence and one head at a time, and random batches for their tests."""
import math

import torch

HD = 128


def make_batch(new, ctx, Hkv, page, shared=0, spare_rows=0, seed=0, device="cuda", junk=float("nan"), copies=False):
    """A cache in random page order whose slots behind every sequence's last key,
    and whose unused pages, hold `junk`; the first `shared` keys of all sequences
    lie in the same pages where those are full (the page that `shared` ends in is
    a copy of the first sequence's in every other one)."""
    g = torch.Generator().manual_seed(seed)
    B = len(new)
    kv_len = [shared + a + b for a, b in zip(new, ctx)]
    need = [-(-n // page) for n in kv_len]
    width = max(max(need), 1)
    full = 0 if copies else shared // page
    n_pages = full + sum(max(n - full, 0) for n in need) + 2
    order = torch.randperm(n_pages, generator=g).tolist()
    common = [order.pop() for _ in range(full)]
    table = torch.full((B, width), -7, dtype=torch.int32)
    for b in range(B):
        row = (common + [order.pop() for _ in range(max(need[b] - full, 0))])[:need[b]]
        table[b, :need[b]] = torch.tensor(row, dtype=torch.int32)
    dg = torch.Generator(device=device).manual_seed(seed)
    kv = []
    for _ in range(2):
        t = torch.randn(n_pages, Hkv, page, HD, generator=dg, device=device).to(torch.bfloat16)
        live = torch.zeros(n_pages, page, dtype=torch.bool, device=device)
        for b in range(B):
            for i in range(need[b]):
                live[table[b, i], : min(page, kv_len[b] - i * page)] = True
        for i in range(full, -(-shared // page)):  # own copies of the shared keys past the common pages
            for b in range(1, B):
                t[table[b, i], :, : min(page, shared - i * page)] = t[table[0, i], :, : min(page, shared - i * page)]
        t.masked_fill_(~live[:, None, :, None], junk)
        kv.append(t)
    cu = [0]
    for q in new:
        cu.append(cu[-1] + q)
    i32 = dict(dtype=torch.int32, device=device)
    return dict(k=kv[0], v=kv[1], cu=torch.tensor(cu, **i32), kv_len=torch.tensor(kv_len, **i32),
                table=table.to(device), n=cu[-1] + spare_rows, n_pages=n_pages, new=list(new), lens=kv_len,
                max_new=max(max(new), 1))


def attend(s, q, H, causal=True):
    """(o, lse, a, rough): o and the log2-sum-exp in 64 bits, a = sum_j p_j |v_j|,
    rough = max_j sum_c |q_c k_jc| / sqrt(128) (what a score's rounding goes by)."""
    Hkv, page = s["k"].shape[1], s["k"].shape[2]
    G, n = H // Hkv, q.shape[0]
    o = torch.zeros(n, H, HD, dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    rough = torch.zeros(n, H, dtype=torch.float64, device=q.device)
    first = 0
    for b, (new, length) in enumerate(zip(s["new"], s["lens"])):
        pages = s["table"][b, : -(-length // page)].long()
        rows = slice(first, first + new)
        first += new
        if new == 0 or length == 0:
            continue
        sees = torch.arange(length, device=q.device)[None, :] <= length - new + torch.arange(new, device=q.device)[:, None]
        if not causal:
            sees = torch.ones_like(sees)
        some = sees.any(1)
        for h in range(H):
            k = s["k"][pages, h // G].reshape(-1, HD)[:length].double()
            v = s["v"][pages, h // G].reshape(-1, HD)[:length].double()
            x = q[rows, h * HD:(h + 1) * HD].double()
            z = (x @ k.T / math.sqrt(HD)).masked_fill(~sees, -math.inf)
            p = torch.where(some[:, None], torch.softmax(z, 1), 0.0)
            o[rows, h], a[rows, h] = p @ v, p @ v.abs()
            lse[rows, h] = torch.logsumexp(z, 1) / math.log(2.0)
            rough[rows, h] = (x.abs() @ k.abs().T / math.sqrt(HD)).amax(1)
    return o.view(n, H * HD), lse, a.view(n, H * HD), rough


def rotate(x, pos, inv_freq, interleaved, scale=1.0):
    """x [n, heads, 128] in 64 bits -> (rotated, size): size bounds what each
    element is summed from."""
    if inv_freq is None:
        return x, x.abs()
    r = 2 * inv_freq.numel()
    angle = pos.double()[:, None] * inv_freq.double()[None]
    c, s = angle.cos()[:, None] * scale, angle.sin()[:, None] * scale
    out, size = x.clone(), x.abs()
    lo, hi = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    out[..., lo], out[..., hi] = x[..., lo] * c - x[..., hi] * s, x[..., hi] * c + x[..., lo] * s
    size[..., lo] = size[..., hi] = (x[..., lo].abs() + x[..., hi].abs()) * abs(scale)
    return out, size


def split_qkv(qkv, H, Hkv, T):
    """Packed projections -> q [n, H, 128], k and v [n, Hkv, 128]."""
    n = qkv.shape[0]
    x = qkv.view(n, T, (H + 2 * Hkv) // T, HD)
    return (x[:, :, :H // T].reshape(n, H, HD), x[:, :, H // T:(H + Hkv) // T].reshape(n, Hkv, HD),
            x[:, :, (H + Hkv) // T:].reshape(n, Hkv, HD))


def positions(s):
    return torch.tensor([length - new + i for new, length in zip(s["new"], s["lens"]) for i in range(new)],
                        device=s["cu"].device)
