"""What an append writes when a batch names a page, length or offset out of range:
the whole of both caches, all of it finite, against what it ought to hold."""
import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_kv_cache import HD, _cache, _modules

pytestmark = pytest.mark.gpu

BATCHES = [  # new, ctx, H, Hkv, T, page: single tokens; several heads to a warp and more tokens than warps
    ([1, 1, 1], [100, 60, 200], 4, 2, 2, 16),
    ([700, 650, 3], [40, 9, 0], 12, 4, 2, 32),
]


def _make(new, ctx, H, Hkv, T, page):
    s = ref.make_batch(new, ctx, Hkv, page, spare_rows=1, seed=71, junk=3.0)
    cache, batch = _cache(s, H, T)
    g = torch.Generator(device="cuda").manual_seed(9)
    qkv = torch.randn(s["n"], (H + 2 * Hkv) * HD, generator=g, device="cuda").to(torch.bfloat16)
    assert torch.isfinite(s["k"]).all() and torch.isfinite(s["v"]).all()
    return s, cache, batch, qkv, [t.clone() for t in (s["k"], s["v"])]


def _store(s, H, Hkv, T, page, qkv, k, v, rows):
    """The rows' keys and values into k and v, through the batch's own table."""
    _, kk, vv = ref.split_qkv(qkv, H, Hkv, T)
    pos = ref.positions(s)
    seq = torch.tensor([b for b, n in enumerate(s["new"]) for _ in range(n)], device="cuda")
    rows = torch.tensor(rows, device="cuda")
    pages = s["table"][seq[rows], pos[rows] // page].long()
    k[pages, :, pos[rows] % page] = kk[rows]
    v[pages, :, pos[rows] % page] = vv[rows]


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page", BATCHES)
def test_a_bad_page_loses_its_tokens_and_nothing_else(new, ctx, H, Hkv, T, page):
    abi = _modules()[0]
    s, cache, batch, qkv, (k0, v0) = _make(new, ctx, H, Hkv, T, page)
    keep = s["table"].clone()
    at = (s["lens"][1] - 1) // page  # the second sequence's last page
    first = at * page
    starts = [sum(new[:b]) for b in range(len(new))]
    gone = {starts[1] + i for i in range(new[1]) if s["lens"][1] - new[1] + i >= first}
    good = [r for r in range(sum(new)) if r not in gone]
    assert gone
    for bad in (-1, s["n_pages"], s["n_pages"] + 5, 2 ** 31 - 1, -2 ** 31):
        s["k"].copy_(k0)
        s["v"].copy_(v0)
        k, v = k0.clone(), v0.clone()
        _store(s, H, Hkv, T, page, qkv, k, v, good)
        s["table"][1, at] = bad
        q = cache.append(qkv, batch, q=torch.full((s["n"], H * HD), 5.0, dtype=torch.bfloat16, device="cuda"))
        assert cache.last_device_error() == abi.TP_ERR_BATCH
        assert torch.equal(s["k"], k) and torch.equal(s["v"], v)
        x = ref.split_qkv(qkv, H, Hkv, T)[0].reshape(s["n"], -1)
        assert torch.equal(q[:-1], x[:-1]) and (q[-1] == 5.0).all()
        s["table"].copy_(keep)
    cache.append(qkv, batch)
    assert cache.last_device_error() == abi.TP_OK


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page", BATCHES)
def test_a_bad_length_or_offset_stays_in_its_sequence(new, ctx, H, Hkv, T, page):
    abi = _modules()[0]
    s, cache, batch, qkv, (k0, v0) = _make(new, ctx, H, Hkv, T, page)
    total, cap = sum(new), s["table"].shape[1] * page
    s["table"].clamp_(min=0)  # (unused entries too name pages, here)
    cases = [("kv_len", 1, cap + new[1], {1}, True), ("kv_len", 1, 2 ** 31 - 1, {1}, True),
             ("kv_len", 1, 0, {1}, True), ("kv_len", 1, -2 ** 31, {1}, True),
             ("cu", 3, 10 ** 6, {2}, False), ("cu", 0, -3, {0}, False), ("cu", 1, -3, {0, 1}, False)]
    for name, i, bad, hit, nothing in cases:
        s["k"].copy_(k0)
        s["v"].copy_(v0)
        k, v = k0.clone(), v0.clone()
        starts = [sum(new[:b]) for b in range(4)]
        _store(s, H, Hkv, T, page, qkv, k, v, [r for b in range(3) if b not in hit for r in range(starts[b], starts[b + 1])])
        was = s[name][i].item()
        s[name][i] = bad
        cache.append(qkv, batch)
        if name == "kv_len" or bad > 0:  # (rows in front of the first offset are nobody's)
            assert cache.last_device_error() == abi.TP_ERR_BATCH, (name, bad)
        s[name][i] = was
        free = torch.ones(s["n_pages"], dtype=torch.bool, device="cuda")
        if not nothing:  # what the sequences at fault are left with is unspecified, within their pages
            free[s["table"][list(hit)].flatten().long()] = False
        assert torch.equal(s["k"][free], k[free]) and torch.equal(s["v"][free], v[free]), (name, bad)
    cache.append(qkv, batch)
    assert cache.last_device_error() == abi.TP_OK and total == s["n"] - 1


def test_a_negative_offset_is_reported():
    """The tokens of its sequence are not stored: the call says so."""
    abi = _modules()[0]
    s, cache, batch, qkv, _ = _make(*BATCHES[0])
    for i, bad in ((0, -1), (0, -2 ** 31), (1, -3)):
        was = s["cu"][i].item()
        s["cu"][i] = bad
        cache.append(qkv, batch)
        assert cache.last_device_error() == abi.TP_ERR_BATCH, (i, bad)
        s["cu"][i] = was
    s["cu"][0] = 1  # rows in front of the first offset are nobody's: no fault
    cache.append(qkv, batch)
    assert cache.last_device_error() == abi.TP_OK
