"""Attention over the paged cache with NaN and infinities in what rows see: they
stay in the rows that see them, however the batch is cut between blocks, and
leave every other row's bits alone.

No tolerances: a row is NaN or it is not, and the others are compared bit for
bit with the call that has finite values only (each row's sums are its own)."""
import math

import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_kv_cache import HD, _cache, _q

pytestmark = pytest.mark.gpu

BATCHES = [  # new, ctx, H, Hkv, T, page, shared, causal
    ([1] * 700, [5] * 700, 4, 1, 1, 16, 0, True),                        # few rows, an item to a block
    ([1], [9000], 4, 2, 1, 64, 0, True),                                 # few rows, items cut between many blocks
    ([1], [3], 4, 1, 1, 16, 0, True),                                    # one tile
    ([6, 2, 1], [3000, 40, 0], 8, 2, 2, 16, 0, True),                    # 24 rows to a key head
    ([70], [0], 1, 1, 1, 16, 0, True),                                   # many rows, a few tiles
    ([300, 40], [1500, 20], 4, 2, 2, 64, 0, True),                       # many rows, cut
    ([40] * 200, [10] * 200, 2, 2, 1, 16, 0, False),                     # many rows, an item to a block
    ([1, 1, 1, 1], [7, 0, 130, 64], 32, 8, 8, 32, 8704, True),           # shared keys of 16 rows
    ([2, 1, 2, 1], [7, 0, 130, 64], 32, 8, 8, 32, 8704, True),           # of 24 rows
    ([1] * 64, [(i * 29) % 200 for i in range(64)], 32, 8, 8, 16, 700, True),   # of many, own rows few
    ([9 + i % 8 for i in range(30)], [(61 * i) % 300 for i in range(30)], 32, 8, 8, 16, 1900, True),  # both many
]


def _clean(new, ctx, H, Hkv, T, page, shared, causal):
    s = ref.make_batch(new, ctx, Hkv, page, shared, seed=len(new) + page)
    cache, batch = _cache(s, H, T, causal)
    q = _q(s["n"], H, 3)
    o, lse = cache.attend(q, batch, shared_len=shared, lse=True)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    return s, cache, batch, q, o.view(-1, H, HD), lse


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared,causal", BATCHES)
def test_a_query_that_is_not_finite(new, ctx, H, Hkv, T, page, shared, causal, value):
    """One element of a query.  NaN makes every score of the row NaN; an infinity
    makes each an infinity of its key's sign (the keys' column is set to +-1 so
    that both signs are among those that every chosen row sees), and the weight
    of a score of +inf is inf / inf."""
    s, cache, batch, q, _, _ = _clean(new, ctx, H, Hkv, T, page, shared, causal)
    if not math.isnan(value):
        signs = torch.ones(page, device="cuda", dtype=torch.bfloat16)
        signs[1::2] = -1
        s["k"][..., 17] = torch.where(s["k"][..., 17].isnan(), s["k"][..., 17], signs)
    o, lse = cache.attend(q, batch, shared_len=shared, lse=True)
    o = o.view(-1, H, HD)
    hit = torch.zeros(s["n"], H, dtype=torch.bool, device="cuda")
    first = 0
    for b, (rows, length) in enumerate(zip(s["new"], s["lens"])):
        for i in {0, rows // 2, rows - 1}:
            if not causal or length - rows + i >= 1:  # keys 0 and 1 are seen
                hit[first + i, (3 * b + i) % H] = b % 7 == 0 or len(new) < 9
        first += rows
    assert hit.any() and not hit.all()
    bad = q.clone().view(-1, H, HD)
    bad[..., 17][hit] = value
    got, got_lse = cache.attend(bad.view(-1, H * HD), batch, shared_len=shared, lse=True)
    got = got.view(-1, H, HD)
    assert cache.last_device_error() == 0
    assert got[hit].isnan().all()
    assert got_lse[hit].isnan().all()
    assert torch.equal(got[~hit], o[~hit]) and torch.equal(got_lse[~hit], lse[~hit])


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared,causal", BATCHES)
def test_a_key_that_is_nan(new, ctx, H, Hkv, T, page, shared, causal):
    """The last key of a sequence: the rows that see it are NaN, those before it and
    the other sequences' are not."""
    s, cache, batch, q, o, lse = _clean(new, ctx, H, Hkv, T, page, shared, causal)
    b = len(new) // 2
    last = s["lens"][b] - 1
    s["k"][s["table"][b, last // page].item(), 0, last % page, 5] = math.nan
    got, got_lse = cache.attend(q, batch, shared_len=shared, lse=True)
    got = got.view(-1, H, HD)
    hit = torch.zeros(s["n"], H, dtype=torch.bool, device="cuda")
    end = s["cu"][b + 1].item()
    hit[end - 1 if causal else s["cu"][b].item():end, :H // Hkv] = True
    assert got[hit].isnan().all() and got_lse[hit].isnan().all()
    assert torch.equal(got[~hit], o[~hit]) and torch.equal(got_lse[~hit], lse[~hit])


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared,causal", [b for b in BATCHES if b[6]])
def test_a_shared_key_that_is_nan(new, ctx, H, Hkv, T, page, shared, causal):
    s, cache, batch, q, o, lse = _clean(new, ctx, H, Hkv, T, page, shared, causal)
    s["k"][s["table"][0, 1].item(), Hkv - 1, page - 1, 100] = math.nan
    got, got_lse = cache.attend(q, batch, shared_len=shared, lse=True)
    got, G = got.view(-1, H, HD), H // Hkv
    assert got[:, H - G:].isnan().all() and got_lse[:, H - G:].isnan().all()
    assert torch.equal(got[:, :H - G], o[:, :H - G]) and torch.equal(got_lse[:, :H - G], lse[:, :H - G])


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared,causal", BATCHES)
def test_scores_that_are_all_minus_infinity(new, ctx, H, Hkv, T, page, shared, causal):
    """A row that sees keys, all with a weight of 2^-inf: 0 / 0, not the zeros of a
    row that sees none; the log2 of their sum is -inf."""
    s, cache, batch, q, _, _ = _clean(new, ctx, H, Hkv, T, page, shared, causal)
    s["k"][..., 17] = torch.where(s["k"][..., 17].isnan(), s["k"][..., 17], 1.0)
    o, lse = cache.attend(q, batch, shared_len=shared, lse=True)
    o = o.view(-1, H, HD)
    hit = torch.zeros(s["n"], H, dtype=torch.bool, device="cuda")
    hit[::5, H // 2] = True
    bad = q.clone().view(-1, H, HD)
    bad[..., 17][hit] = -math.inf
    got, got_lse = cache.attend(bad.view(-1, H * HD), batch, shared_len=shared, lse=True)
    got = got.view(-1, H, HD)
    assert cache.last_device_error() == 0
    assert got[hit].isnan().all() and (got_lse[hit] == -math.inf).all()
    assert torch.equal(got[~hit], o[~hit]) and torch.equal(got_lse[~hit], lse[~hit])


@pytest.mark.parametrize("new,shared", [([9, 1, 5, 3], 0), ([90, 1, 50, 30], 0), ([2] * 30, 1000), ([9] * 30, 1600)])
def test_rows_without_keys_beside_scores_of_minus_infinity(new, shared):
    """Rows that see no key get zeros, those that see only such scores NaN."""
    H, Hkv = 32, 8
    s = ref.make_batch(new, [20] * len(new), Hkv, 16, shared, seed=4)
    for b, n in ((0, new[0] - 1), (1, 0), (2, 1)):
        s["lens"][b] = n
    s["kv_len"].copy_(torch.tensor(s["lens"]))
    s["k"][..., 17] = torch.where(s["k"][..., 17].isnan(), s["k"][..., 17], 1.0)
    cache, batch = _cache(s, H, 8)
    q = _q(s["n"], H, 3).view(-1, H, HD)
    q[..., 17] = -math.inf
    o, lse = cache.attend(q.view(-1, H * HD), batch, shared_len=shared, lse=True)
    assert cache.last_device_error() == 0 and (lse == -math.inf).all()
    seen = torch.tensor([length - rows + i + 1 > 0 for rows, length in zip(s["new"], s["lens"]) for i in range(rows)],
                        device="cuda")
    assert (~seen).any() and o[seen].isnan().all() and (o[~seen] == 0).all()


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared,causal", [b for b in BATCHES if max(b[1]) > 50])
def test_a_score_of_minus_infinity(new, ctx, H, Hkv, T, page, shared, causal):
    """One key of many: its weight is 0, as that of a score of -2600."""
    s, cache, batch, q, _, _ = _clean(new, ctx, H, Hkv, T, page, shared, causal)
    q.view(-1, H, HD)[..., 17] = 1.0
    out = []
    for low in (-30000.0, -math.inf):
        s["k"][s["table"][0, 0].item(), :, 1, 17] = low
        out.append(cache.attend(q, batch, shared_len=shared, lse=True))
    assert torch.isfinite(out[0][0]).all()
    for a, b in zip(*out):
        assert torch.equal(a, b)
