"""Serving operators of the attention sublayer against plain 64-bit forms:
appending to the paged cache with the rotation by position, and attention over
the cache with and without a shared prefix.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value.
 * Append, unrotated columns and values: equal.  Rotated ones: 2^-8 |ref| for
   the output's rounding, plus the 32-bit error of x cos - y sin: sine and
   cosine are within 2^-22 (an angle reduced to half a turn and rounded to 24
   bits is off by 2 pi 2^-26 < 2^-23, the functions by less than 2^-23), two
   products and a sum add 2^-23, so 2^-20 (|x| + |y|) covers it four times.
 * Attention: the rounding of o (2^-8 |o|), the rounding of each probability
   before the second product (2^-8 sum p |v|), and the scores' error d: 128
   products summed in 32 bits are off by at most 2^7 2^-24 sum |q k|, which
   changes p by a factor within exp(2 d); likewise the sum over L keys in 32
   bits, L 2^-24, both relative to sum p |v|.  (1 + 2^-8) covers products of
   these.  In root mean square the roundings of single probabilities average:
   the relative error stays below 2^-8.
 * lse: d log2 e from the scores and 2^-22 (|lse| + L 2^-2) from 32-bit sums.
"""
import math

import pytest
import torch

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

HD = 128
U = 2.0 ** -8


def _modules():
    from megatron_tensor_transformer_w1_gb300 import tpffn as abi
    from megatron_tensor_transformer_w1_gb300.attention import TensorParallelAttention
    from megatron_tensor_transformer_w1_gb300.kv_cache import KVBatch, PagedKVCache
    return abi, TensorParallelAttention, KVBatch, PagedKVCache


def _cache(s, H, T, causal=True, **kw):
    _, Attention, _, Cache = _modules()
    Hkv, page = s["k"].shape[1], s["k"].shape[2]
    attn = Attention(256, H, Hkv, HD, T, causal=causal)
    cache = Cache(attn, s["n_pages"], page, k=s["k"], v=s["v"], **kw)
    return cache, cache.batch(s["cu"], s["kv_len"], s["table"], n_tokens=s["n"], max_new=s["max_new"])


def _q(n, H, seed, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    return (torch.randn(n, H * HD, generator=g, device="cuda") * scale).to(torch.bfloat16)


def check_attend(s, q, H, o, lse, causal=True):
    rows = s["cu"][-1].item()
    want, want_lse, a, rough = ref.attend(s, q[:rows], H, causal)
    longest = max(s["lens"])
    d = 2.0 ** -17 * rough
    wide = lambda t: t.repeat_interleave(HD, 1)
    tol = (1 + U) * (U * want.abs() + a * (U + 2 * wide(d) + longest * 2.0 ** -24)) + 1e-30
    err = (o[:rows].double() - want).abs()
    assert torch.isfinite(o[:rows]).all()
    assert (err <= tol).all(), f"largest error over its bound: {(err / tol).max().item():.2f}"
    rms = want.square().mean().sqrt()
    assert err.square().mean().sqrt() <= U * rms + 1e-30, (err.square().mean().sqrt() / rms).item()
    if lse is not None:
        none = want_lse == -math.inf
        assert torch.equal(none, lse[:rows] == -math.inf)
        lim = d * math.log2(math.e) + 2.0 ** -22 * (want_lse.abs() + longest / 4)
        assert ((lse[:rows].double() - want_lse).abs()[~none] <= lim[~none]).all()
        assert (o[:rows].view(rows, H, HD)[none] == 0).all()


ATTEND = [  # new, ctx, H, Hkv, T, page, shared, causal
    ([1], [0], 4, 4, 2, 16, 0, True),                                  # one key
    ([1], [511], 8, 2, 2, 16, 0, True),
    ([1, 1, 1], [63, 64, 65], 4, 1, 1, 64, 0, True),                   # around a tile's end
    ([1] * 5, [0, 1, 7, 8, 1000], 16, 2, 2, 8, 0, True),               # around a page's end
    ([1, 0, 3, 0, 2], [30, 50, 129, 0, 0], 4, 2, 2, 32, 0, True),      # sequences without new tokens
    ([2, 5, 1], [100, 0, 333], 8, 8, 4, 128, 0, True),
    ([4, 4], [700, 3], 32, 2, 2, 256, 0, True),                        # 64 rows to a key head
    ([3, 1], [77, 2050], 25, 5, 5, 16, 0, True),                       # groups of five
    ([2, 3], [200, 90], 10, 1, 1, 1024, 0, True),                      # groups of ten, long pages
    ([2, 3], [200, 90], 4, 2, 1, 16, 0, False),
    ([1] * 3, [5, 40, 1], 8, 2, 2, 16, 256, True),                     # a shared prefix of whole pages
    ([1, 2, 1, 0], [5, 0, 130, 9], 4, 2, 2, 16, 100, True),            # that ends inside a page and a tile
    ([3, 1], [0, 0], 8, 4, 4, 64, 1030, True),                         # no own context behind it
    ([2, 1], [300, 10], 8, 2, 2, 32, 70, False),
    ([1] * 40, [i * 3 for i in range(40)], 2, 2, 2, 8, 512, True),     # 40 rows against the prefix
    ([1] * 131, [(i * 37) % 300 for i in range(131)], 2, 1, 1, 16, 0, True),  # more sequences than threads
]


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared,causal", ATTEND)
def test_attend(new, ctx, H, Hkv, T, page, shared, causal):
    s = ref.make_batch(new, ctx, Hkv, page, shared, spare_rows=2, seed=len(new) + page)
    cache, batch = _cache(s, H, T, causal)
    q = _q(s["n"], H, page)
    out = torch.full((s["n"], H * HD), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = cache.attend(q, batch, shared_len=shared, lse=True, out=out)
    assert cache.last_device_error() == 0
    check_attend(s, q, H, o, lse, causal)
    assert (o[-2:] == 7.0).all()  # rows behind the last sequence stay as they were
    again, _ = cache.attend(q, batch, shared_len=shared, lse=True)
    rows = s["cu"][-1].item()
    assert torch.equal(o[:rows], again[:rows])
    if shared:  # the same keys, each sequence on its own
        check_attend(s, q, H, cache.attend(q, batch), None, causal)


MANY = [  # more than 64 rows to a key head: the tensor-memory kernel
    ([65], [0], 1, 1, 1, 16, 0, True),                                 # just more; only own keys
    ([17], [100], 4, 1, 1, 8, 0, True),
    ([128], [128], 2, 2, 1, 64, 0, True),                              # whole tiles
    ([129, 1, 257], [0, 300, 127], 4, 2, 2, 16, 0, True),              # around the tiles' ends, a single token among them
    ([300], [1000], 8, 2, 2, 128, 0, True),
    ([40, 0, 3, 90], [7, 500, 0, 129], 5, 1, 1, 32, 0, True),          # groups of five across row tiles
    ([200, 13], [50, 900], 4, 4, 4, 1024, 0, True),
    ([100, 30], [77, 260], 8, 2, 2, 256, 0, False),
    ([700, 100], [3000, 0], 8, 2, 2, 64, 0, True),                     # items cut between blocks
    ([1] * 40, [i * 3 for i in range(40)], 4, 2, 2, 8, 512, True),     # a shared prefix for 80 rows
    ([1] * 70, [(i * 29) % 200 for i in range(70)], 16, 2, 2, 16, 1000, True),  # 560 rows, ends inside a page
    ([2] * 33, [5] * 33, 8, 8, 4, 128, 129, False),
    ([90, 1, 1, 1, 1, 1, 1, 1, 1], [3] * 9, 4, 2, 2, 16, 300, True),   # a prompt among single tokens
    ([100, 80], [30, 40], 8, 2, 2, 32, 640, True),                     # prompts behind a prefix
    ([(37 * i) % 300 for i in range(24)], [(431 * i) % 2500 for i in range(24)], 16, 4, 4, 16, 0, True),  # many cut items
    ([1 + (13 * i) % 64 for i in range(150)], [(7 * i) % 40 for i in range(150)], 4, 2, 2, 8, 0, False),  # many short ones
]


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared,causal", MANY)
def test_attend_many_rows(new, ctx, H, Hkv, T, page, shared, causal):
    test_attend(new, ctx, H, Hkv, T, page, shared, causal)


SHARED = [  # shared keys worth taking together: (sequences - 1) x keys x key heads x 512 bytes from 96 MiB on
    ([1] * 7, [5, 40, 1, 0, 300, 64, 63], 32, 16, 4, 16, 2048, True),         # 14 rows: few
    ([1, 2, 1, 0, 1, 3, 1, 1], [5, 0, 130, 9, 0, 1, 2, 3], 32, 16, 4, 64, 1800, True),   # 20 rows, ends inside a page
    ([2] * 8, [30] * 8, 16, 8, 2, 16, 3600, False),                           # 32 rows, all keys seen
    ([3] * 11, [5 * i for i in range(11)], 32, 8, 8, 128, 2500, True),        # 132 rows: many
    ([1] * 80, [(i * 29) % 200 for i in range(80)], 8, 2, 2, 16, 1301, True),  # 320 rows, two row tiles
    ([1] * 70, [3] * 70, 10, 2, 1, 1024, 1500, False),                        # groups of five
    ([200] + [1] * 59, [3] * 60, 2, 2, 2, 64, 1700, True),                    # a prompt among single tokens
    ([9, 1] * 10, [0] * 20, 40, 5, 5, 8, 2100, True),                         # no own context; own rows: many
    ([1] * 9, [0] * 9, 32, 8, 8, 64, 4000, True),                             # fewer own tiles than blocks
    ([1] * 20, [(701 * i) % 7000 for i in range(20)], 32, 8, 8, 32, 1300, True),  # long own keys, ragged
    ([2] * 33, [(97 * i) % 900 for i in range(33)], 64, 16, 4, 16, 500, False),   # short shared keys
    ([9 + i % 8 for i in range(30)], [(61 * i) % 700 for i in range(30)], 32, 8, 8, 16, 1000, True),  # own rows: many, ragged
]


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared,causal", SHARED)
def test_attend_shared_keys(new, ctx, H, Hkv, T, page, shared, causal):
    assert (len(new) - 1) * shared * Hkv * 512 >= 96 << 20
    test_attend(new, ctx, H, Hkv, T, page, shared, causal)


@pytest.mark.parametrize("new", [1, 5])
def test_attend_shared_keys_longer_than_sequences(new):
    """Behind shared keys that some sequences do not reach the end of: cut rows, no
    keys at all, more new tokens than keys."""
    B, Hkv, H = 60, 2, 8
    s = ref.make_batch([new] * B, [3] * B, Hkv, 16, shared=1700, seed=6)
    for b, n in ((0, 1650), (1, 0), (2, 1), (3, 3), (7, 1699), (8, 1701), (59, 64)):
        s["lens"][b] = n
    s["kv_len"].copy_(torch.tensor(s["lens"]))
    cache, batch = _cache(s, H, 2)
    q = _q(s["n"], H, 2)
    o, lse = cache.attend(q, batch, shared_len=1700, lse=True)
    assert cache.last_device_error() == 0
    check_attend(s, q, H, o, lse)


def test_attend_shared_keys_of_idle_sequences():
    """The first sequence has no keys and no table: the shared pages are found all the same."""
    B, Hkv, H = 60, 2, 8
    s = ref.make_batch([0] + [1] * (B - 1), [0] * B, Hkv, 16, shared=1700, seed=16)
    s["lens"][0] = 0
    s["kv_len"][0] = 0
    s["table"][0] = -5
    cache, batch = _cache(s, H, 2)
    q = _q(s["n"], H, 2)
    o, lse = cache.attend(q, batch, shared_len=1700, lse=True)
    assert cache.last_device_error() == 0
    check_attend(s, q, H, o, lse)
    # a bad shared page is reported
    s["table"][:, 3] = s["n_pages"]
    o = cache.attend(q, batch, shared_len=1700)
    assert cache.last_device_error() == _modules()[0].TP_ERR_BATCH and torch.isfinite(o).all()


def test_attend_shared_keys_bad_offsets():
    """Offsets that descend, or begin behind the first row, leave rows that the shared
    keys' work does not cover: nothing is read for them, and the call reports it."""
    abi = _modules()[0]
    B, Hkv, H = 5, 8, 64
    s = ref.make_batch([40] * B, [3] * B, Hkv, 64, shared=6400, seed=26)
    assert (B - 1) * 6400 * Hkv * 512 >= 96 << 20
    cache, batch = _cache(s, H, 8)
    q = _q(s["n"], H, 12)
    good = cache.attend(q, batch, shared_len=6400)
    assert cache.last_device_error() == abi.TP_OK
    check_attend(s, q, H, good, None)
    keep = s["cu"].clone()
    for bad in ([0, 40, 80, 120, 160, 3], [0, 40, 80, 120, 160, 0], [0, 200, 3, 120, 2, 1], [0, -7, 80, 120, 160, 200]):
        s["cu"].copy_(torch.tensor(bad))
        assert torch.isfinite(cache.attend(q, batch, shared_len=6400, out=torch.zeros_like(good))).all()
        assert cache.last_device_error() == abi.TP_ERR_BATCH
    s["cu"].copy_(keep)
    s["cu"][0] = 33  # the first sequence's last seven rows; those before are nobody's
    o = torch.full_like(good, 7.0)
    cache.attend(q, batch, shared_len=6400, out=o)
    assert (o[:33] == 7).all()
    check_attend(dict(s, new=[7] + [40] * 4, cu=s["cu"] - 33), q[33:], H, o[33:], None)
    s["cu"].copy_(keep)
    assert torch.equal(cache.attend(q, batch, shared_len=6400), good)
    assert cache.last_device_error() == abi.TP_OK


def test_attend_many_rows_that_see_nothing():
    """A prompt cut off by kv_len: its first rows see no key, whole row tiles among them."""
    s = ref.make_batch([600, 70, 80], [0, 0, 10], 1, 16, seed=15)
    s["lens"] = [40, 0, 90]
    s["kv_len"].copy_(torch.tensor(s["lens"]))
    cache, batch = _cache(s, 2, 1)
    q = _q(s["n"], 2, 7)
    o, lse = cache.attend(q, batch, lse=True)
    assert cache.last_device_error() == 0
    check_attend(s, q, 2, o, lse)


def test_attend_many_rows_sharp_scores():
    s = ref.make_batch([150, 70], [900, 2000], 2, 16, seed=12)
    s["k"].mul_(torch.linspace(0.1, 6, s["k"].shape[0], device="cuda").to(torch.bfloat16)[:, None, None, None])
    cache, batch = _cache(s, 4, 2)
    q = _q(s["n"], 4, 5, scale=6.0)
    check_attend(s, q, 4, *cache.attend(q, batch, lse=True))


def test_many_rows_bad_batches():
    abi = _modules()[0]
    s = ref.make_batch([80, 70, 90], [100, 60, 200], 2, 16, seed=22)
    cache, batch = _cache(s, 4, 2)
    q = _q(s["n"], 4, 6)
    good = cache.attend(q, batch)
    assert cache.last_device_error() == abi.TP_OK
    keep = s["table"].clone()
    for bad in (-1, s["n_pages"], 2 ** 31 - 1, -2 ** 31):
        s["table"][1, 2] = bad
        o = cache.attend(q, batch)
        assert cache.last_device_error() == abi.TP_ERR_BATCH
        assert torch.equal(o[:80], good[:80]) and torch.equal(o[150:], good[150:]) and torch.isfinite(o).all()
        s["table"].copy_(keep)
    for name, at, bad in (("kv_len", 1, -5), ("cu", 3, 10 ** 6), ("cu", 1, -3)):
        was = s[name][at].item()
        s[name][at] = bad
        cache.attend(q, batch)
        assert cache.last_device_error() == abi.TP_ERR_BATCH, name
        s[name][at] = was
    assert torch.equal(cache.attend(q, batch), good)
    assert cache.last_device_error() == abi.TP_OK


def test_many_rows_bounded_wait_expires_and_context_survives():
    """A copy that is never issued: its waits run out, the call reports it, and the
    next call is as ever."""
    abi = _modules()[0]
    s = ref.make_batch([80, 70, 200], [100, 60, 2000], 2, 16, seed=23)
    cache, batch = _cache(s, 4, 2)
    q = _q(s["n"], 4, 8)
    good = cache.attend(q, batch)
    with pytest.raises(Exception, match="TP_ERR_TIMEOUT"):
        cache.attend(q, batch, flags=abi.TP_FLAG_DEBUG_SKIP_LOAD | abi.TP_FLAG_SYNC)
    assert torch.equal(cache.attend(q, batch, flags=abi.TP_FLAG_SYNC), good)


def test_calls_are_refused():
    """Tensors of the wrong type, shape, layout or place."""
    abi, Attention, KVBatch, Cache = _modules()
    s = ref.make_batch([1, 2], [10, 20], 2, 16, seed=24, spare_rows=1)
    cache, batch = _cache(s, 4, 2)
    q, qkv = _q(s["n"], 4, 1), torch.zeros(s["n"], 8 * HD, dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros(s["n"], 1024, dtype=torch.bfloat16, device="cuda")
    for bad in (q.float(), q[1:], q.cpu(), q.t().contiguous().t(), wide[:, :512]):
        with pytest.raises(ValueError):
            cache.attend(bad, batch)
        with pytest.raises(ValueError):
            cache.attend(q, batch, out=bad)
        with pytest.raises(ValueError):
            cache.append(qkv, batch, q=bad)
    for bad in (qkv.float(), qkv[:-1], qkv.cpu(), wide[:, ::1][:, 1:]):
        with pytest.raises(ValueError):
            cache.append(bad, batch)
    with pytest.raises(ValueError):
        cache.attend(q, KVBatch(s["cu"].cpu(), s["kv_len"].cpu(), s["table"].cpu(), s["n"], 2))
    for shared in (-1, s["table"].shape[1] * 16 + 1):
        with pytest.raises(abi.TPFFNError):
            cache.attend(q, batch, shared_len=shared)
    attn = cache.attn
    for kw in (dict(page_size=4), dict(page_size=24), dict(page_size=2048), dict(n_pages=0), dict(k=s["k"].float()),
               dict(k=s["k"][:-1]), dict(v=s["v"].cpu()), dict(inv_freq=torch.ones(12, device="cuda")),
               dict(inv_freq=torch.ones(72, device="cuda")), dict(inv_freq=torch.ones(64, device="cuda").double())):
        args = dict(n_pages=s["n_pages"], page_size=16, k=s["k"], v=s["v"])
        args.update(kw)
        with pytest.raises(ValueError):
            Cache(attn, **args)
    other = Attention(256, 4, 2, HD, 2)
    with pytest.raises(ValueError):
        other.decode(wide[:, :256].contiguous(), cache, batch, None, None)


def test_empty_calls():
    """No new tokens, no sequences: no work, and the cache as it was."""
    abi = _modules()[0]
    s = ref.make_batch([1, 2], [10, 20], 2, 16, seed=25)
    cache, _ = _cache(s, 4, 2)
    k0 = s["k"].clone()
    none = torch.zeros(0, 8 * HD, dtype=torch.bfloat16, device="cuda")
    batch = cache.batch(torch.zeros(3, dtype=torch.int32, device="cuda"), s["kv_len"], s["table"], 0, 0)
    q = cache.append(none, batch)
    o, lse = cache.attend(q, batch, lse=True)
    assert q.shape == o.shape == (0, 4 * HD) and lse.shape == (0, 4) and cache.last_device_error() == abi.TP_OK
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = cache.batch(torch.zeros(1, **i32), torch.zeros(0, **i32), torch.zeros(0, 3, **i32), 5, 1)
    x = torch.full((5, 4 * HD), 3.0, dtype=torch.bfloat16, device="cuda")
    cache.append(torch.zeros(5, 8 * HD, dtype=torch.bfloat16, device="cuda"), batch, q=x)
    cache.attend(_q(5, 4, 1), batch, out=x)
    assert (x == 3).all() and cache.last_device_error() == abi.TP_OK
    assert torch.equal(k0.nan_to_num(), s["k"].nan_to_num())


def test_rows_behind_the_last_sequence_in_a_replayed_graph():
    """A graph for 8 sequences of at most 4 new tokens each, replayed with batches of fewer."""
    s = ref.make_batch([4] * 8, [100] * 8, 2, 16, seed=26)
    cache, batch = _cache(s, 8, 2)
    q = _q(s["n"], 8, 9)
    out = torch.zeros(s["n"], 8 * HD, dtype=torch.bfloat16, device="cuda")
    cache.attend(q, batch, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(q, batch, out=out)
    for new in ([4] * 8, [1] * 8, [0, 3, 0, 0, 1, 2, 0, 0], [0] * 8, [4, 1, 4, 1, 4, 1, 4, 1]):
        s["new"] = new
        s["lens"] = [50 + 7 * b + n for b, n in enumerate(new)]
        s["cu"].copy_(torch.tensor([0] + new).cumsum(0))
        s["kv_len"].copy_(torch.tensor(s["lens"]))
        out.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        rows = sum(new)
        assert (out[rows:] == 5).all()
        if rows:
            check_attend(s, q, 8, out, None)


def test_offsets_beyond_32_bits():
    """Pages far behind 2^31 elements of the cache."""
    Hkv, page, H = 16, 64, 16
    n_pages = 2 ** 31 // (Hkv * page * HD) + 40  # 4.3 GB each of keys and values
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[n_pages - 1, 3, n_pages - 7]], **i32)
    k, v = (torch.empty(n_pages, Hkv, page, HD, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(8)
    for new in (1, 70):
        s = dict(k=k, v=v, cu=torch.tensor([0, new], **i32), kv_len=torch.tensor([150], **i32), table=table, n=new,
                 n_pages=n_pages, new=[new], lens=[150], max_new=new)
        for p in table[0].tolist():
            k[p].normal_(generator=g)
            v[p].normal_(generator=g)
        cache, batch = _cache(s, H, 4)
        qkv = torch.randn(new, 48 * HD, generator=g, device="cuda").to(torch.bfloat16)
        q = cache.append(qkv, batch)
        _, kk, vv = ref.split_qkv(qkv, H, Hkv, 4)
        assert torch.equal(k[n_pages - 7, :, 149 - 128], kk[-1]) and torch.equal(v[n_pages - 7, :, 149 - 128], vv[-1])
        check_attend(s, q, H, *cache.attend(q, batch, lse=True))
        assert cache.last_device_error() == 0


def test_attend_rows_that_see_nothing():
    """More new tokens than keys (the first rows see none), and no keys at all."""
    s = ref.make_batch([3, 2, 4], [40, 0, 0], 2, 16, seed=5)
    s["lens"] = [43, 0, 2]
    s["kv_len"].copy_(torch.tensor(s["lens"]))
    cache, batch = _cache(s, 8, 2)
    q = _q(s["n"], 8, 1)
    o, lse = cache.attend(q, batch, lse=True)
    assert cache.last_device_error() == 0
    check_attend(s, q, 8, o, lse)
    # behind a prefix that is longer than some sequences
    s = ref.make_batch([2, 1, 1], [9, 5, 60], 2, 16, shared=96, seed=6)
    s["lens"] = [107, 40, 0]
    s["kv_len"].copy_(torch.tensor(s["lens"]))
    cache, batch = _cache(s, 8, 2)
    q = _q(s["n"], 8, 2)
    o, lse = cache.attend(q, batch, shared_len=96, lse=True)
    check_attend(s, q, 8, o, lse)


def test_attend_long_sequence_among_short_ones():
    """One sequence takes most of the blocks: its rows are joined from many parts."""
    s = ref.make_batch([1, 1, 1, 1], [40000, 3, 17, 0], 1, 64, seed=9)
    cache, batch = _cache(s, 4, 1)
    q = _q(s["n"], 4, 3)
    check_attend(s, q, 4, *cache.attend(q, batch, lse=True))
    s = ref.make_batch([1] * 200, [20000] + [2] * 199, 1, 64, seed=10)
    cache, batch = _cache(s, 8, 1)
    q = _q(s["n"], 8, 4)
    check_attend(s, q, 8, *cache.attend(q, batch, lse=True))


def test_attend_sharp_scores():
    """Scores in the hundreds, rising along the keys: the running maximum moves often."""
    s = ref.make_batch([1, 2], [900, 2000], 2, 16, seed=11)
    s["k"].mul_(torch.linspace(0.1, 6, s["k"].shape[0], device="cuda").to(torch.bfloat16)[:, None, None, None])
    cache, batch = _cache(s, 4, 2)
    q = _q(s["n"], 4, 5, scale=6.0)
    check_attend(s, q, 4, *cache.attend(q, batch, lse=True))


APPEND = [  # new, ctx, H, Hkv, T, page, rotary, interleaved, scale
    ([1], [0], 4, 4, 4, 16, 128, False, 1.0),
    ([1], [1000], 32, 8, 8, 64, 128, False, 1.0),
    ([1, 0, 7, 2], [5, 9, 15, 16], 8, 2, 2, 8, 64, True, 1.0),
    ([33, 1], [0, 70000], 4, 1, 1, 32, 96, False, 1.25),
    ([5, 3], [100000, 2], 10, 2, 1, 16, 16, True, 0.5),
    ([9, 40], [3, 0], 25, 5, 5, 128, 128, True, 1.0),
    ([2, 2], [3, 6], 4, 2, 2, 1024, 0, False, 1.0),
    ([1] * 70, list(range(70)), 2, 2, 1, 8, 32, False, 1.0),
    ([700, 1300], [12, 1], 4, 2, 2, 64, 128, False, 1.0),              # more rows than blocks
]


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,rotary,interleaved,scale", APPEND)
def test_append(new, ctx, H, Hkv, T, page, rotary, interleaved, scale):
    s = ref.make_batch(new, ctx, Hkv, page, spare_rows=1, seed=3, junk=3.0)
    freq = 10000.0 ** (-torch.arange(rotary // 2, device="cuda") * 2 / max(rotary, 1)) if rotary else None
    cache, batch = _cache(s, H, T, inv_freq=freq, interleaved=interleaved, rotary_scale=scale)
    g = torch.Generator(device="cuda").manual_seed(17)
    qkv = torch.randn(s["n"], (H + 2 * Hkv) * HD, generator=g, device="cuda").to(torch.bfloat16)
    k0, v0 = s["k"].clone(), s["v"].clone()
    q = cache.append(qkv, batch, q=torch.full((s["n"], H * HD), 5.0, dtype=torch.bfloat16, device="cuda"))
    assert cache.last_device_error() == 0
    assert (q[-1] == 5.0).all()
    rows = s["cu"][-1].item()
    pos = ref.positions(s)
    x, k, v = (t.double() for t in ref.split_qkv(qkv[:rows], H, Hkv, T))
    for got, inp in ((q[:rows].view(rows, H, HD), x), (None, k)):
        want, size = ref.rotate(inp, pos, freq, interleaved, scale)
        if got is None:  # where the keys were stored
            seq = torch.bucketize(torch.arange(rows, device="cuda"), s["cu"][1:].long(), right=True)
            pages = s["table"][seq, pos // page].long()
            got = s["k"][pages, :, pos % page]
            assert torch.equal(s["v"][pages, :, pos % page].double(), v)
            k0[pages, :, pos % page] = got
            v0[pages, :, pos % page] = s["v"][pages, :, pos % page]
        assert torch.equal(got[..., rotary:].double(), want[..., rotary:])
        tol = (1 + U) * (U * want.abs() + 2.0 ** -20 * size)
        assert ((got.double() - want).abs() <= tol).all()
    assert torch.equal(k0, s["k"]) and torch.equal(v0, s["v"])  # nothing else was written


def test_append_tokens_without_a_place():
    """More new tokens than kv_len: those at negative positions are not stored, their q is zero."""
    s = ref.make_batch([4], [6], 2, 16, seed=1, junk=0.0)
    s["kv_len"].fill_(2)
    cache, batch = _cache(s, 4, 1)
    qkv = torch.ones(4, 8 * HD, dtype=torch.bfloat16, device="cuda")
    k0 = s["k"].clone()
    q = cache.append(qkv, batch)
    assert (q[:2] == 0).all() and (q[2:] == 1).all()
    page = s["table"][0, 0].item()
    k0[page, :, :2] = 1
    assert torch.equal(k0, s["k"])
    assert cache.last_device_error() == _modules()[0].TP_ERR_BATCH


def test_bad_batches_are_reported_and_touch_nothing_else():
    """Pages outside the cache and lengths outside the table: reported, the other
    sequences' results as ever."""
    abi = _modules()[0]
    s = ref.make_batch([1, 1, 1], [100, 60, 200], 2, 16, seed=21)
    cache, batch = _cache(s, 4, 2)
    q = _q(s["n"], 4, 6)
    good = cache.attend(q, batch)
    assert cache.last_device_error() == abi.TP_OK
    keep = s["table"].clone()
    for bad in (-1, s["n_pages"], 2 ** 31 - 1, -2 ** 31):
        s["table"][1, 2] = bad
        o = cache.attend(q, batch)
        assert cache.last_device_error() == abi.TP_ERR_BATCH
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2]) and torch.isfinite(o).all()
        k0, v0 = s["k"].clone(), s["v"].clone()
        s["table"][1, 3] = bad
        cache.append(torch.ones(3, 8 * HD, dtype=torch.bfloat16, device="cuda"), batch)
        assert cache.last_device_error() == abi.TP_ERR_BATCH
        changed = (s["k"] != k0).flatten(1).any(1) & ~s["k"].isnan().flatten(1).any(1)
        assert not changed[[p for p in range(s["n_pages"]) if p not in keep[[0, 2]].flatten().tolist()]].any()
        s["k"].copy_(k0)
        s["v"].copy_(v0)
        s["table"].copy_(keep)
    for name, at, bad in (("kv_len", 1, 10 ** 9), ("kv_len", 1, -5), ("cu", 3, 10 ** 6), ("cu", 1, -3)):
        was = s[name][at].item()
        s[name][at] = bad
        o = cache.attend(q, batch)
        assert cache.last_device_error() == abi.TP_ERR_BATCH, name
        s[name][at] = was
    assert torch.equal(cache.attend(q, batch), good)
    assert cache.last_device_error() == abi.TP_OK


def _step(cache, batch, qkv, shared=0):
    q = cache.append(qkv, batch)
    return cache.attend(q, batch, shared_len=shared, lse=True)


def test_append_then_attend_over_several_steps():
    """A prompt, then single tokens, page after page: each step's rows against the
    64-bit form on what the cache then holds."""
    Hkv, H, T, page = 2, 8, 2, 8
    full = ref.make_batch([30, 11, 4], [0, 0, 0], Hkv, page, seed=31)
    freq = 10000.0 ** (-torch.arange(64, device="cuda") / 64)
    s = dict(full, lens=[9, 3, 0], new=[9, 3, 0])
    cache, _ = _cache(s, H, T, inv_freq=freq)
    g = torch.Generator(device="cuda").manual_seed(2)
    for step in range(8):
        cu = [0] + torch.tensor(s["new"]).cumsum(0).tolist()
        n = cu[-1]
        batch = cache.batch(torch.tensor(cu, dtype=torch.int32, device="cuda"),
                            torch.tensor(s["lens"], dtype=torch.int32, device="cuda"), s["table"], n, max(s["new"]))
        qkv = torch.randn(n, (H + 2 * Hkv) * HD, generator=g, device="cuda").to(torch.bfloat16)
        q = cache.append(qkv, batch)
        o, lse = cache.attend(q, batch, lse=True)
        assert cache.last_device_error() == 0
        check_attend(dict(s, cu=batch.cu_tokens), q, H, o, lse)
        s["new"] = [3, 1, 0 if step < 4 else 1]
        s["lens"] = [a + b for a, b in zip(s["lens"], s["new"])]


def test_two_streams_and_a_graph():
    """Calls on two streams at once, and a captured step replayed on changed contents."""
    shared = 2600
    s = ref.make_batch([1] * 6, [300, 20, 999, 0, 64, 128], 16, 16, shared=shared, seed=41)
    cache, batch = _cache(s, 64, 2, inv_freq=10000.0 ** (-torch.arange(32, device="cuda") / 32))
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = [torch.randn(s["n"], 96 * HD, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    eager = []
    for x in qkv:
        o, lse = _step(cache, batch, x, shared)
        eager.append((o.clone(), lse.clone()))
    qs = [cache.append(x, batch).clone() for x in qkv]
    cache.append(qkv[0], batch)
    torch.cuda.synchronize()
    one = [cache.attend(q, batch, shared_len=shared) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for st, q, out in zip(streams, qs, got):
            with torch.cuda.stream(st):
                out.append(cache.attend(q, batch, shared_len=shared))
    torch.cuda.synchronize()
    for out, want in zip(got, one):
        assert all(torch.equal(o, want) for o in out)
    graphs, held = [], []
    x = qkv[0].clone()
    for _ in range(2):  # two graphs of the same calls
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(_step(cache, batch, x, shared))
        graphs.append(graph)
    for i in (1, 2, 0):
        x.copy_(qkv[i])
        for graph, (o, lse) in zip(graphs, held):
            o.fill_(9)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, eager[i][0]) and torch.equal(lse, eager[i][1])


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("new,ctx,shared", [([1] * 5, [3, 50, 0, 7, 200], 48), ([2, 1, 5], [16, 90, 0], 0)])
def test_decode_is_the_composition(new, ctx, shared, fused):
    """TensorParallelAttention.decode against its parts called one by one, and the
    parts' projections against 64 bits."""
    abi, Attention, _, Cache = _modules()
    H, Hkv, T, d, page = 8, 2, 2, 512, 16
    s = ref.make_batch(new, ctx, Hkv, page, shared, seed=51)
    attn = Attention(d, H, Hkv, HD, T)
    freq = 10000.0 ** (-torch.arange(64, device="cuda") / 64)
    g = torch.Generator(device="cuda").manual_seed(4)
    w = lambda *sh: (torch.randn(*sh, generator=g, device="cuda") / math.sqrt(sh[1])).to(torch.bfloat16)
    Wq, Wk, Wv, Wo = w(H * HD, d), w(Hkv * HD, d), w(Hkv * HD, d), w(d, H * HD)
    wqkv, wo = attn.pack(Wq, Wk, Wv, Wo)
    x = torch.randn(s["n"], d, generator=g, device="cuda").to(torch.bfloat16)
    pages = []
    for _ in range(2):
        cache = Cache(attn, s["n_pages"], page, k=s["k"].clone(), v=s["v"].clone(), inv_freq=freq)
        pages.append((cache, cache.batch(s["cu"], s["kv_len"], s["table"], s["n"], s["max_new"])))
    (c0, b0), (c1, b1) = pages
    y = attn.decode(x, c0, b0, wqkv, wo, shared_len=shared, fused=fused)
    assert c0.last_device_error() == abi.TP_OK
    # the parts: x is rounded to bf16 after the q/k/v projection
    z = torch.cat([x.double() @ W.double().T for W in (Wq, Wk, Wv)], 1)
    order = []
    for t in range(T):
        for first, heads in ((0, H), (H, Hkv), (H + Hkv, Hkv)):
            order += range((first + t * heads // T) * HD, (first + (t + 1) * heads // T) * HD)
    qkv = z[:, order].to(torch.bfloat16).contiguous()
    q = c1.append(qkv, b1)
    o = c1.attend(q, b1, shared_len=shared)
    want = o.double() @ Wo.double().T
    # the two paths round q, k, v alike but where the 32-bit product falls on the
    # other side of a rounding border; both outputs are rounded once: in root mean
    # square both stay below 2^-8 each
    rel = ((y.double() - want).square().mean() / want.square().mean()).sqrt()
    assert rel <= 2 * U, rel.item()
    new_k = (c0.k.double() - c1.k.double()).nan_to_num().abs()
    assert (new_k <= 2 * U * c1.k.double().nan_to_num().abs() + 2.0 ** -16).all()


def test_decode_in_a_graph_and_with_the_overlapped_sum():
    abi, Attention, _, Cache = _modules()
    H, Hkv, T, d = 8, 2, 2, 512
    s = ref.make_batch([1, 3, 2, 40], [100, 0, 30, 7], Hkv, 16, seed=52, junk=0.0)
    attn = Attention(d, H, Hkv, HD, T)
    g = torch.Generator(device="cuda").manual_seed(5)
    w = lambda *sh: (torch.randn(*sh, generator=g, device="cuda") / math.sqrt(sh[1])).to(torch.bfloat16)
    wqkv, wo = attn.pack(w(H * HD, d), w(Hkv * HD, d), w(Hkv * HD, d), w(d, H * HD))
    x = torch.randn(s["n"], d, generator=g, device="cuda").to(torch.bfloat16)
    cache = Cache(attn, s["n_pages"], 16, k=s["k"], v=s["v"], inv_freq=1e4 ** (-torch.arange(64, device="cuda") / 64))
    batch = cache.batch(s["cu"], s["kv_len"], s["table"], s["n"], s["max_new"])
    y = attn.decode(x, cache, batch, wqkv, wo)
    assert torch.equal(attn.decode(x, cache, batch, wqkv, wo, overlap=True), y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = attn.decode(x, cache, batch, wqkv, wo)
    for _ in range(2):
        held.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, y)
    assert cache.last_device_error() == abi.TP_OK


def test_decode_matches_the_training_forward():
    """Without rotation, a whole sequence through decode is the causal forward."""
    abi, Attention, _, Cache = _modules()
    H, Hkv, T, d = 4, 2, 2, 256
    attn = Attention(d, H, Hkv, HD, T)
    g = torch.Generator(device="cuda").manual_seed(6)
    w = lambda *sh: (torch.randn(*sh, generator=g, device="cuda") / math.sqrt(sh[1])).to(torch.bfloat16)
    wqkv, wo = attn.pack(w(H * HD, d), w(Hkv * HD, d), w(Hkv * HD, d), w(d, H * HD))
    S = 24
    x = torch.randn(S, d, generator=g, device="cuda").to(torch.bfloat16)
    y, _ = attn.forward(x, 1, S, wqkv, wo)
    cache = Cache(attn, 4, 16)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    got = [attn.decode(x[:7].contiguous(), cache, cache.batch(i32(0, 7), i32(7), table, 7, 7), wqkv, wo)]
    for t in range(7, S):
        got.append(attn.decode(x[t:t + 1].contiguous(), cache, cache.batch(i32(0, 1), i32(t + 1), table, 1, 1),
                               wqkv, wo))
    rel = ((torch.cat(got).double() - y.double()).square().mean() / y.double().square().mean()).sqrt()
    assert rel <= 2 * U, rel.item()  # each side rounds its probabilities and outputs, 2^-8 in root mean square
