"""Attention over the paged cache at the borders of its kernels, each case with
the kernels that it is meant for by name: up to 16 and up to 32 query rows to a
key head (new tokens of the longest sequence, or for shared keys all rows of the
buffers, times the query heads of a group) go to the few-rows kernel's two forms,
more to the tensor-memory kernel.

Tolerances: those of test_gpu_kv_cache.check_attend."""
import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_kv_cache import HD, _cache, _modules, _q, check_attend

pytestmark = pytest.mark.gpu

FEW, MANY, S_FEW, S_MANY = "kv_attend_few", "kv_attend_many", "kv_attend_shared_few", "kv_attend_shared_many"

CASES = [  # new, ctx, H, Hkv, T, page, shared, causal, rows behind the last sequence, kernels
    # own keys: 16, 17, 32 and 33 rows
    ([4, 1, 3], [500, 0, 63], 8, 2, 2, 16, 0, True, 3, [FEW]),
    ([17, 2], [100, 900], 3, 3, 1, 32, 0, True, 0, [FEW]),
    ([8, 8, 1], [3000, 5, 64], 8, 2, 2, 64, 0, True, 1, [FEW]),
    ([32], [1], 1, 1, 1, 8, 0, False, 0, [FEW]),
    ([33, 1], [1000, 31], 2, 2, 2, 16, 0, True, 0, [MANY]),
    ([11, 4], [70, 129], 6, 2, 2, 128, 0, True, 2, [MANY]),
    ([2], [300], 34, 2, 2, 16, 0, True, 0, [MANY]),                     # 17 query heads to a key head
    ([2, 1, 1], [300, 0, 50], 16, 1, 1, 16, 0, True, 0, [FEW]),         # 16
    # shared keys: 16, 17, 32 and 33 rows
    ([1] * 4, [3, 0, 200, 65], 32, 8, 8, 32, 11000, True, 0, [S_FEW, FEW]),
    ([1] * 3, [3, 0, 200], 40, 8, 4, 64, 17000, True, 0, [S_FEW, FEW]),           # 15, groups of five
    ([1] * 15, [7 * i for i in range(15)], 8, 8, 8, 16, 2400, False, 1, [S_FEW, FEW]),
    ([1] * 16, [7 * i for i in range(16)], 8, 8, 8, 16, 2300, True, 1, [S_FEW, FEW]),
    ([1] * 8, [30, 0, 1, 2, 64, 63, 700, 5], 32, 8, 2, 128, 4700, True, 0, [S_FEW, FEW]),
    ([17, 1, 1, 1], [9, 0, 80, 3], 8, 8, 1, 16, 11100, True, 12, [S_FEW, FEW]),   # 32; own 17
    ([1] * 10, [40 * i for i in range(10)], 24, 8, 8, 64, 3700, True, 1, [S_MANY, FEW]),
    ([33], [5], 1, 1, 1, 16, 100, True, 0, [MANY]),                     # one sequence shares with nobody
    ([12, 11, 12, 11], [2, 0, 64, 130], 24, 8, 4, 32, 11111, True, 0, [S_MANY, MANY]),
    # 128 and 256 shared rows and one more
    ([1] * 32, [i % 5 for i in range(32)], 32, 8, 8, 16, 1100, True, 0, [S_MANY, FEW]),
    ([1] * 32, [i % 5 for i in range(32)], 32, 8, 8, 16, 1100, False, 1, [S_MANY, FEW]),
    ([2] * 32, [90] * 32, 32, 8, 8, 16, 1100, True, 0, [S_MANY, FEW]),
    ([2] * 32, [90] * 32, 32, 8, 8, 16, 1100, True, 1, [S_MANY, FEW]),
    # more sequences than a block has lanes to look at them
    ([1] * 200, [(i * 37) % 150 for i in range(200)], 8, 2, 2, 16, 700, True, 0, [S_MANY, FEW]),
    ([i % 3 for i in range(300)], [(i * 53) % 90 for i in range(300)], 4, 2, 2, 32, 450, True, 2, [S_MANY, FEW]),
    ([9 + i % 8 for i in range(150)], [(i * 61) % 200 for i in range(150)], 8, 2, 2, 16, 1700, True, 0, [S_MANY, MANY]),
    ([int(i % 20 == 3) for i in range(150)], [(i * 37) % 150 for i in range(150)], 8, 2, 2, 16, 900, True, 0,
     [S_FEW, FEW]),
    # few rows and many of single sequences behind keys that all share; ragged own rows
    ([9, 1] * 10, [0] * 20, 40, 5, 5, 8, 2700, True, 0, [S_MANY, MANY]),
    ([9 + i % 8 for i in range(30)], [(61 * i) % 700 for i in range(30)], 32, 8, 8, 16, 1900, True, 2, [S_MANY, MANY]),
    # as many bytes of shared keys, but more rows to join than those reads cost
    ([16] * 128, [i % 40 for i in range(128)], 32, 8, 8, 64, 256, True, 0, [MANY]),
    ([16] * 4, [i for i in range(4)], 32, 8, 8, 64, 9600, True, 0, [S_MANY, MANY]),
    ([1] * 64, [i for i in range(64)], 32, 8, 8, 64, 320, True, 0, [FEW]),
    ([1] * 64, [i for i in range(64)], 32, 8, 8, 64, 512, True, 0, [S_MANY, FEW]),
    ([int(i % 20 == 3) for i in range(150)], [(i * 37) % 150 for i in range(150)], 8, 2, 2, 16, 0, True, 0, [FEW]),
]


@pytest.mark.parametrize("new,ctx,H,Hkv,T,page,shared,causal,spare,kernels", CASES)
def test_at_the_borders_of_the_kernels(new, ctx, H, Hkv, T, page, shared, causal, spare, kernels):
    abi = _modules()[0]
    s = ref.make_batch(new, ctx, Hkv, page, shared, spare_rows=spare, seed=len(new) + page)
    cache, batch = _cache(s, H, T, causal)
    q = _q(s["n"], H, page)
    out = torch.full((s["n"], H * HD), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = cache.attend(q, batch, shared_len=shared, lse=True, out=out, flags=abi.TP_FLAG_TIMING)
    names = [name for name, _ in abi.tp_attn_kernel_times(cache.attn.plan)]
    assert names[:-1] == kernels and names[-1] == "kv_combine"
    assert cache.last_device_error() == abi.TP_OK
    check_attend(s, q, H, o, lse, causal)
    rows = sum(new)
    assert (o[rows:] == 7.0).all()
    for _ in range(2):
        again, again_lse = cache.attend(q, batch, shared_len=shared, lse=True)
        assert torch.equal(o[:rows], again[:rows]) and torch.equal(lse[:rows], again_lse[:rows])


@pytest.mark.parametrize("new,shared", [(1, 1700), (5, 2100)])
def test_shared_keys_longer_than_sequences(new, shared):
    """Behind shared keys that some sequences do not reach the end of: cut rows, no
    keys at all, more new tokens than keys."""
    abi = _modules()[0]
    B, Hkv, H = 60, 2, 8
    s = ref.make_batch([new] * B, [3] * B, Hkv, 16, shared=shared, seed=6)
    for b, n in ((0, shared - 50), (1, 0), (2, 1), (3, 3), (7, shared - 1), (8, shared + 1), (59, 64)):
        s["lens"][b] = n
    s["kv_len"].copy_(torch.tensor(s["lens"]))
    cache, batch = _cache(s, H, 2)
    q = _q(s["n"], H, 2)
    o, lse = cache.attend(q, batch, shared_len=shared, lse=True, flags=abi.TP_FLAG_TIMING)
    assert [name for name, _ in abi.tp_attn_kernel_times(cache.attn.plan)] == [S_MANY, FEW, "kv_combine"]
    assert cache.last_device_error() == 0
    check_attend(s, q, H, o, lse)


def test_shared_keys_of_many_own_rows_bad_offsets():
    """Offsets that descend, or begin behind the first row, leave rows that the shared
    keys' work does not cover: what they get is unspecified, the call reports it and
    the sequences' other rows, where there are any, are as ever."""
    abi = _modules()[0]
    B, new, Hkv, H, shared = 40, 8, 8, 64, 1920
    s = ref.make_batch([new] * B, [3] * B, Hkv, 64, shared=shared, seed=26)
    cache, batch = _cache(s, H, 8)
    q = _q(s["n"], H, 12)
    good = cache.attend(q, batch, shared_len=shared, flags=abi.TP_FLAG_TIMING)
    assert [name for name, _ in abi.tp_attn_kernel_times(cache.attn.plan)] == [S_MANY, MANY, "kv_combine"]
    assert cache.last_device_error() == abi.TP_OK
    check_attend(s, q, H, good, None)
    keep = s["cu"].clone()
    for at, bad in ((B, 3), (B, 0), (B, -2 ** 31), (B // 2, 2 ** 31 - 1), (1, 300), (0, -7), (B - 1, 5)):
        s["cu"][at] = bad
        cache.attend(q, batch, shared_len=shared)
        assert cache.last_device_error() == abi.TP_ERR_BATCH, (at, bad)
        s["cu"].copy_(keep)
    for bad in (list(range(320, -1, -8)), [0, 320] * 20 + [0], [160] * 41, [2 ** 31 - 1] * 41, [-1] * 41):
        s["cu"].copy_(torch.tensor(bad))
        cache.attend(q, batch, shared_len=shared)
        assert cache.last_device_error() == (abi.TP_OK if bad[0] == 160 else abi.TP_ERR_BATCH), bad
        s["cu"].copy_(keep)
    s["cu"][0] = 5  # the first sequence's last three rows; those before are nobody's
    o = torch.full_like(good, 7.0)
    cache.attend(q, batch, shared_len=shared, out=o)
    assert cache.last_device_error() == abi.TP_OK and (o[:5] == 7).all()
    check_attend(dict(s, new=[3] + [new] * (B - 1), cu=s["cu"] - 5), q[5:], H, o[5:], None)
    s["cu"].copy_(keep)
    assert torch.equal(cache.attend(q, batch, shared_len=shared), good)
    assert cache.last_device_error() == abi.TP_OK
