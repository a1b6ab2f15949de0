"""What the 4-bit entry points refuse, on the CPU: status codes come back before
any device work, and the Python layer refuses tensors that do not fit."""
import pytest
import torch


@pytest.fixture(scope="module")
def abi():
    from megatron_tensor_transformer_w1_gb300 import build
    build.build()
    from megatron_tensor_transformer_w1_gb300 import tpffn
    return tpffn


@pytest.fixture(scope="module")
def plans(abi):
    make = lambda *a: abi.tp_ffn_plan_create(*a)[1]
    p = dict(swiglu=make(512, 1024, 8, abi.TP_ACT_SWIGLU, abi.TP_BF16),
             gelu=make(512, 1000, 8, abi.TP_ACT_GELU_TANH, abi.TP_BF16),
             none=abi.tp_attn_out_plan_create(512, 8, 8, 128, 4, abi.TP_BF16)[1],
             f32=make(64, 256, 2, abi.TP_ACT_GELU_TANH, abi.TP_F32))
    yield p
    for plan in p.values():
        abi.tp_ffn_plan_destroy(plan)


A = 4096  # an address that is never used


@pytest.mark.parametrize("name", ["tp_quantize4", "tp_dequantize4"])
def test_quantize_refusals(abi, name):
    def call(a=A, rows=8, cols=64, segments=1, group=32, b=A, c=A):
        args = (a, rows, cols, segments, group, b, c) if name == "tp_quantize4" else (a, b, rows, cols, segments, group, c)
        return getattr(abi, name)(*args)
    for bad in (dict(rows=-1), dict(cols=-1), dict(segments=0), dict(segments=3), dict(group=0), dict(group=16),
                dict(group=96), dict(group=256), dict(a=None), dict(b=None), dict(c=None)):
        assert call(**bad) == abi.TP_ERR_INVALID, bad
    for bad in (dict(a=A + 8), dict(b=A + 2), dict(c=A + 4)):
        assert call(**bad) == abi.TP_ERR_ALIGN, bad
    assert call(cols=(1 << 30) + 32) == abi.TP_ERR_UNSUPPORTED
    assert call(rows=1 << 40, cols=1 << 10) == abi.TP_ERR_UNSUPPORTED
    assert call(rows=0, a=None) == abi.TP_OK and call(cols=0) == abi.TP_OK


def test_packed_bytes(abi, plans):
    # 128-slot tiles in pairs, 128-column chunks: codes 16384 bytes and 512 for each group of a chunk; a factor of
    # 4 bytes for each of a pair's 256 rows and 16 bytes for the whole
    assert abi.tp_ffn_packed4_bytes(plans["swiglu"], 0, 128) == 8 * 4 * (16384 + 512) + 8 * 1024 + 16
    assert abi.tp_ffn_packed4_bytes(plans["gelu"], 0, 64) == 4 * 4 * (16384 + 1024) + 4 * 1024 + 16
    assert abi.tp_ffn_packed4_bytes(plans["gelu"], 1, 32) == 2 * 8 * (16384 + 2048) + 2 * 1024 + 16
    assert abi.tp_ffn_packed4_bytes(plans["none"], 0, 64) == 0
    for args in ((None, 0, 64), (plans["f32"], 0, 64), (plans["gelu"], 2, 64), (plans["gelu"], 0, 48)):
        assert abi.tp_ffn_packed4_bytes(*args) == 0


def test_shard_refusals(abi, plans):
    ok = [A] * 5
    for i in range(5):
        for bad, want in ((None, abi.TP_ERR_INVALID), (A + 8, abi.TP_ERR_ALIGN)):
            args = ok[:i] + [bad] + ok[i + 1:]
            assert abi.tp_ffn_shard_columns4(plans["swiglu"], 64, *args) == want
            assert abi.tp_ffn_unshard_columns4(plans["swiglu"], 64, args[4], *args[:4]) == want
    for plan, group in ((None, 64), (plans["none"], 64), (plans["f32"], 64), (plans["gelu"], 65)):
        assert abi.tp_ffn_shard_columns4(plan, group, A, A, A, A, A) == abi.TP_ERR_INVALID
    for plan, group in ((None, 64), (plans["f32"], 64), (plans["gelu"], 65)):
        assert abi.tp_ffn_shard_rows4(plan, group, A, A, A) == abi.TP_ERR_INVALID
    assert abi.tp_ffn_shard_rows4(plans["gelu"], 64, None, A, A) == abi.TP_ERR_INVALID
    assert abi.tp_ffn_unshard_rows4(plans["gelu"], 64, A, A, A + 1) == abi.TP_ERR_ALIGN


def test_forward_refusals(abi, plans):
    def call(plan="gelu", group=64, n=4, x=A, up=A, down=A, b1=None, b2=None, y=A, ws=A, nbytes=1 << 40):
        return abi.tp_ffn_fwd4(plans.get(plan), group, n, x, up, down, b1, b2, y, ws, nbytes)
    for bad in (dict(plan="no"), dict(group=100), dict(n=-1), dict(x=None), dict(up=None), dict(down=None), dict(y=None),
                dict(ws=None), dict(nbytes=100)):
        assert call(**bad) == abi.TP_ERR_INVALID, bad
    for bad in (dict(plan="f32"), dict(plan="swiglu", b1=A), dict(n=1 << 40)):
        assert call(**bad) == abi.TP_ERR_UNSUPPORTED, bad
    for bad in (dict(x=A + 2), dict(up=A + 2), dict(down=A + 8), dict(b1=A + 8), dict(b2=A + 8), dict(y=A + 2), dict(ws=A + 8)):
        assert call(**bad) == abi.TP_ERR_ALIGN, bad
    assert call(n=0, x=None) == abi.TP_OK
    assert abi.tp_ffn_workspace4_bytes(plans["gelu"], 4) > 0
    assert abi.tp_ffn_workspace4_bytes(plans["f32"], 4) == 0 == abi.tp_ffn_workspace4_bytes(None, 4)


def test_attention_refusals(abi):
    rc, plan = abi.tp_attn_plan_create(256, 8, 2, 128, 2, True, abi.TP_BF16)
    assert rc == abi.TP_OK
    assert abi.tp_attn_packed4_bytes(plan, 0, 64) == 6 * 2 * (16384 + 1024) + 6 * 1024 + 16
    assert abi.tp_attn_packed4_bytes(plan, 0, 60) == 0 == abi.tp_attn_packed4_bytes(None, 0, 64)
    four = [A] * 4
    assert abi.tp_attn_shard_weights4(plan, 64, [A, A, None, A], four, A, A) == abi.TP_ERR_INVALID
    assert abi.tp_attn_shard_weights4(plan, 64, four, [A, A, A, A + 2], A, A) == abi.TP_ERR_ALIGN
    assert abi.tp_attn_shard_weights4(plan, 63, four, four, A, A) == abi.TP_ERR_INVALID
    assert abi.tp_attn_unshard_weights4(plan, 64, None, A, four, four) == abi.TP_ERR_INVALID
    cache, batch = abi.KvCache(A, A, 4, 16), abi.KvBatch(2, 2, 1, 4, A, A, A)
    need = abi.tp_attn_kv_workspace_bytes(plan, batch, 16, 0, abi.TP_KV_DECODE4)
    assert need > abi.tp_attn_kv_workspace_bytes(plan, batch, 16, 0, abi.TP_KV_ATTEND) > 0
    def call(group=64, x=A, up=A, down=A, y=A, ws=A, nbytes=need):
        return abi.tp_attn_decode_fwd4(plan, cache, batch, None, 0, group, x, up, down, y, ws, nbytes)
    for bad in (dict(group=1), dict(x=None), dict(up=None), dict(down=None), dict(y=None), dict(ws=None), dict(nbytes=need - 1)):
        assert call(**bad) == abi.TP_ERR_INVALID, bad
    for bad in (dict(x=A + 8), dict(up=A + 8), dict(down=A + 8), dict(y=A + 8), dict(ws=A + 8)):
        assert call(**bad) == abi.TP_ERR_ALIGN, bad
    abi.tp_attn_plan_destroy(plan)


def test_codes_refusals(abi):
    from megatron_tensor_transformer_w1_gb300.weights4 import Codes4, group_of
    u8, bf = dict(dtype=torch.uint8), dict(dtype=torch.bfloat16)
    ok = Codes4(torch.zeros(3, 50, **u8), torch.zeros(3, 4, **bf), 99, group=32, segments=1)
    assert (ok.rows, ok.cols) == (3, 99)
    for codes, scales, cols, group, segments in (
            (torch.zeros(3, 50, **u8), torch.zeros(3, 4, **bf), 99, 48, 1),
            (torch.zeros(3, 50, **u8), torch.zeros(3, 4, **bf), 99, 32, 2),
            (torch.zeros(3, 49, **u8), torch.zeros(3, 4, **bf), 99, 32, 1),
            (torch.zeros(3, 50, **u8), torch.zeros(3, 3, **bf), 99, 32, 1),
            (torch.zeros(3, 50, **u8), torch.zeros(3, 4), 99, 32, 1),
            (torch.zeros(3, 50), torch.zeros(3, 4, **bf), 99, 32, 1),
            (torch.zeros(50, 3, **u8).T, torch.zeros(3, 4, **bf), 99, 32, 1),
            (torch.zeros(150, **u8), torch.zeros(3, 4, **bf), 99, 32, 1)):
        with pytest.raises(ValueError):
            Codes4(codes, scales, cols, group=group, segments=segments)
    with pytest.raises(ValueError):
        group_of(64, ok)
    assert group_of(None, ok) == 32 and group_of(None) == 128
