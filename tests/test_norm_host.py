"""What the norms' entry points refuse, on the CPU: status codes come back before any
device work."""
import pytest


@pytest.fixture(scope="module")
def abi():
    from megatron_tensor_transformer_w1_gb300 import build
    build.build()
    from megatron_tensor_transformer_w1_gb300 import tpffn
    return tpffn


A = 4096  # an address that is never used
NAMES = "n n_gates x b w_after c_after gate w_before c_before r out stats".split()
BACK = ("n n_gates b r stats w_after c_after gate w_before dr dout dx db dw_after dc_after dgate dw_before dc_before "
        "workspace workspace_bytes").split()


def _norm(abi, **kw):
    d = dict(d=64, kind=abi.TP_NORM_RMS, dtype=abi.TP_BF16, before=1, after=1, eps=1e-5, scale=1.0)
    d.update(kw)
    return abi.Norm(*(d[k] for k in ("d", "kind", "dtype", "before", "after", "eps", "scale")))


def _forward(abi, norm=None, **kw):
    args = dict.fromkeys(NAMES, A)
    args.update(n=6, n_gates=2)
    args.update(kw)
    return abi.tp_norm_fwd(norm if norm is not None else _norm(abi), *(args[k] for k in NAMES))


def _backward(abi, norm=None, **kw):
    args = dict.fromkeys(BACK, A)
    args.update(n=6, n_gates=2, workspace_bytes=1 << 40)
    args.update(kw)
    return abi.tp_norm_bwd(norm if norm is not None else _norm(abi), *(args[k] for k in BACK))


def test_sizes(abi):
    for bad in (dict(d=0), dict(d=-8), dict(kind=2), dict(dtype=5), dict(before=2), dict(after=-1)):
        assert _forward(abi, _norm(abi, **bad)) == abi.TP_ERR_INVALID == _backward(abi, _norm(abi, **bad)), bad
        assert abi.tp_norm_workspace_bytes(_norm(abi, **bad), 6, 2) == 0
    for bad in (dict(d=60), dict(d=8200)):
        assert _forward(abi, _norm(abi, **bad)) == abi.TP_ERR_UNSUPPORTED == _backward(abi, _norm(abi, **bad)), bad
    for kw, want in ((dict(n=-1), abi.TP_ERR_INVALID), (dict(n=(1 << 30) + 2), abi.TP_ERR_UNSUPPORTED),
                     (dict(n=7), abi.TP_ERR_INVALID), (dict(n_gates=-1), abi.TP_ERR_INVALID),
                     (dict(n_gates=4), abi.TP_ERR_INVALID), (dict(n=0), abi.TP_OK)):
        assert _forward(abi, **kw) == want, kw
        assert _backward(abi, **kw) == want, kw
    assert abi.tp_norm_fwd(None, 6, *[A] * 11) == abi.TP_ERR_INVALID
    assert abi.tp_norm_workspace_bytes(_norm(abi), 6, 2) > 0


def test_forward_pointers(abi):
    for name in ("x", "b", "gate", "r", "out"):
        assert _forward(abi, **{name: None}) == abi.TP_ERR_INVALID, name
    for name in NAMES[2:]:
        assert _forward(abi, **{name: A + 8}) == abi.TP_ERR_ALIGN, name
    plain = _norm(abi, before=0, after=0)
    for name in ("w_after", "c_after", "w_before", "c_before", "out"):
        args = dict(w_after=None, c_after=None, w_before=None, c_before=None, out=None)
        args[name] = A
        assert _forward(abi, plain, **args) == abi.TP_ERR_INVALID, name


def test_backward_pointers(abi):
    for name in ("b", "r", "stats", "gate", "dout", "workspace"):
        assert _backward(abi, **{name: None}) == abi.TP_ERR_INVALID, name
    for name in BACK[2:-1]:
        assert _backward(abi, **{name: A + 8}) == abi.TP_ERR_ALIGN, name
    need = abi.tp_norm_workspace_bytes(_norm(abi), 6, 2)
    assert _backward(abi, workspace_bytes=need - 1) == abi.TP_ERR_INVALID
    gone = dict(w_after=None, c_after=None, w_before=None, dout=None, dw_after=None, dc_after=None, dw_before=None, dc_before=None)
    for name in gone:
        assert _backward(abi, _norm(abi, before=0, after=0), **dict(gone, **{name: A})) == abi.TP_ERR_INVALID, name
