"""Refusals of the language operators' C entries that need no GPU: every argument is checked before the context,
so a null context shows which calls pass the checks (DM0_EINVAL with good arguments, the documented status with
bad ones)."""
import ctypes

import pytest

from vla_dual_expert_b200 import build

EINVAL, ESHAPE = -1, -2
P = 1 << 20   # a made-up aligned address: no entry reads it before its checks are done


@pytest.fixture(scope="module")
def abi():
    build.build()
    from vla_dual_expert_b200 import _abi
    return _abi


def _status(lib, name, order, good, **bad):
    a = {**good, **bad}
    assert set(bad) <= set(good), bad
    return getattr(lib, name)(None, *(a[k] for k in order))


EMBED = dict(table=P, ids=P, wide=1, B=2, T=3, vocab=10, hidden=64, scale=1.0, out=P, f32=0, bs=3 * 64, rs=64, stream=None)


@pytest.mark.parametrize("bad, status", [
    (dict(), EINVAL), (dict(table=None), EINVAL), (dict(ids=None), EINVAL), (dict(out=None), EINVAL),
    (dict(B=0), ESHAPE), (dict(T=0), ESHAPE), (dict(B=1 << 13, T=1 << 13), ESHAPE), (dict(vocab=0), ESHAPE),
    (dict(vocab=(1 << 22) + 1), ESHAPE), (dict(hidden=4), ESHAPE), (dict(hidden=60), ESHAPE),
    (dict(hidden=65544, rs=65544, bs=3 * 65544), ESHAPE),
    (dict(table=P + 2), EINVAL), (dict(out=P + 8), EINVAL), (dict(rs=56), EINVAL), (dict(rs=68), EINVAL),
    (dict(bs=-64), EINVAL), (dict(bs=64), EINVAL), (dict(bs=0), EINVAL)])
def test_embed_refusals(abi, bad, status):
    assert _status(abi.load_library(), "dm0_embed", EMBED, EMBED, **bad) == status


EGRAD = dict(ids=P, wide=0, B=2, T=3, vocab=10, hidden=64, scale=1.0, dout=P, f32=1, bs=3 * 64, rs=64, grad=P, acc=0,
             ws=P, wb=1 << 30, stream=None)


@pytest.mark.parametrize("bad, status", [
    (dict(), EINVAL), (dict(ids=None), EINVAL), (dict(dout=None), EINVAL), (dict(grad=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(B=0), ESHAPE), (dict(T=-1), ESHAPE), (dict(vocab=0), ESHAPE), (dict(hidden=0), ESHAPE),
    (dict(hidden=12), ESHAPE), (dict(rs=66), EINVAL), (dict(grad=P + 4), EINVAL), (dict(ws=P + 8), EINVAL)])
def test_embed_grad_refusals(abi, bad, status):
    lib = abi.load_library()
    assert _status(lib, "dm0_embed_grad", EGRAD, EGRAD, **bad) == status


def test_embed_grad_workspace(abi):
    lib = abi.load_library()
    n = lib.dm0_embed_grad_workspace(2, 3, 10, 64)
    assert n >= 2 * 6 * 4 + 11 * 4 + 2 * 64 * 4
    assert lib.dm0_embed_grad_workspace(0, 3, 10, 64) == 0 and lib.dm0_embed_grad_workspace(2, 3, 0, 64) == 0
    for k in (0, n - 1):
        assert _status(lib, "dm0_embed_grad", EGRAD, EGRAD, wb=k) == EINVAL


def _norm(abi, **kw):
    a = dict(batch=2, tokens=3, hidden=64, h_f32=1, y_f32=0, scale=1.0, post_gain=P, gate=P, gate_stride=64, pre_gain=P,
             mod_scale=P, mod_shift=P, mod_stride=64)
    a.update(kw)
    return abi.Dm0Norm(*a.values())


NORM_BAD = [(dict(batch=0), ESHAPE), (dict(tokens=0), ESHAPE), (dict(batch=1 << 13, tokens=1 << 13), ESHAPE),
            (dict(hidden=0), ESHAPE), (dict(hidden=60), ESHAPE), (dict(hidden=8200), ESHAPE),
            (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(gate_stride=32), EINVAL),
            (dict(mod_stride=66), EINVAL), (dict(mod_stride=-64), EINVAL), (dict(pre_gain=P + 4), EINVAL),
            (dict(gate=P + 8), EINVAL), (dict(mod_shift=P + 1), EINVAL)]


@pytest.mark.parametrize("bad, status", [(dict(), EINVAL)] + NORM_BAD)
def test_residual_norm_refusals(abi, bad, status):
    lib = abi.load_library()
    a = _norm(abi, **bad)
    assert lib.dm0_residual_norm(None, ctypes.byref(a), P, P, P, P, P, P, None) == status
    g = abi.Dm0NormGrads(P, P, P, P, P)
    assert lib.dm0_residual_norm_grad(None, ctypes.byref(a), P, 0, P, P, P, P, P, P, P, ctypes.byref(g), P, 1 << 30,
                                      None) == status


def test_residual_norm_null_and_misaligned(abi):
    lib = abi.load_library()
    a = _norm(abi)
    full = [P] * 6   # h, y, h_out, n_out, r_post, r_pre
    for i in range(6):
        for v in ((None,) if i > 3 else (None, P + 2)):
            args = list(full)
            args[i] = v
            assert lib.dm0_residual_norm(None, ctypes.byref(a), *args, None) == EINVAL
    assert lib.dm0_residual_norm(None, None, *full, None) == EINVAL


def test_residual_norm_grad_asks_for_vectors_that_are_there(abi):
    lib = abi.load_library()
    n = lib.dm0_residual_norm_grad_workspace(ctypes.byref(_norm(abi)))
    assert n >= 2 * 3 * 64 * 4
    bare = _norm(abi, post_gain=None, gate=None, pre_gain=None, mod_scale=None, mod_shift=None)
    for k in range(5):
        g = abi.Dm0NormGrads(*(P if i == k else None for i in range(5)))
        assert lib.dm0_residual_norm_grad(None, ctypes.byref(bare), P, 0, P, P, P, P, P, P, P, ctypes.byref(g), P,
                                          1 << 30, None) == EINVAL
    assert lib.dm0_residual_norm_grad_workspace(ctypes.byref(_norm(abi, hidden=12))) == 0
    g = abi.Dm0NormGrads(P, P, P, P, P)
    a = _norm(abi)
    assert lib.dm0_residual_norm_grad(None, ctypes.byref(a), P, 0, P, P, P, P, P, P, P, ctypes.byref(g), P, n - 1,
                                      None) == EINVAL


LOSS = dict(h=P, w=P, t=P, wide=1, tokens=5, vocab=100, hidden=128, loss=P, lse=P, ws=P, wb=1 << 40, stream=None)


@pytest.mark.parametrize("bad, status", [
    (dict(), EINVAL), (dict(h=None), EINVAL), (dict(w=None), EINVAL), (dict(t=None), EINVAL), (dict(loss=None), EINVAL),
    (dict(lse=None), EINVAL), (dict(ws=None), EINVAL), (dict(tokens=0), ESHAPE), (dict(tokens=(1 << 24) + 1), ESHAPE),
    (dict(vocab=0), ESHAPE), (dict(vocab=(1 << 22) + 1), ESHAPE), (dict(hidden=0), ESHAPE), (dict(hidden=96), ESHAPE),
    (dict(hidden=65600), ESHAPE), (dict(h=P + 2), EINVAL), (dict(w=P + 8), EINVAL), (dict(ws=P + 4), EINVAL),
    (dict(wb=0), EINVAL)])
def test_vocab_loss_refusals(abi, bad, status):
    assert _status(abi.load_library(), "dm0_vocab_loss", LOSS, LOSS, **bad) == status


LGRAD = dict(h=P, w=P, t=P, wide=1, lse=P, dloss=P, tokens=5, vocab=100, hidden=128, dh=P, dh32=0, dw=P, dw32=1, acc=1,
             ws=P, wb=1 << 40, stream=None)


@pytest.mark.parametrize("bad, status", [
    (dict(), EINVAL), (dict(lse=None), EINVAL), (dict(dloss=None), EINVAL), (dict(dh=None, dw=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(dw32=0), EINVAL), (dict(dh=P + 2), EINVAL), (dict(dw=P + 4), EINVAL),
    (dict(wb=255), EINVAL), (dict(hidden=32), ESHAPE), (dict(tokens=-1), ESHAPE)])
def test_vocab_loss_grad_refusals(abi, bad, status):
    assert _status(abi.load_library(), "dm0_vocab_loss_grad", LGRAD, LGRAD, **bad) == status


def test_vocab_workspaces(abi):
    lib = abi.load_library()
    assert lib.dm0_vocab_loss_workspace(0, 10, 64) == 0 and lib.dm0_vocab_loss_grad_workspace(5, 0, 64) == 0
    small, large = lib.dm0_vocab_loss_workspace(5, 100, 128), lib.dm0_vocab_loss_workspace(4096, 131072, 2048)
    assert 0 < small < large < 4096 * 131072   # no logits
    grad = lib.dm0_vocab_loss_grad_workspace(8192, 131072, 2048)
    assert 0 < grad < 2 ** 30 < 2 * 8192 * 131072


# ------------------------------------------------------------------------------ the binding's own checks (no GPU)
@pytest.fixture(scope="module")
def ops():
    """The operators of an Engine without a context: every call here is refused by the native binding before it."""
    build.build()
    from vla_dual_expert_b200 import language
    language._bind()
    o = language.LanguageOps()
    o.device, o.h = 0, ctypes.c_void_p()
    return o


def _cpu():
    import torch
    bf, f32, i64 = torch.bfloat16, torch.float32, torch.int64
    return dict(table=torch.zeros(9, 64, dtype=bf), ids=torch.zeros(2, 3, dtype=i64), d=torch.zeros(2, 3, 64),
                h=torch.zeros(2, 3, 64), g=torch.zeros(64), m=torch.zeros(2, 64), x=torch.zeros(5, 64, dtype=bf),
                t=torch.zeros(5, dtype=i64), l=torch.zeros(5), r=torch.zeros(2, 3, dtype=f32))


def test_binding_refuses_host_tensors(ops):
    c = _cpu()
    for call in (lambda: ops.embed(c["table"], c["ids"]), lambda: ops.embed_grad(c["ids"], c["d"], 9),
                 lambda: ops.residual_norm(c["h"]), lambda: ops.vocab_loss(c["x"], c["table"], c["t"]),
                 lambda: ops.residual_norm_grad(c["h"], None, c["h"], None, None, c["r"]),
                 lambda: ops.vocab_loss_grad(c["x"], c["table"], c["t"], c["l"], c["l"])):
        with pytest.raises(TypeError, match="cuda:0"):
            call()


def test_binding_refuses_what_is_no_tensor(ops):
    c = _cpu()
    with pytest.raises(TypeError, match="table must be a tensor"):
        ops.embed([1.0], c["ids"])
    with pytest.raises(TypeError, match="ids must be a tensor"):
        ops.embed(c["table"], [0, 1])
    with pytest.raises(TypeError, match="r_pre must be a tensor"):
        ops.residual_norm_grad(c["h"], None, c["h"], None, None, None)
    with pytest.raises(TypeError):
        ops.vocab_loss(c["x"], c["table"], None)


def test_binding_refuses_shapes(ops):
    import torch
    c = _cpu()
    with pytest.raises(ValueError, match="ids must be"):
        ops.embed(c["table"], torch.zeros(2, 2, 2, dtype=torch.int64))
    with pytest.raises(ValueError, match="hidden must be"):
        ops.vocab_loss(c["x"], torch.zeros(9, 128, dtype=torch.bfloat16), c["t"])
    with pytest.raises(ValueError, match="hidden must be"):
        ops.vocab_loss(c["x"][0], c["table"], c["t"])
    with pytest.raises(ValueError, match="residual stream"):
        ops.residual_norm(torch.zeros(64))
    with pytest.raises(ValueError):
        ops.prefill_tokens(torch.zeros(2, 4, 64, dtype=torch.bfloat16), c["table"], c["ids"][:1])


def test_binding_counts_its_arguments(ops):
    from vla_dual_expert_b200 import _language
    for name in ("embed", "embed_grad", "residual_norm", "residual_norm_grad", "vocab_loss", "vocab_loss_grad"):
        with pytest.raises(TypeError, match="expected"):
            getattr(_language, name)(0, 0)
