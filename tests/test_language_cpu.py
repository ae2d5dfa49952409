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
    """The operators' argument handling, on CPU tensors: their get_device() is -1, which stands for the context's."""
    from vla_dual_expert_b200 import language
    language._bind()
    o = language.LanguageOps()
    o.device = -1
    return language, o


def test_binding_refuses_types_shapes_and_strides(ops):
    import torch
    lang, o = ops
    t = torch.zeros(3, 4, 16)
    f32 = (torch.float32,)
    assert lang._check(t, -1, f32, (3, 4, 16), "t") == t.data_ptr()
    for bad in (t.double(), t.transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises(TypeError):
            lang._check(bad, -1, f32, (3, 4, 16), "t")
    with pytest.raises(TypeError):
        lang._check(t, 0, f32, (3, 4, 16), "t")        # another device
    with pytest.raises(ValueError):
        lang._check(t, -1, f32, (3, 4, 15), "t")
    assert lang._check_rows(t[:, 1:3], -1, (3, 2, 16), "t") == (64, 16)
    assert lang._check_rows(t[:1, 1:2], -1, (1, 1, 16), "t") == (0, 16)   # strides of dimensions of one say nothing
    assert lang._check_rows(t.transpose(0, 1), -1, (4, 3, 16), "t") == (16, 64)
    with pytest.raises(ValueError):
        lang._check_rows(t.transpose(1, 2), -1, (3, 16, 4), "t")
    with pytest.raises(TypeError):
        lang._check_rows(t.half(), -1, (3, 4, 16), "t")
    with pytest.raises(ValueError):
        o._ids(torch.zeros(2, 2, 2, dtype=torch.int64))
    with pytest.raises(TypeError):
        o._ids(torch.zeros(2, 2))


def test_binding_vectors_per_sample(ops):
    import torch
    _, o = ops
    m = torch.zeros(3, 40)
    assert o._vector(None, 3, 16, "v") == (None, 0)
    assert o._vector(m[0, :16], 3, 16, "v")[1] == 0
    assert o._vector(m[:, 8:24], 3, 16, "v") == (m.data_ptr() + 32, 40)   # rows of a wider table
    assert o._vector(m[:1, :16], 1, 16, "v")[1] == 0
    with pytest.raises(ValueError):
        o._vector(m[:2, :16], 3, 16, "v")
    with pytest.raises(ValueError):
        o._vector(m[0, :16].expand(3, 16), 3, 16, "v")     # one row seen three times: its gradient would have none
    with pytest.raises(TypeError):
        o._vector(m.double()[0, :16], 3, 16, "v")
    h = torch.zeros(3, 2, 16)
    with pytest.raises(ValueError):
        o._norm(h, None, None, None, 1.0, None, m[:, :16], torch.zeros(3, 16))   # scale and shift laid out differently
    with pytest.raises(ValueError):
        o._norm(h, torch.zeros(3, 2, 8), None, None, 1.0, None, None, None)
    with pytest.raises(ValueError):
        o._norm(torch.zeros(16), None, None, None, 1.0, None, None, None)


def test_binding_accumulation_needs_a_gradient(ops):
    import torch
    _, o = ops
    ids, d = torch.zeros(2, dtype=torch.int64), torch.zeros(2, 16)
    with pytest.raises(ValueError):
        o.embed_grad(ids, d, 4, accumulate=True)
    h, w, l = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(5, 64, dtype=torch.bfloat16), torch.zeros(2)
    with pytest.raises(ValueError):
        o.vocab_loss_grad(h, w, ids, l, l, accumulate=True)
    with pytest.raises(ValueError):
        o.vocab_loss(h, torch.zeros(5, 128, dtype=torch.bfloat16), ids)
