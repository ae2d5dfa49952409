"""Which check refuses a call of the language operators' C entries.  Every argument is checked before the context, so
without one a call that passes ends at "null context", and another message names the check that did not."""
import ctypes

import pytest

from tests.test_language_cpu import EGRAD, EINVAL, EMBED, ESHAPE, LGRAD, LOSS, P, _norm, abi  # noqa: F401

PASSED = "null context"
GOOD = {"dm0_embed": EMBED, "dm0_embed_grad": EGRAD, "dm0_vocab_loss": LOSS, "dm0_vocab_loss_grad": LGRAD}


def refusal(lib, st):
    return st, lib.dm0_last_refusal().decode()


def call(lib, name, **bad):
    a = {**GOOD[name], **bad}
    assert set(bad) <= set(GOOD[name])
    return refusal(lib, getattr(lib, name)(None, *a.values()))


NULL, SIZES, ROWS = "null argument", "bad batch, tokens or vocab", "rows must be 16-byte aligned"
HIDDEN8, SMALL, OVERLAP = "hidden must be a multiple of 8", "workspace too small", "the rows of out overlap"
VOCAB, HIDDEN64, OPERANDS = "tokens or vocab out of range", "hidden must be a multiple of 64", "hidden states and weights"
WHERE = "gradients and workspace must be 16-byte aligned"


@pytest.mark.parametrize("name", GOOD)
def test_good_arguments_pass_every_check(abi, name):  # noqa: F811
    assert call(abi.load_library(), name) == (EINVAL, PASSED)


@pytest.mark.parametrize("name, bad, status, why", [
    *[("dm0_embed", {k: None}, EINVAL, NULL) for k in ("table", "ids", "out")],
    *[("dm0_embed", b, ESHAPE, SIZES) for b in (dict(B=0), dict(T=0), dict(B=1 << 13, T=(1 << 11) + 1), dict(vocab=0),
                                                dict(vocab=(1 << 22) + 1), dict(B=-1, T=-3))],
    *[("dm0_embed", b, ESHAPE, HIDDEN8) for b in (dict(hidden=0), dict(hidden=4), dict(hidden=60, rs=64),
                                                  dict(hidden=65544, rs=65544, bs=3 * 65544))],
    ("dm0_embed", dict(table=P + 2), EINVAL, "the table must be 16-byte aligned"),
    *[("dm0_embed", b, EINVAL, ROWS) for b in (dict(out=P + 8), dict(rs=56), dict(rs=68, bs=3 * 72), dict(bs=-192),
                                               dict(bs=196), dict(rs=66, bs=256, f32=1), dict(rs=-64))],
    *[("dm0_embed", b, EINVAL, OVERLAP) for b in (dict(bs=64), dict(bs=0), dict(bs=184), dict(bs=128),
                                                  dict(bs=64, rs=64, B=3), dict(bs=64, rs=184, B=3))],
    *[("dm0_embed_grad", {k: None}, EINVAL, NULL) for k in ("ids", "dout", "grad", "ws")],
    *[("dm0_embed_grad", b, ESHAPE, SIZES) for b in (dict(B=0), dict(T=-1), dict(B=1 << 24, T=2), dict(vocab=0))],
    *[("dm0_embed_grad", b, ESHAPE, HIDDEN8) for b in (dict(hidden=0), dict(hidden=12), dict(hidden=1 << 17, rs=1 << 17))],
    *[("dm0_embed_grad", b, EINVAL, "grad and workspace must be 16-byte aligned") for b in (dict(grad=P + 4),
                                                                                            dict(ws=P + 8))],
    *[("dm0_embed_grad", b, EINVAL, ROWS) for b in (dict(dout=P + 4), dict(rs=66), dict(rs=60), dict(bs=194),
                                                    dict(rs=68, f32=0), dict(bs=-4))],
    *[("dm0_vocab_loss", {k: None}, EINVAL, NULL) for k in ("h", "w", "t", "loss", "lse", "ws")],
    *[("dm0_vocab_loss", b, ESHAPE, VOCAB) for b in (dict(tokens=0), dict(tokens=(1 << 24) + 1), dict(vocab=0),
                                                     dict(vocab=(1 << 22) + 1))],
    *[("dm0_vocab_loss", b, ESHAPE, HIDDEN64) for b in (dict(hidden=0), dict(hidden=96), dict(hidden=65600))],
    *[("dm0_vocab_loss", b, EINVAL, OPERANDS) for b in (dict(h=P + 2), dict(w=P + 8))],
    ("dm0_vocab_loss", dict(ws=P + 4), EINVAL, "the workspace must be 16-byte aligned"),
    *[("dm0_vocab_loss_grad", b, EINVAL, NULL) for b in (dict(h=None), dict(w=None), dict(t=None), dict(lse=None),
                                                         dict(dloss=None), dict(ws=None), dict(dh=None, dw=None))],
    *[("dm0_vocab_loss_grad", b, ESHAPE, VOCAB) for b in (dict(tokens=-1), dict(vocab=-5))],
    *[("dm0_vocab_loss_grad", b, ESHAPE, HIDDEN64) for b in (dict(hidden=32), dict(hidden=1 << 20))],
    *[("dm0_vocab_loss_grad", b, EINVAL, WHERE) for b in (dict(dh=P + 2), dict(dw=P + 4), dict(ws=P + 8))],
    ("dm0_vocab_loss_grad", dict(dw32=0), EINVAL, "only an fp32 weight gradient accumulates")])
def test_the_check_that_refuses(abi, name, bad, status, why):  # noqa: F811
    st, said = call(abi.load_library(), name, **bad)
    assert st == status and said.startswith(why), (st, said)


@pytest.mark.parametrize("name, bad", [
    ("dm0_embed", dict(bs=192)), ("dm0_embed", dict(bs=64, rs=128, B=2)), ("dm0_embed", dict(B=1, bs=0)),
    ("dm0_embed", dict(rs=68, bs=204, f32=1)), ("dm0_embed", dict(T=1, bs=64)), ("dm0_embed_grad", dict(bs=0)),
    ("dm0_embed_grad", dict(dout=P + 16, rs=68)), ("dm0_vocab_loss_grad", dict(dh=None)),
    ("dm0_vocab_loss_grad", dict(dw=None, dw32=0)), ("dm0_vocab_loss_grad", dict(dw32=0, acc=0))])
def test_calls_at_the_edge_of_the_checks_pass(abi, name, bad):  # noqa: F811
    assert call(abi.load_library(), name, **bad) == (EINVAL, PASSED)


def test_workspaces_one_byte_short(abi):  # noqa: F811
    lib = abi.load_library()
    sizes = {"dm0_embed_grad": lib.dm0_embed_grad_workspace(2, 3, 10, 64),
             "dm0_vocab_loss": lib.dm0_vocab_loss_workspace(5, 100, 128),
             "dm0_vocab_loss_grad": lib.dm0_vocab_loss_grad_workspace(5, 100, 128)}
    for name, n in sizes.items():
        assert n > 0
        assert call(lib, name, wb=n) == (EINVAL, PASSED)
        assert call(lib, name, wb=n - 1) == (EINVAL, SMALL) and call(lib, name, wb=0) == (EINVAL, SMALL)
    for kw in (dict(), dict(gate_stride=0, mod_stride=0), dict(batch=1, tokens=700)):
        a = _norm(abi, **kw)
        n = lib.dm0_residual_norm_grad_workspace(ctypes.byref(a))
        assert n > 0
        assert norm_grad(abi, a, bytes=n) == (EINVAL, PASSED) and norm_grad(abi, a, bytes=n - 1) == (EINVAL, SMALL)


def norm(abi, a, **bad):  # noqa: F811
    lib, t = abi.load_library(), dict(h=P, y=P, h_out=P, n_out=P, r_post=P, r_pre=P)
    assert set(bad) <= set(t)
    return refusal(lib, lib.dm0_residual_norm(None, a and ctypes.byref(a), *{**t, **bad}.values(), None))


def norm_grad(abi, a, grads=(P,) * 5, **bad):  # noqa: F811
    lib = abi.load_library()
    t = dict(dn=P, f32=0, dh_out=P, h_out=P, y=P, r_post=P, r_pre=P, dh=P, dy=P, g=abi.Dm0NormGrads(*grads), ws=P,
             bytes=1 << 30)
    assert set(bad) <= set(t)
    t.update(bad)
    t["g"] = t["g"] and ctypes.byref(t["g"])
    return refusal(lib, lib.dm0_residual_norm_grad(None, a and ctypes.byref(a), *t.values(), None))


STRIDES, VECTORS = "per-sample strides are 0 or at least hidden", "gain, gate and modulation vectors must be 16-byte"


@pytest.mark.parametrize("bad, status, why", [
    (dict(), EINVAL, PASSED),
    *[(b, ESHAPE, "bad batch or tokens") for b in (dict(batch=0), dict(tokens=0), dict(batch=1 << 13, tokens=1 << 13))],
    *[(b, ESHAPE, "the norms take hidden sizes") for b in (dict(hidden=0), dict(hidden=60), dict(hidden=8200))],
    *[(dict(scale=s), EINVAL, "the residual scale must be finite") for s in (float("nan"), float("inf"), -float("inf"))],
    *[(b, EINVAL, STRIDES) for b in (dict(gate_stride=32), dict(gate_stride=66), dict(mod_stride=66),
                                     dict(mod_stride=-64))],
    *[(dict(**{k: P + 4}), EINVAL, VECTORS) for k in ("post_gain", "gate", "pre_gain", "mod_scale", "mod_shift")],
    *[(dict(**{k: None}), EINVAL, PASSED) for k in ("pre_gain", "mod_shift")],
    (dict(gate_stride=68, mod_stride=128), EINVAL, PASSED), (dict(gate_stride=0, mod_stride=0), EINVAL, PASSED)])
def test_norm_arguments(abi, bad, status, why):  # noqa: F811
    a = _norm(abi, **bad)
    given = [None if x is None else P for x in (a.post_gain, a.gate, a.pre_gain, a.mod_scale, a.mod_shift)]
    for st, said in (norm(abi, a), norm_grad(abi, a, given)):
        assert st == status and said.startswith(why), (st, said)


def test_norm_tensors(abi):  # noqa: F811
    a = _norm(abi)
    rows = "row tensors must be 16-byte aligned"
    assert norm(abi, None) == (EINVAL, NULL) and norm_grad(abi, None) == (EINVAL, NULL)
    for k in ("h", "h_out", "n_out", "r_pre", "r_post"):
        assert norm(abi, a, **{k: None}) == (EINVAL, NULL), k
    for k in ("h", "y", "h_out", "n_out"):
        assert norm(abi, a, **{k: P + 8}) == (EINVAL, rows), k
    for k in ("dn", "h_out", "r_pre", "dh", "g", "ws", "dy", "r_post"):
        assert norm_grad(abi, a, **{k: None}) == (EINVAL, NULL), k
    for k in ("dn", "dh_out", "h_out", "y", "dh", "dy", "ws"):
        assert norm_grad(abi, a, **{k: P + 8})[1].startswith("row tensors and workspace"), k
    assert norm_grad(abi, a, dh_out=None) == (EINVAL, PASSED)
    alone = "a post gain or gate needs a block output"
    for b in (_norm(abi, gate=None), _norm(abi, post_gain=None)):
        assert norm(abi, b, y=None) == (EINVAL, alone) and norm_grad(abi, b, y=None) == (EINVAL, alone)
    bare = _norm(abi, gate=None, post_gain=None)
    assert norm(abi, bare, y=None, r_post=None) == (EINVAL, PASSED)
    assert norm_grad(abi, bare, (None, None, P, P, P), y=None, dy=None, r_post=None) == (EINVAL, PASSED)


def test_norm_gradients_of_vectors_that_are_not_there(abi):  # noqa: F811
    names = ("post_gain", "gate", "pre_gain", "mod_scale", "mod_shift")
    for i, k in enumerate(names):
        a = _norm(abi, **{k: None})
        only = [P if j == i else None for j in range(5)]
        rest = [None if j == i else P for j in range(5)]
        assert norm_grad(abi, a, only) == (EINVAL, "a gradient was asked for a vector that is not there")
        assert norm_grad(abi, a, rest) == (EINVAL, PASSED)


def test_a_refusal_is_the_calling_threads(abi):  # noqa: F811
    import threading
    lib, said = abi.load_library(), []
    call(lib, "dm0_embed", T=0)
    t = threading.Thread(target=lambda: said.append(lib.dm0_last_refusal()))
    t.start()
    t.join()
    assert said == [b""] and lib.dm0_last_refusal().decode() == SIZES
    assert lib.dm0_last_error(None) == b"null context"


@pytest.mark.parametrize("bad", [dict(B=0), dict(T=0), dict(vocab=0), dict(vocab=(1 << 22) + 1), dict(hidden=4),
                                 dict(hidden=12), dict(hidden=65544)])
def test_no_workspace_for_refused_table_gradients(abi, bad):  # noqa: F811
    a = {**dict(B=2, T=3, vocab=10, hidden=64), **bad}
    assert abi.load_library().dm0_embed_grad_workspace(*a.values()) == 0


@pytest.mark.parametrize("bad", [dict(tokens=0), dict(tokens=(1 << 24) + 1), dict(vocab=0), dict(vocab=(1 << 22) + 1),
                                 dict(hidden=32), dict(hidden=96), dict(hidden=65600)])
def test_no_workspace_for_refused_losses(abi, bad):  # noqa: F811
    a = {**dict(tokens=5, vocab=100, hidden=128), **bad}
    lib = abi.load_library()
    assert lib.dm0_vocab_loss_workspace(*a.values()) == 0 and lib.dm0_vocab_loss_grad_workspace(*a.values()) == 0
