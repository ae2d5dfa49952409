"""The language operators against their definitions in 64 bits.

Tolerances count roundings (u = 2^-24 in fp32, half a step of bf16 = 2^-8), each against the sum of the magnitudes
that enter the value, so cancellation does not loosen or break them."""
import math
import types

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
BAD_INDEX = 1 << 3
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def eng():
    from vla_dual_expert_b200 import Engine, build
    build.build()
    dims = types.SimpleNamespace(layers=1, hidden_v=128, inter_v=128, hidden_a=128, inter_a=128, n_q=4, n_kv=2,
                                 head_dim=32, chunk=4, action_dim=8, rope_theta=1e6, rms_eps=1e-6)
    e = Engine(dims, 1, 16)
    yield e
    e.sync()
    e.close()


@pytest.fixture(autouse=True)
def unwritten_memory_is_nan():
    """Fills what torch's allocator will hand out next with NaN, so that a value that a kernel left out shows."""
    held = [torch.full((n,), float("nan"), device="cuda") for n in [2 ** k for k in range(7, 18)] * 24 + [2 ** 22] * 8
            + [2 ** 26] * 2]
    torch.cuda.synchronize()
    del held
    yield


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def ids_of(g, shape, vocab, dtype=torch.int64, missing=0.2):
    v = (vocab * torch.rand(shape, generator=g, device="cuda", dtype=torch.float64) ** 3).long().clamp(max=vocab - 1)
    return torch.where(torch.rand(shape, generator=g, device="cuda") < missing, -1, v).to(dtype)


def within(got, ref, bound, what):
    """Every element: |got - ref| <= bound (64 bits); infinities and NaN nowhere."""
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), what
    d = (got - ref).abs()
    worst = (d / bound.clamp(min=1e-300)).max().item() if d.numel() else 0.0
    print(f"  {what}: {worst:.3f} of the bound")
    assert (d <= bound).all(), (what, worst)


def out_step(dtype):
    return BF if dtype == BF16 else U


# ------------------------------------------------------------------------------------------------ embedding
@pytest.mark.parametrize("B, T, V, H", [(1, 1, 1, 8), (1, 1, 1000, 2048), (3, 5, 17, 264), (2, 48, 3001, 1024),
                                        (4, 33, 50, 2056), (1, 3000, 777, 128)])
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("idt", [torch.int64, torch.int32])
def test_embed(eng, B, T, V, H, out, idt):
    g = rng(1)
    table, ids = randn(g, V, H, dtype=BF16, std=0.02), ids_of(g, (B, T), V, idt)
    scale = math.sqrt(H)
    prefix = torch.full((B, T + 3, H), 7.0, device="cuda", dtype=out)
    got = eng.embed(table, ids, scale, out=prefix[:, 2:2 + T])
    ref = table[ids.long().clamp(min=0)].float() * scale      # one fp32 product, rounded once
    ref = torch.where((ids >= 0)[..., None], ref, 0.0).to(out)
    assert torch.equal(got, ref)
    assert (prefix[:, :2] == 7).all() and (prefix[:, 2 + T:] == 7).all()
    if out == BF16:
        assert torch.equal(eng.embed(table, ids[0], scale), ref[0])


def test_embed_interleaved_rows_and_odd_scales(eng):
    g = rng(2)
    table, ids = randn(g, 11, 64, dtype=BF16), ids_of(g, (3, 4), 11)
    out = torch.empty(4, 3, 64, device="cuda", dtype=BF16)
    eng.embed(table, ids, 1.0, out=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), torch.where((ids >= 0)[..., None], table[ids.clamp(min=0)], 0.0))
    got = eng.embed(table, torch.tensor([-1, -5, -2 ** 40], device="cuda"), float("nan"))
    assert (got == 0).all() and not torch.signbit(got).any()   # a missing token's row is zero whatever the scale
    assert (eng.embed(table, torch.tensor([3], device="cuda"), 0.0) == 0).all()


def emb_grad_ref(ids, dout, V, scale):
    flat, rows = ids.long().reshape(-1), dout.reshape(-1, dout.shape[-1]).double() * scale
    held = flat >= 0
    ref = torch.zeros(V, dout.shape[-1], device="cuda", dtype=torch.float64)
    mag, cnt = ref.clone(), torch.zeros(V, device="cuda", dtype=torch.float64)
    ref.index_add_(0, flat[held], rows[held])
    mag.index_add_(0, flat[held], rows[held].abs())
    cnt.index_add_(0, flat[held], torch.ones_like(flat[held], dtype=torch.float64))
    return ref, mag, cnt


@pytest.mark.parametrize("B, T, V, H", [(1, 1, 1, 8), (1, 1, 131072, 64), (3, 5, 17, 264), (2, 48, 3001, 1024),
                                        (4, 333, 50, 2056), (1, 64, 3, 64), (1, 65, 1, 64), (1, 128, 2, 72),
                                        (2, 4000, 5003, 128), (1, 9000, 1, 256), (1, 700, 300000, 64)])
@pytest.mark.parametrize("dt, idt", [(F32, torch.int64), (BF16, torch.int32)])
def test_embed_grad(eng, B, T, V, H, dt, idt):
    g = rng(3)
    ids = ids_of(g, (B, T), V, idt)
    dout = randn(g, B, T + 2, H, dtype=dt)[:, 1:T + 1]
    scale = 1.7
    ref, mag, cnt = emb_grad_ref(ids, dout, V, 1.7)
    # additions in fp32 in some order, the scale's rounding, its product, the accumulation
    bound = (cnt[:, None] + 3) * U * mag
    got = eng.embed_grad(ids, dout, V, scale)
    within(got, ref, bound, "embed_grad")
    assert (got[cnt == 0] == 0).all()
    assert torch.equal(got, eng.embed_grad(ids, dout, V, scale))   # the same bits again
    old = randn(g, V, H)
    acc = eng.embed_grad(ids, dout, V, scale, grad=old.clone(), accumulate=True)
    within(acc, old.double() + ref, bound + U * (old.double().abs() + mag), "embed_grad accumulate")
    assert torch.equal(acc[cnt == 0], old[cnt == 0])


def test_embed_grad_without_any_token(eng):
    ids = torch.full((2, 70), -1, device="cuda")
    dout = torch.full((2, 70, 64), float("nan"), device="cuda")   # rows without a token are not read into it
    assert (eng.embed_grad(ids, dout, 9) == 0).all()
    one = torch.ones(9, 64, device="cuda")
    assert (eng.embed_grad(ids, dout, 9, grad=one, accumulate=True) == 1).all()


def test_embed_adjoint(eng):
    """<embed(E), D> = <E, embed_grad(D)> : the gradient is the transpose of the lookup."""
    g = rng(4)
    table, ids = randn(g, 301, 128, dtype=BF16), ids_of(g, (3, 200), 301)
    d = randn(g, 3, 200, 128)
    out = torch.empty(3, 200, 128, device="cuda")
    eng.embed(table, ids, 0.5, out=out)
    grad = eng.embed_grad(ids, d, 301, 0.5)
    a, b = (out.double() * d.double()), (table.double() * grad.double())
    # per product: the lookup's rounding; per table entry: its additions (at most 600) and two products
    assert abs(a.sum() - b.sum()) <= 605 * U * (a.abs().sum() + (table.double().abs() * emb_grad_ref(ids, d.abs(), 301, 0.5)[0]).sum())


def test_bad_ids_are_reported_and_count_as_none(eng):
    g = rng(5)
    V, H = 40, 64
    table, d = randn(g, V, H, dtype=BF16), randn(g, 4, H)
    ids = torch.tensor([3, V, 2 ** 40, 39], device="cuda")
    ok = torch.tensor([3, -1, -1, 39], device="cuda")
    h, w = randn(g, 4, H, dtype=BF16), table
    good = eng.embed(table, ok), eng.embed_grad(ok, d, V), *eng.vocab_loss(h, w, ok)
    ones = torch.ones(4, device="cuda")
    good += eng.vocab_loss_grad(h, w, ok, good[3], ones)
    eng.sync()
    calls = [lambda: [eng.embed(table, ids)], lambda: [eng.embed_grad(ids, d, V)], lambda: eng.vocab_loss(h, w, ids),
             lambda: eng.vocab_loss_grad(h, w, ids, good[3], ones)]
    from vla_dual_expert_b200 import Dm0Error
    i = 0
    for call in calls:
        got = call()
        with pytest.raises(Dm0Error):
            eng.sync()
        assert eng.device_error() == BAD_INDEX
        eng.clear_error()
        for t in got:
            assert torch.equal(t, good[i])
            i += 1
    eng.sync()


# ------------------------------------------------------------------------------------------- residual norms
def norm_case(g, B, T, H, hd, yd, post, gate, mod, pre, y=True):
    return dict(h=randn(g, B, T, H, dtype=hd, std=2.0), y=randn(g, B, T, H, dtype=yd, std=0.7) if y else None,
                post_gain=1 + randn(g, H, std=0.2) if post else None, pre_gain=1 + randn(g, H, std=0.2) if pre else None,
                gate={"none": None, "shared": randn(g, H), "sample": randn(g, B, H)}[gate],
                mod_scale={"none": None, "shared": randn(g, H, std=0.3), "sample": randn(g, B, H, std=0.3)}[mod],
                mod_shift={"none": None, "shared": randn(g, H, std=0.3), "sample": randn(g, B, H, std=0.3)}[mod])


def rows(v):
    return v if v is None or v.dim() == 1 else v[:, None]


def norm_ref(c, scale, eps=1e-6):
    """(values, error bounds) of the forward pass in 64 bits.  A row's 1/rms is off by at most 64 u: up to 8 squares
    per piece and 8 pieces added in a row, five exchanges and up to 4 partial sums, mean and eps, halved by the root
    (42 u), and rsqrtf (2 steps = 4 u), rounded up; a product by u."""
    d = {k: v.double() if v is not None else None for k, v in c.items()}
    out = {}
    u = torch.zeros_like(d["h"]) if d["y"] is None else d["y"]
    if d["post_gain"] is not None:
        out["r_post"] = (u.square().mean(-1) + eps).rsqrt()
        u = u * out["r_post"][..., None] * d["post_gain"]
    if d["gate"] is not None:
        u = u * rows(d["gate"])
    h = scale * d["h"] + u
    eh = 70 * U * u.abs() + 3 * U * (scale * d["h"]).abs()
    out["h"] = h
    out["r_pre"] = r = (h.square().mean(-1) + eps).rsqrt()
    er = 64 * U + (h.abs() * eh).mean(-1) * r * r   # relative, with what h's error does to the mean
    a = torch.ones_like(h)
    if d["pre_gain"] is not None:
        a = a * d["pre_gain"]
    if d["mod_scale"] is not None:
        a = a * (1 + rows(d["mod_scale"]))
    n = h * r[..., None] * a
    en = n.abs() * (er[..., None] + 6 * U) + eh * r[..., None] * a.abs()
    if d["mod_shift"] is not None:
        n = n + rows(d["mod_shift"])
        en = en + U * n.abs()
    out["n"] = n
    bound = {"h": eh + out_step(c["h"].dtype) * (h.abs() + eh), "n": en + BF * (n.abs() + en), "r_pre": er * r}
    if "r_post" in out:
        bound["r_post"] = 64 * U * out["r_post"]
    return out, bound


NORMS = [  # B, T, H, h, y, post, gate, mod, pre, scale
    (1, 1, 8, F32, BF16, True, "none", "none", True, 1.0),
    (1, 50, 1024, F32, BF16, False, "sample", "sample", False, 1.0),
    (3, 7, 264, BF16, F32, True, "sample", "shared", True, 0.5),
    (2, 33, 2048, F32, BF16, True, "shared", "none", True, 1.0),
    (2, 5, 2056, BF16, BF16, True, "none", "sample", True, -1.5),
    (5, 3, 4096, F32, F32, True, "sample", "sample", True, 1.0),
    (1, 6, 8192, BF16, BF16, True, "shared", "shared", False, 1.0),
    (16, 1, 512, F32, F32, False, "none", "none", False, 0.0),
    (1, 700, 128, F32, BF16, True, "shared", "none", True, 1.0),
    (7, 101, 136, BF16, F32, False, "sample", "sample", True, 1.0)]


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_residual_norm(eng, case):
    B, T, H, hd, yd, post, gate, mod, pre, scale = case
    c = norm_case(rng(6), B, T, H, hd, yd, post, gate, mod, pre)
    ref, bound = norm_ref(c, scale)
    kw = {k: v for k, v in c.items() if k not in ("h", "y")}
    h, n, r_post, r_pre = eng.residual_norm(c["h"], c["y"], scale=scale, **kw)
    assert h.dtype == hd and n.dtype == BF16
    for name, got in (("h", h), ("n", n), ("r_pre", r_pre), ("r_post", r_post)):
        if got is not None:
            within(got, ref[name], bound[name], name)
    assert (r_post is None) == (not post)
    same = c["h"].clone()   # in place
    h2, n2, _, _ = eng.residual_norm(same, c["y"], scale=scale, h_out=same, **kw)
    assert torch.equal(h2, h) and torch.equal(n2, n)


def test_residual_norm_without_a_block(eng):
    c = norm_case(rng(7), 2, 9, 256, F32, F32, False, "none", "sample", True, y=False)
    ref, bound = norm_ref(c, 1.0)
    kw = {k: v for k, v in c.items() if k not in ("h", "y")}
    h, n, _, r = eng.residual_norm(c["h"], **kw)
    assert torch.equal(h, c["h"])
    within(n, ref["n"], bound["n"], "n")
    got = eng.residual_norm_grad(n, None, h, None, None, r, **kw)
    assert set(got) == {"h", "pre_gain", "mod_scale", "mod_shift"}
    check_norm_grad(c, 1.0, n, None, h, None, r, got)


def test_residual_norm_zero_rows_stay_finite(eng):
    h, y = torch.zeros(1, 3, 128, device="cuda"), torch.zeros(1, 3, 128, device="cuda")
    g = torch.ones(128, device="cuda")
    ho, n, rp, rr = eng.residual_norm(h, y, post_gain=g, pre_gain=g)
    assert (ho == 0).all() and (n == 0).all() and torch.isfinite(rp).all() and torch.isfinite(rr).all()
    got = eng.residual_norm_grad(torch.ones_like(h), None, ho, y, rp, rr, post_gain=g, pre_gain=g)
    assert all(torch.isfinite(v).all() for v in got.values())


def test_a_row_with_nan_spoils_no_other(eng):
    c = norm_case(rng(8), 1, 20, 1024, F32, BF16, True, "shared", "none", True)
    kw = {k: v for k, v in c.items() if k not in ("h", "y")}
    h, n, _, _ = eng.residual_norm(c["h"], c["y"], **kw)
    bad = c["h"].clone()
    bad[0, 4, 17], bad[0, 11, 3] = float("nan"), float("inf")
    h2, n2, _, _ = eng.residual_norm(bad, c["y"], **kw)
    keep = [i for i in range(20) if i not in (4, 11)]
    assert torch.equal(h[:, keep], h2[:, keep]) and torch.equal(n[:, keep], n2[:, keep])
    assert n2[0, 4].isnan().all()


def check_norm_grad(c, scale, dn, dh_out, h_out, r_post, r_pre, got):
    """The adjoint's formula in 64 bits on the same inputs.  Means over a row are sums of at most 32 + 8 + 5 fp32
    additions (128 u with the products in front, rounded up), each bounded by the mean of magnitudes; sums over rows
    add at most `rows` more."""
    d = {k: v.double() if v is not None else None for k, v in c.items()}
    B, T, H = h_out.shape
    one = torch.ones(H, device="cuda", dtype=torch.float64)
    k = 128 * U
    r = r_pre.double()[..., None]
    x, n = h_out.double() * r, dn.double()
    gp = one if d["pre_gain"] is None else d["pre_gain"]
    ms = one if d["mod_scale"] is None else 1 + rows(d["mod_scale"])
    a = gp * ms
    dho = torch.zeros_like(x) if dh_out is None else dh_out.double()
    m1 = (a * n * x).mean(-1, keepdim=True)
    dH = dho + r * (a * n - x * m1)
    S = dho.abs() + r * ((a * n).abs() + x.abs() * (a * n * x).abs().mean(-1, keepdim=True))   # magnitudes in dH
    eps = lambda t: out_step(t.dtype)
    within(got["h"], scale * dH, abs(scale) * S * k + eps(got["h"]) * (scale * dH).abs() * (1 + 1e-3), "dh")
    total = lambda v, per: v.sum(1) if per else v.sum((0, 1))
    per = lambda v: v is not None and v.dim() == 2
    R = B * T
    def check_sum(name, terms, mags):
        p = per(c[name])
        ref, mag = total(terms, p), total(mags, p)
        within(got[name], ref.reshape(got[name].shape), ((R + 200) * U * mag).reshape(got[name].shape), name)
    if d["pre_gain"] is not None:
        check_sum("pre_gain", n * x * ms, (n * x * ms).abs() + (n * x).abs())
    if d["mod_scale"] is not None:
        check_sum("mod_scale", n * x * gp, (n * x * gp).abs())
    if d["mod_shift"] is not None:
        check_sum("mod_shift", n, n.abs())
    if c["y"] is None:
        return
    rp = torch.ones_like(r) if r_post is None else r_post.double()[..., None]
    z = d["y"] * rp
    gq = one if d["post_gain"] is None else d["post_gain"]
    gt = one if d["gate"] is None else rows(d["gate"])
    w = gq * gt
    if d["post_gain"] is None:
        dy, mag = w * dH, (w * S).abs()
    else:
        dy = rp * (w * dH - z * (w * dH * z).mean(-1, keepdim=True))
        # the mean is taken as (sum of w z (dho + r a n)) - m1 (sum of w z x)
        mean = (w * z).abs() * S
        mag = rp * ((w * S).abs() + z.abs() * (mean.mean(-1, keepdim=True) + r * (a * n * x).abs().mean(-1, keepdim=True) * (w * z * x).abs().mean(-1, keepdim=True)))
    within(got["y"], dy, 3 * k * mag + eps(got["y"]) * (dy.abs() + 3 * k * mag), "dy")
    if d["gate"] is not None:
        check_sum("gate", dH * z * gq, (S * z * gq).abs() * (1 + 128 / (R + 200)))
    if d["post_gain"] is not None:
        check_sum("post_gain", dH * z * gt, (S * z * gt).abs() * (1 + 128 / (R + 200)))


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
@pytest.mark.parametrize("dnt, up", [(BF16, True), (F32, False)])
def test_residual_norm_grad(eng, case, dnt, up):
    B, T, H, hd, yd, post, gate, mod, pre, scale = case
    g = rng(9)
    c = norm_case(g, B, T, H, hd, yd, post, gate, mod, pre)
    kw = {k: v for k, v in c.items() if k not in ("h", "y")}
    h, n, r_post, r_pre = eng.residual_norm(c["h"], c["y"], scale=scale, **kw)
    dn, dho = randn(g, B, T, H, dtype=dnt), randn(g, B, T, H, dtype=hd) if up else None
    got = eng.residual_norm_grad(dn, dho, h, c["y"], r_post, r_pre, scale=scale, **kw)
    check_norm_grad(c, scale, dn, dho, h, r_post, r_pre, got)
    for name in kw:
        assert (name in got) == (kw[name] is not None)
        if name in got:
            assert got[name].shape == kw[name].shape and got[name].dtype == F32
    again = eng.residual_norm_grad(dn, dho, h, c["y"], r_post, r_pre, scale=scale, **kw)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_residual_norm_grad_against_differences(eng):
    """Directional differences of the 64-bit definition: d/dt <n, dn> + <h', dh'> along a random direction of every input."""
    g = rng(10)
    B, T, H, scale = 2, 6, 64, 0.7
    c = norm_case(g, B, T, H, F32, F32, True, "sample", "sample", True)
    kw = {k: v for k, v in c.items() if k not in ("h", "y")}
    h, n, r_post, r_pre = eng.residual_norm(c["h"], c["y"], scale=scale, **kw)
    dn, dho = randn(g, B, T, H), randn(g, B, T, H)
    got = eng.residual_norm_grad(dn, dho, h, c["y"], r_post, r_pre, scale=scale, **kw)
    step = 1e-5
    for name, v in c.items():
        e = torch.randn(v.shape, generator=g, device="cuda", dtype=torch.float64)
        vals = []
        for s in (step, -step):
            moved = {**{k: x.double() for k, x in c.items()}, name: v.double() + s * e}
            ref, _ = norm_ref(moved, scale)
            vals.append((ref["n"] * dn.double()).sum() + (ref["h"] * dho.double()).sum())
        diff = (vals[0] - vals[1]) / (2 * step)
        mine = (got[name].double() * e).sum()
        # central differences: step^2 of third-order terms (values of order 1 over B T H of them), 2^-52 / step of
        # cancellation; the kernel's fp32 roundings
        mag = (got[name].double() * e).abs().sum() + 1
        assert abs(diff - mine) <= 1e-4 * mag, (name, diff.item(), mine.item())


# ------------------------------------------------------------------------------------------ vocabulary loss
def loss_case(g, N, V, H, idt=torch.int64, missing=0.2):
    w = randn(g, V, H, dtype=BF16, std=H ** -0.5)
    t = ids_of(g, (N,), V, idt, missing)
    h = randn(g, N, H) + 3 * torch.rand(N, 1, generator=g, device="cuda") * w[t.long().clamp(min=0)].float()
    return h.to(BF16), w, t


def logits_ref(h, w):
    """Logits in 64 bits and their error bound: products of bf16 are exact in fp32, sixteen are added at a time into
    an fp32 accumulator that may truncate (2 u a step)."""
    hd, wd = h.double(), w.double()
    return hd @ wd.T, 2 * U * (h.shape[1] / 16 + 16) * (hd.abs() @ wd.abs().T)


LOSSES = [(1, 1, 64), (1, 17, 128), (7, 1000, 320), (127, 255, 64), (128, 256, 128), (129, 257, 1088), (300, 5003, 192),
          (2, 40000, 256), (513, 999, 2048), (20, 300, 4160), (140, 300, 4160)]


@pytest.mark.parametrize("N, V, H", LOSSES)
@pytest.mark.parametrize("idt", [torch.int64, torch.int32])
def test_vocab_loss(eng, N, V, H, idt):
    h, w, t = loss_case(rng(11), N, V, H, idt)
    loss, lse = eng.vocab_loss(h, w, t)
    z, ez = logits_ref(h, w)
    ref = torch.logsumexp(z, 1)
    # exp: 2^-22 and its argument's rounding (|z| log2 e, twice); sums of V terms in groups; the logarithm
    e = ez.amax(1) + 2 ** -21 + 4 * U * z.abs().amax(1) + (256 + V / 256) * U + 4 * U * ref.abs()
    within(lse, ref, e, "lse")
    picked = z.gather(1, t.long().clamp(min=0)[:, None])[:, 0]
    within(loss, torch.where(t >= 0, ref - picked, 0.0), torch.where(t >= 0, 2 * e + U * picked.abs(), 0.0), "loss")
    again = eng.vocab_loss(h, w, t)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


def check_loss_grad(h, w, t, lse, dl, dh, dw, old=None):
    z, ez = logits_ref(h, w)
    N, V = z.shape
    H = h.shape[1]
    held = (t >= 0) & (t < V)
    dlr = torch.where(held, dl.double(), 0.0)[:, None]
    p = torch.exp(z - lse.double()[:, None])
    one = torch.zeros_like(z)
    one[held, t.long()[held]] = 1
    G = (p - one) * dlr
    # an entry: the exponent's error, exp's 2^-22, two fp32 roundings and the one to bf16; a probability below the
    # smallest normal number counts as zero, which is at most 2^-126 off (at logits 64 * 64 away, half of them are:
    # a bound relative to them alone would ask for subnormal results)
    eG = (p * (ez + 2 ** -21 + 4 * U * (z.abs() + lse.double().abs()[:, None])) + 4 * U * (p + one) + 2.0 ** -126) * dlr.abs()
    eG = eG + BF * (G.abs() + eG)
    for name, got, k, ref, mag, err in (
            ("dhidden", dh, V, G @ w.double(), G.abs() @ w.double().abs(), eG @ w.double().abs()),
            ("dweight", dw, N, G.T @ h.double(), G.T.abs() @ h.double().abs(), eG.T @ h.double().abs())):
        if got is None:
            continue
        if name == "dweight" and old is not None:
            ref = ref + old.double()
            mag = mag + old.double().abs()
        b = err + 2 * U * (k / 16 + 64) * (mag + err)
        within(got, ref, b + out_step(got.dtype) * (ref.abs() + b), name)
        norm = ref.norm()
        if norm > 0 and k > 1:   # roundings of both steps are independent: together below two half steps
            rel = ((got.double() - ref).norm() / norm).item()
            print(f"  {name}: relative {rel:.2e}")
            assert rel <= 2 * BF


@pytest.mark.parametrize("N, V, H", LOSSES)
@pytest.mark.parametrize("dt", [F32, BF16])
def test_vocab_loss_grad(eng, N, V, H, dt):
    g = rng(12)
    h, w, t = loss_case(g, N, V, H)
    _, lse = eng.vocab_loss(h, w, t)
    dl = torch.rand(N, generator=g, device="cuda") / N
    dh, dw = eng.vocab_loss_grad(h, w, t, lse, dl, dhidden=torch.empty(N, H, device="cuda", dtype=dt),
                                 dweight=torch.empty(V, H, device="cuda", dtype=dt))
    check_loss_grad(h, w, t, lse, dl, dh, dw)
    assert (dh[t < 0] == 0).all()
    again = eng.vocab_loss_grad(h, w, t, lse, dl, dhidden=torch.empty_like(dh), dweight=torch.empty_like(dw))
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)
    only_h, none = eng.vocab_loss_grad(h, w, t, lse, dl, dhidden=torch.empty_like(dh), dweight=False)
    assert none is None and torch.equal(only_h, dh)
    none, only_w = eng.vocab_loss_grad(h, w, t, lse, dl, dhidden=False, dweight=torch.empty_like(dw))
    assert none is None and torch.equal(only_w, dw)


@pytest.mark.parametrize("N, V, H", [(2100, 70001, 64), (1, 300, 64), (40, 20000, 128)])
def test_vocab_loss_grad_pieces_and_accumulation(eng, N, V, H):
    """The first size takes two pieces of the vocabulary."""
    g = rng(13)
    h, w, t = loss_case(g, N, V, H)
    loss, lse = eng.vocab_loss(h, w, t)
    dl = torch.full((N,), 1 / 3, device="cuda")
    old = randn(g, V, H, std=0.1)
    dh, dw = eng.vocab_loss_grad(h, w, t, lse, dl, dweight=old.clone(), accumulate=True)
    check_loss_grad(h, w, t, lse, dl, dh, dw, old)


def test_vocab_loss_mean_is_not_rounded_into_the_gradient(eng):
    """A constant dloss takes no part in the rounding to bf16: the gradients of 1 and of 1/3 are proportional."""
    h, w, t = loss_case(rng(14), 200, 999, 128)
    _, lse = eng.vocab_loss(h, w, t)
    kw = lambda: dict(dhidden=torch.empty(200, 128, device="cuda"), dweight=torch.empty(999, 128, device="cuda"))
    one = eng.vocab_loss_grad(h, w, t, lse, torch.ones(200, device="cuda"), **kw())
    third = eng.vocab_loss_grad(h, w, t, lse, torch.full((200,), 1 / 3, device="cuda"), **kw())
    for a, b in zip(one, third):
        within(b, a.double() * torch.tensor(1 / 3, device="cuda").double(), U * b.double().abs() * 1.01 + 1e-40, "third")


def test_vocab_loss_rows_without_a_target(eng):
    h, w, t = loss_case(rng(15), 150, 700, 128, missing=0.0)
    t[:] = -1
    loss, lse = eng.vocab_loss(h, w, t)
    assert (loss == 0).all() and torch.isfinite(lse).all()
    dl = torch.full((150,), float("nan"), device="cuda")   # not read where there is no target
    dh, dw = eng.vocab_loss_grad(h, w, t, lse, dl)
    assert (dh == 0).all() and (dw == 0).all()
    t[3] = 5
    dl[3] = 0.0
    dh, dw = eng.vocab_loss_grad(h, w, t, lse, dl)
    assert (dh == 0).all() and (dw == 0).all()


def test_vocab_loss_grad_keeps_infinities_in_their_rows(eng):
    """A weight of infinity or NaN on one token reaches that token's dhidden and no other's."""
    h, w, t = loss_case(rng(17), 40, 300, 64, missing=0.0)
    _, lse = eng.vocab_loss(h, w, t)
    dl = torch.full((40,), 0.3, device="cuda")
    want, _ = eng.vocab_loss_grad(h, w, t, lse, dl)
    dl[7], dl[21] = float("inf"), float("nan")
    got, dw = eng.vocab_loss_grad(h, w, t, lse, dl)
    keep = [i for i in range(40) if i not in (7, 21)]
    assert torch.equal(got[keep], want[keep])
    assert not torch.isfinite(got[7]).any() and got[21].isnan().all() and dw.isnan().all()


def test_vocab_loss_extreme_logits(eng):
    """Logits of +-1000s: the maximum is taken out before the exponentials."""
    N, V, H = 130, 600, 64
    h = torch.zeros(N, H, device="cuda", dtype=BF16)
    w = torch.zeros(V, H, device="cuda", dtype=BF16)
    h[:, 0] = 64
    w[:, 0] = torch.linspace(-64, 64, V, device="cuda")
    t = (torch.arange(N, device="cuda") * 4) % V
    loss, lse = eng.vocab_loss(h, w, t)
    z = h.double() @ w.double().T
    ref = torch.logsumexp(z, 1)
    within(lse, ref, 8 * U * z.abs().amax(1) + 2 ** -20, "lse")
    within(loss, ref - z.gather(1, t[:, None])[:, 0], 16 * U * z.abs().amax(1) + 2 ** -20, "loss")
    dh, dw = eng.vocab_loss_grad(h, w, t, lse, torch.ones(N, device="cuda"))
    check_loss_grad(h, w, t, lse, torch.ones(N, device="cuda"), dh, dw)


def test_vocab_loss_grad_against_differences(eng):
    g = rng(16)
    N, V, H = 20, 90, 64
    h, w, t = loss_case(g, N, V, H)
    _, lse = eng.vocab_loss(h, w, t)
    dl = torch.rand(N, generator=g, device="cuda")
    dh, dw = eng.vocab_loss_grad(h, w, t, lse, dl, dhidden=torch.empty(N, H, device="cuda"), dweight=torch.empty(V, H, device="cuda"))

    def f(hd, wd):
        z = hd @ wd.T
        per = torch.logsumexp(z, 1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0]
        return (torch.where(t >= 0, per, 0.0) * dl.double()).sum()
    s = 1e-5
    eh, ew = (torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64) for x in (h, w))
    H0, W0 = h.double(), w.double()
    for got, e, diff in ((dh, eh, f(H0 + s * eh, W0) - f(H0 - s * eh, W0)), (dw, ew, f(H0, W0 + s * ew) - f(H0, W0 - s * ew))):
        mag = (got.double() * e).abs().sum()
        assert abs(diff / (2 * s) - (got.double() * e).sum()) <= 2 * BF * mag   # G's rounding to bf16
