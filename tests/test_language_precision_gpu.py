"""Where the vocabulary loss could lose bits: many tiles a worker, targets that the model is sure of, long sums.

Tolerances count roundings in units of u = 2^-24, and are derived beside each case; the inputs are chosen so that the
logits are exact in fp32 where the sums behind them are what is tested."""
import math

import pytest
import torch

from tests.test_language_gpu import BF, BF16, F32, U, eng, randn, rng, unwritten_memory_is_nan, within  # noqa: F401

pytestmark = pytest.mark.gpu


def exact_logits(N, V, H=64):
    """hidden, weight and logits z[i][v] = c[i] x[v], x in sixteenths of 0..255, c in 64ths from 1 on: both fit bf16 and
    one product makes each logit, so z is exact."""
    x = torch.randint(0, 256, (V,), generator=rng(61), device="cuda") / 16
    c = 1 + (torch.arange(N, device="cuda") % 64) / 64
    h, w = torch.zeros(N, H, device="cuda", dtype=BF16), torch.zeros(V, H, device="cuda", dtype=BF16)
    h[:, 0], w[:, 0] = c, x
    assert torch.equal(h[:, 0].float(), c) and torch.equal(w[:, 0].float(), x)
    return h, w, c[:, None].double() * x[None].double()


@pytest.mark.parametrize("N, V", [(64, 1 << 20), (128, 500_000), (200, 1 << 20)])
def test_statistics_keep_their_bits_over_many_tiles(eng, N, V):  # noqa: F811
    """Up to 128 tokens a worker keeps one running (max, sum) over its tiles (2^20 entries: 56 tiles of 128 x 128 a
    worker; 200 tokens in pairs: 56 of 256)."""
    h, w, z = exact_logits(N, V)
    t = torch.arange(N, device="cuda") * 977 % V
    loss, lse = eng.vocab_loss(h, w, t)
    ref = torch.logsumexp(z, 1)
    # the sum: 32 additions in a chain of a tile, 2 to join the chains, 56 tiles, 3 workers a lane, 11 over the lanes and
    # the maximum's one (104 u); an exponential and the factor of the tile (2^-22 each: 8 u); the exponents' roundings
    # and log2 e's, u each of |z - max| log2 e, at most 20 on average over the weights, in natural units (28 u); the
    # logarithm and the sum with the maximum (u each of at most 16 and 64: 80 u)
    within(lse, ref, torch.full_like(ref, 220 * U), "lse")
    picked = z.gather(1, t[:, None])[:, 0]
    # the same with mx - z and the result rounded (u of at most 32 and 48)
    within(loss, ref - picked, torch.full_like(ref, 220 * U), "loss")


@pytest.mark.parametrize("N, V", [(5, 1000), (70, 40000), (200, 1000), (600, 999)])
def test_loss_of_a_sure_token_is_not_below_zero_nor_a_unit_of_its_logit(eng, N, V):  # noqa: F811
    """The target's logit lies 64 or more above all others: the loss is below V e^-64, whatever the logit's size."""
    H = 64
    h, w = torch.zeros(N, H, device="cuda", dtype=BF16), torch.zeros(V, H, device="cuda", dtype=BF16)
    h[:, 0] = 64 + (torch.arange(N, device="cuda") % 128) / 2
    at = V // 2 + 1
    w[at, 0] = 1 + 1 / 128
    t = torch.full((N,), at, device="cuda")
    loss, lse = eng.vocab_loss(h, w, t)
    z = h[:, 0].double() * w[at, 0].double()
    assert (loss >= 0).all()
    # the maximum's own term is an exponential near zero times the tile's factor near one: 2^-22 each, their rounding
    within(loss, torch.zeros_like(z), torch.full_like(z, 2 ** -21 + 4 * U), "loss")
    within(lse, z, 2 ** -21 + U * (z + 4), "lse")


@pytest.mark.parametrize("N, V, H", [(40, 2000, 2048), (300, 2000, 2048), (300, 1999, 1088), (24, 700, 4160)])
def test_gradient_of_sure_tokens(eng, N, V, H):  # noqa: F811
    """Tokens whose target has all but 1e-2 to 1e-5 of the probability: each one's row of dhidden against its own size.
    The reference is the definition in 64 bits; the kernels' lse takes the place of its own."""
    g = rng(62)
    w = randn(g, V, H, dtype=BF16, std=0.9 * H ** -0.5)
    t = torch.arange(N, device="cuda") * 31 % V
    wt = w[t].float()
    size = torch.linspace(13.5, 22, N, device="cuda")[:, None]
    h = (randn(g, N, H) + size * wt / wt.norm(dim=1, keepdim=True)).to(BF16)
    loss, lse = eng.vocab_loss(h, w, t)
    dh, _ = eng.vocab_loss_grad(h, w, t, lse, torch.ones(N, device="cuda"), dhidden=torch.empty(N, H, device="cuda"),
                                dweight=False)
    hd, wd = h.double(), w.double()
    z = hd @ wd.T
    p = torch.softmax(z, 1)
    rest = p.scatter(1, t[:, None], 0.0)          # the others' probabilities
    q = rest.sum(1, keepdim=True)                 # 1 - p of the target
    assert q.max() > 3e-3 and q.min() < 3e-5
    G = rest.scatter(1, t[:, None], -q)
    # a logit: products exact, 1024 / 16 additions of up to 2 u in a stretch (and 16 to spare), then the stretches in fp32
    ez = (2 * U * (64 + 16) + U * H / 512) * (hd.abs() @ wd.abs().T)
    # another entry: its logit's and the target's error against it, exp's 2^-22 and four roundings of exponents below 64
    eo = rest * (ez + ez.gather(1, t[:, None]) + 2 ** -21 + 4 * U * (z.abs() + lse.double().abs()[:, None]))
    # the target: 1 - p = 1 - exp(z - lse) takes the same relative errors, as lse is that of the same logits, and what
    # the sum that holds a term of one may lose (32 additions of a chain, 2 and 1 to join, 12 over tiles and lanes, the
    # term itself 2^-21: 55 u) and lse's rounding (u of at most 32)
    et = q * (2 * ez.amax(1, keepdim=True) + 2 ** -20) + (55 + 32) * U
    eG = eo.scatter(1, t[:, None], et)
    eG = eG + BF * (G.abs() + eG) + 2.0 ** -126
    ref = G @ wd
    bound = eG @ wd.abs() + 2 * U * (V / 16 + 64) * (G.abs() @ wd.abs())
    within(dh, ref, bound + U * (ref.abs() + bound), "dhidden")
    rel = (dh.double() - ref).norm(dim=1) / ref.norm(dim=1)
    for lo, hi in ((3e-3, 1), (1e-3, 3e-3), (1e-4, 1e-3), (1e-5, 1e-4)):
        rows = ((q >= lo) & (q < hi))[:, 0]
        print(f"  1 - p from {lo:.0e}: rows off by up to", f"{rel[rows].max().item():.1e}" if rows.any() else "-")
    # in the whole row the others' errors go in all directions: a row is off by little more than its target's entry
    lim = et[:, 0] / q[:, 0] + 2 * BF
    assert (rel <= lim).all()


@pytest.mark.parametrize("N, dt", [(1 << 17, F32), (1 << 17, BF16), (40000, F32)])
def test_weight_gradient_of_many_tokens(eng, N, dt):  # noqa: F811
    """Sums of one sign over all tokens: G is 2^-8, and 2^-8 - 1 at the target, both exact in bf16, so only the sums round."""
    V, H = 256, 64
    h = (1 + torch.rand(N, H, generator=rng(63), device="cuda")).to(BF16)
    w = torch.zeros(V, H, device="cuda", dtype=BF16)
    t = torch.zeros(N, dtype=torch.int64, device="cuda")
    lse = torch.full((N,), math.log(V), device="cuda")
    _, dw = eng.vocab_loss_grad(h, w, t, lse, torch.ones(N, device="cuda"), dhidden=False,
                                dweight=torch.empty(V, H, device="cuda", dtype=dt))
    total = h.double().sum(0)
    ref = (total / V).expand(V, H).clone()
    ref[0] -= total
    # 16384 / 16 additions of up to 2 u in a stretch (and 16 to spare), then the stretches in fp32, and the factor of one
    k = 2 * (1024 + 16) + math.ceil(N / 16384) + 1
    within(dw, ref, ref.abs() * (k * U + (BF if dt == BF16 else U) * (1 + k * U)), "dweight")
    old = torch.full((V, H), 3.0, device="cuda")
    if dt == F32:
        _, acc = eng.vocab_loss_grad(h, w, t, lse, torch.ones(N, device="cuda"), dhidden=False, dweight=old.clone(),
                                     accumulate=True)
        within(acc, ref + 3, ref.abs() * k * U + (ref + 3).abs() * 2 * U, "accumulated")


@pytest.mark.parametrize("N, V", [(1, 1 << 22), (300, 400_000)])
def test_hidden_gradient_over_a_long_vocabulary(eng, N, V):  # noqa: F811
    """Equal logits: G is 1 / V but at the target, and weights of one sign add up over the whole vocabulary."""
    H = 64
    w = (1 + torch.rand(V, H, generator=rng(64), device="cuda")).to(BF16)
    h = torch.zeros(N, H, device="cuda", dtype=BF16)
    t = torch.arange(N, device="cuda") * 7919 % V
    loss, lse = eng.vocab_loss(h, w, t)
    dh, _ = eng.vocab_loss_grad(h, w, t, lse, torch.ones(N, device="cuda"), dhidden=torch.empty(N, H, device="cuda"),
                                dweight=False)
    g = torch.tensor(1 / V).to(BF16).double().item()   # every entry's rounding to bf16 is the same; the target's is 1 - 1 / V
    others = g * (w.double().sum(0) - w[t].double())
    one = torch.tensor(1 - 1 / V).to(BF16).double().item()
    ref, mag = others - one * w[t].double(), others.abs() + one * w[t].double()
    # a stretch as above, and the splits (at most 256) and pieces (at most 2) in fp32; an exponential that is 2^-21 off
    # falls to another bf16 only where 1 / V lies that near to a border
    assert abs(abs((1 / V) / g - 1) - BF / 2) > 2 ** -19 or g * V == 1
    within(dh, ref, mag * (2 * (1024 + 16) + 256 + 2 + 4) * U, "dhidden")
