"""The language operators as they are used together: from token ids through the boundary norms to the loss and
back to the tied table, in graphs, on streams, at large offsets, and in front of the prefix pass."""
import math

import numpy as np
import pytest
import torch

from synth import inputs as I
from tests.test_language_gpu import (BF, BF16, F32, eng, ids_of, loss_case, norm_case, randn, rng,  # noqa: F401
                                     unwritten_memory_is_nan)

pytestmark = pytest.mark.gpu


class Step:
    """Tokens -> embedding -> boundary behind a block -> final norm's output -> loss, and all gradients back, with the
    loss's weights and the embedding table one tensor."""

    def __init__(self, eng, seed, B=3, T=37, V=501, H=192):  # noqa: F811
        g = rng(seed)
        self.eng, self.scale, self.H, self.V = eng, math.sqrt(H), H, V
        self.table = randn(g, V, H, dtype=BF16, std=0.05)
        self.ids, self.targets = ids_of(g, (B, T), V), ids_of(g, (B * T,), V)
        self.block = randn(g, B, T, H, dtype=BF16)           # the output of the block between
        self.post, self.gate, self.pre = 1 + randn(g, H, std=0.1), randn(g, B, H), 1 + randn(g, H, std=0.1)
        self.dloss = torch.full((B * T,), 1.0 / (B * T), device="cuda")

    def run(self, stream=None):
        e, kw = self.eng, dict(post_gain=self.post, gate=self.gate, pre_gain=self.pre, scale=0.7, stream=stream)
        x = e.embed(self.table, self.ids, self.scale, stream=stream)
        h, n, r_post, r_pre = e.residual_norm(x, self.block, **kw)
        flat = n.view(-1, self.H)
        loss, lse = e.vocab_loss(flat, self.table, self.targets, stream=stream)
        dtable = torch.empty(self.V, self.H, device="cuda")
        dn, _ = e.vocab_loss_grad(flat, self.table, self.targets, lse, self.dloss, dweight=dtable, stream=stream)
        out = e.residual_norm_grad(dn.view_as(n), None, h, self.block, r_post, r_pre, **kw)
        e.embed_grad(self.ids, out.pop("h"), self.V, self.scale, grad=dtable, accumulate=True, stream=stream)
        return {"loss": loss, "table": dtable, **out}

    def reference(self):
        """The same in 64 bits with automatic differentiation, without any rounding between."""
        leaf = {k: getattr(self, k).double().requires_grad_() for k in ("table", "block", "post", "gate", "pre")}
        ids = self.ids
        x = torch.where((ids >= 0)[..., None], leaf["table"][ids.clamp(min=0)], 0.0) * self.scale
        norm = lambda v: v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        h = 0.7 * x + leaf["gate"][:, None] * norm(leaf["block"]) * leaf["post"]
        z = (norm(h) * leaf["pre"]).view(-1, self.H) @ leaf["table"].T
        t = self.targets
        loss = torch.where(t >= 0, torch.logsumexp(z, 1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
        got = torch.autograd.grad((loss * self.dloss.double()).sum(), list(leaf.values()))
        names = dict(table="table", block="y", post="post_gain", gate="gate", pre="pre_gain")
        return {"loss": loss.detach(), **{names[k]: v for k, v in zip(leaf, got)}}


def test_training_step_of_a_tied_table(eng):  # noqa: F811
    s = Step(eng, 21)
    got, ref = s.run(), s.reference()
    assert set(got) == set(ref)
    for k, v in ref.items():
        rel = ((got[k].double() - v).norm() / v.norm()).item()
        print(f"  {k}: {rel:.2e}")
        # five roundings to bf16 lie on the way (embedded rows, h, n, G, dn), each at most half a step, 2^-8, of its value
        # and the values' parts add with independent signs; h passes through a norm that can double a change
        assert rel <= 6 * BF, (k, rel)


def test_captured_steps_replay_and_do_not_share_scratch(eng):  # noqa: F811
    """Two captured steps, replayed in turn and at the same time on two streams, after their inputs changed."""
    a, b = Step(eng, 22), Step(eng, 23, B=2, T=80, V=3003, H=64)
    want = []
    graphs, outs = [], []
    for s in (a, b):
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):   # the capturing stream named once, once not
            outs.append(s.run(stream=torch.cuda.current_stream() if s is a else None))
        graphs.append(g)
    for s in (a, b):    # new inputs in the captured tensors
        s.ids.copy_(torch.where(s.ids < 0, 1, s.ids.flip(-1)))
        s.block.mul_(0.5)
        s.dloss.mul_(3)
        want.append(s.run())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for o in outs:
            for v in o.values():
                v.fill_(float("nan"))
        torch.cuda.synchronize()
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(o[k], w[k]) for k in w)
    eng.sync()
    del graphs


def test_a_stream_of_their_own(eng):  # noqa: F811
    s = Step(eng, 24)
    want = s.run()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for handle in (st, st.cuda_stream):
        st.wait_stream(torch.cuda.current_stream())
        got = s.run(stream=handle)
        st.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)


def test_two_contexts_on_two_threads(eng):  # noqa: F811
    """A context is not thread-safe, two contexts are independent: calls overlap on the host and on the GPU."""
    import concurrent.futures
    from vla_dual_expert_b200 import Engine
    other = Engine(eng.dims, 1, 16)
    try:
        steps = [Step(eng, 33), Step(other, 34, B=1, T=300, V=2000, H=128)]
        want = [s.run() for s in steps]
        torch.cuda.synchronize()

        def work(k):
            with torch.cuda.stream(torch.cuda.Stream()):
                got = [steps[k].run() for _ in range(10)]
                torch.cuda.current_stream().synchronize()
            return all(torch.equal(g[n], want[k][n]) for g in got for n in g)
        with concurrent.futures.ThreadPoolExecutor(2) as pool:
            assert all(pool.map(work, (0, 1)))
        other.sync()
    finally:
        other.close()


def test_launches_are_counted(eng):  # noqa: F811
    s = Step(eng, 25)
    n = eng.launch_count()
    s.run()
    # embed 1, norm 1, loss 2, gradient 3 (one piece), norm gradient 2, table gradient 1 (3 above 256 tokens)
    assert eng.launch_count() - n == 10


def test_long_lists_of_frequent_ids(eng):  # noqa: F811
    """Segments of thousands of places next to short ones, at every alignment to the tiles."""
    g = rng(26)
    for lens in ([33, 1, 32, 31, 64, 65], [1, 5000, 1], [32] * 40, [63, 33] * 9, [7000]):
        ids = torch.cat([torch.full((n,), i * 128 + (i % 3)) for i, n in enumerate(lens)])
        ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))].cuda()
        d = randn(g, len(ids), 72)
        V = 128 * len(lens) + 3
        got = eng.embed_grad(ids, d, V, 1.0)
        ref = torch.zeros(V, 72, device="cuda", dtype=torch.float64).index_add_(0, ids, d.double())
        mag = torch.zeros_like(ref).index_add_(0, ids, d.double().abs())
        assert ((got.double() - ref).abs() <= (max(lens) + 3) * 2.0 ** -24 * mag).all()


def test_more_ids_than_one_round_of_the_sort(eng):  # noqa: F811
    g = rng(27)
    for n, V, same in ((40000, 1000, 0), (70001, 200001, 0), (50000, 300, 40000)):
        ids = ids_of(g, (n,), V, torch.int32)
        ids[7:7 + same] = 129   # more of one id in a warp's stretch than it lists
        d = randn(g, n, 8)
        got = eng.embed_grad(ids, d, V)
        held = ids >= 0
        ref = torch.zeros(V, 8, device="cuda", dtype=torch.float64).index_add_(0, ids[held].long(), d[held].double())
        mag = torch.zeros_like(ref).index_add_(0, ids[held].long(), d[held].double().abs())
        assert ((got.double() - ref).abs() <= n * 2.0 ** -24 * mag).all()


def test_offsets_beyond_32_bits(eng):  # noqa: F811
    """Tables and rows of more than 2^31 values: the far end gives what a small call gives."""
    V, H = 1_100_000, 2048
    table = torch.zeros(V, H, device="cuda", dtype=BF16)
    g = rng(28)
    table[-40:] = randn(g, 40, H, dtype=BF16)
    ids = torch.arange(V - 40, V, device="cuda")
    assert torch.equal(eng.embed(table, ids), table[-40:])
    d = randn(g, 40, H)
    grad = eng.embed_grad(ids, d, V)
    assert torch.equal(grad[-40:], d) and (grad[:100] == 0).all() and (grad[V // 2:V // 2 + 1000] == 0).all()
    del grad
    h = randn(g, 3, H, dtype=BF16)
    t = torch.tensor([V - 1, V - 40, 5], device="cuda")
    _, lse = eng.vocab_loss(h, table, t)
    _, dw = eng.vocab_loss_grad(h, table, t, lse, torch.ones(3, device="cuda"))
    small = table[-40:].clone()
    z = h.double() @ small.double().T
    p = torch.exp(z - lse.double()[:, None])
    p[0, 39] -= 1
    p[1, 0] -= 1
    ref = p.T @ h.double()
    assert ((dw[-40:].double() - ref).norm() / ref.norm()).item() <= 2 * BF
    del dw, table
    y = torch.zeros(V, H, device="cuda", dtype=BF16)
    y[-50:] = randn(g, 50, H, dtype=BF16)
    gain = 1 + randn(g, H, std=0.1)
    ho, n, rp, rr = eng.residual_norm(y, y, post_gain=gain, pre_gain=gain)
    ho2, n2, rp2, rr2 = eng.residual_norm(y[-50:], y[-50:], post_gain=gain, pre_gain=gain)
    assert torch.equal(ho[-50:], ho2) and torch.equal(n[-50:], n2)
    got = eng.residual_norm_grad(n, None, ho, y, rp, rr, post_gain=gain, pre_gain=gain)
    got2 = eng.residual_norm_grad(n2, None, ho2, y[-50:], rp2, rr2, post_gain=gain, pre_gain=gain)
    assert torch.equal(got["h"][-50:], got2["h"]) and torch.equal(got["y"][-50:], got2["y"])


def test_vectors_that_are_rows_of_a_wider_table(eng):  # noqa: F811
    """Modulation tables hold [scale | shift | gate] of a sample side by side; the gradients come dense."""
    c = norm_case(rng(29), 4, 6, 128, F32, F32, True, "sample", "sample", True)
    table = torch.cat([c["mod_scale"], c["mod_shift"], c["gate"]], 1)
    wide = dict(mod_scale=table[:, :128], mod_shift=table[:, 128:256], gate=table[:, 256:])
    kw = dict(post_gain=c["post_gain"], pre_gain=c["pre_gain"])
    dense = {k: c[k] for k in wide}
    a, b = eng.residual_norm(c["h"], c["y"], **kw, **wide), eng.residual_norm(c["h"], c["y"], **kw, **dense)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    dn = randn(rng(30), 4, 6, 128)
    ga = eng.residual_norm_grad(dn, dn, a[0], c["y"], a[2], a[3], **kw, **wide)
    gb = eng.residual_norm_grad(dn, dn, a[0], c["y"], a[2], a[3], **kw, **dense)
    assert all(torch.equal(ga[k], gb[k]) and ga[k].is_contiguous() for k in gb)


def test_refusals_leave_the_context_usable(eng):  # noqa: F811
    from vla_dual_expert_b200 import Dm0Error
    g = rng(31)
    table = randn(g, 10, 64, dtype=BF16)
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    shifted = torch.empty(10 * 64 + 1, device="cuda", dtype=BF16)[1:].view(10, 64)
    with pytest.raises(Dm0Error):
        eng.embed(shifted, ids)                                      # 2-byte aligned
    with pytest.raises(Dm0Error):
        eng.embed(table[:, :60].contiguous(), ids)
    with pytest.raises(TypeError):
        eng.embed(table.cpu(), ids)
    f = torch.zeros(3, 40, device="cuda")
    h, gain = torch.zeros(3, 2, 16, device="cuda"), torch.ones(16, device="cuda")
    for bad in (dict(gate=f[:2, :16]), dict(gate=f[0, :16].expand(3, 16)), dict(y=h[:, :1]), dict(pre_gain=gain[:8]),
                dict(mod_scale=f[:, :16], mod_shift=torch.zeros(3, 16, device="cuda"))):
        with pytest.raises(ValueError):
            eng.residual_norm(h, **{"y": h, **bad})
    for bad in (dict(gate=f.double()[:, :16]), dict(y=h.half()), dict(pre_gain=gain.cpu()), dict(h_out=h.bfloat16()),
                dict(post_gain=torch.ones(32, device="cuda")[::2]), dict(y=h.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(TypeError):
            eng.residual_norm(h, **{"y": h, **bad})
    with pytest.raises(ValueError):
        eng.embed_grad(ids, torch.zeros(3, 64, device="cuda"), 10, accumulate=True)
    with pytest.raises(ValueError):
        eng.embed_grad(ids, torch.zeros(4, 64, device="cuda"), 10)
    with pytest.raises(ValueError):
        eng.embed_grad(ids, torch.zeros(64, 3, device="cuda").t(), 10)   # rows that are not contiguous
    with pytest.raises(ValueError):
        eng.embed(table, ids, out=torch.zeros(3, 32, device="cuda"))
    with pytest.raises(TypeError):
        eng.embed(table.t(), ids)
    with pytest.raises(Dm0Error):
        eng.embed(table, ids[:0])
    with pytest.raises(Dm0Error):
        eng.vocab_loss(randn(g, 4, 72, dtype=BF16), randn(g, 5, 72, dtype=BF16), ids.new_zeros(4))
    with pytest.raises(Dm0Error):
        eng.vocab_loss_grad(table, table, ids.new_zeros(10), torch.zeros(10, device="cuda"),
                            torch.zeros(10, device="cuda"), dweight=torch.zeros_like(table), accumulate=True)
    with pytest.raises(Dm0Error):
        eng.residual_norm(randn(g, 2, 64), None, gate=torch.ones(64, device="cuda"))
    with pytest.raises(Dm0Error):
        eng.residual_norm(randn(g, 2, 8200))
    assert torch.equal(eng.embed(table, ids), table[ids])
    eng.sync()


def test_prefix_pass_from_tokens():
    """prefill over [image rows; text rows] passes on the rows that are made by hand here, and gives their cache."""
    from vla_dual_expert_b200 import Engine
    from tests.gpu_util import device_view_bf16
    d = I.TINY
    B, Ti, Tt, V = 2, 40, 9, 77
    e = Engine(d, B, Ti + Tt)
    try:
        e.load_from(I.Weights(d, seed=0))
        emb = I.prefix_embeddings(d, B, Ti)
        image = torch.from_numpy(np.ascontiguousarray(emb, np.float32)).cuda().to(BF16)
        g = rng(32)
        table, ids = randn(g, V, d.hidden_v, dtype=BF16), ids_of(g, (B, Tt), V)
        k, v = e.kv_view()
        shape = (d.layers, B, d.n_kv, Ti + Tt, d.head_dim)
        prefix = e.prefill_tokens(image, table, ids, scale=2.0)
        got = [device_view_bf16(p, shape).clone() for p in (k, v)]
        rows = torch.where((ids >= 0)[..., None], table[ids.clamp(min=0)].float() * 2, 0.0).to(BF16)
        assert torch.equal(prefix, torch.cat([image, rows], 1))
        e.prefill(torch.cat([image, rows], 1))
        e.sync()
        # the prefix pass of at most 128 rows adds its split products in any order (fp32 atomics), so equal prefixes
        # give cache values that may round to neighbouring bf16 values: each within a step, 2 * 2^-8 of it, and all
        # together within half of that
        for a, p in zip(got, (k, v)):
            b = device_view_bf16(p, shape).double()
            assert ((a.double() - b).norm() / b.norm()).item() <= BF
    finally:
        e.close()
