"""The language operators on a stream that is not torch's current one: whose memory their outputs and workspaces take."""
import pytest
import torch

from tests.test_language_gpu import BF16, eng, ids_of, loss_case, norm_case, randn, rng  # noqa: F401

pytestmark = pytest.mark.gpu


def pool_of(t):
    """The stream whose pool of torch's allocator holds the tensor."""
    at = t.data_ptr()
    found = [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"]]
    assert len(found) == 1
    return found[0]


def test_outputs_come_from_the_pool_of_the_calls_stream(eng):  # noqa: F811
    g = rng(51)
    V, H, N = 700, 128, 30
    table, ids, dout = randn(g, V, H, dtype=BF16), ids_of(g, (N,), V), randn(g, N, H)
    c = norm_case(g, 2, 15, H, torch.float32, BF16, True, "sample", "sample", True)
    kw = {k: v for k, v in c.items() if k not in ("h", "y")}
    h, n, r_post, r_pre = eng.residual_norm(c["h"], c["y"], **kw)
    x, w, t = loss_case(g, N, V, H)
    _, lse = eng.vocab_loss(x, w, t)
    one = torch.ones(N, device="cuda")
    calls = [lambda s: [eng.embed(table, ids, stream=s)], lambda s: [eng.embed_grad(ids, dout, V, stream=s)],
             lambda s: eng.residual_norm(c["h"], c["y"], stream=s, **kw),
             lambda s: eng.residual_norm_grad(n, None, h, c["y"], r_post, r_pre, stream=s, **kw).values(),
             lambda s: eng.vocab_loss(x, w, t, stream=s), lambda s: eng.vocab_loss_grad(x, w, t, lse, one, stream=s)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    here = torch.cuda.current_stream().cuda_stream
    for call in calls:
        want = list(call(None))
        assert all(pool_of(v) == here for v in want)
        torch.cuda.synchronize()
        for stream in (side, side.cuda_stream):
            got = list(call(stream))
            assert all(pool_of(v) == side.cuda_stream for v in got)
            side.synchronize()
            assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_work_pending_on_the_current_stream_is_not_disturbed(eng):  # noqa: F811
    """A block of the workspace's size, freed while kernels on the current stream still write it, is not the workspace of
    a call on a stream that waited only for its inputs; neither are the outputs' blocks."""
    N, V, H = 300, 40000, 256
    x, w, t = loss_case(rng(52), N, V, H)
    want = [v.clone() for v in eng.vocab_loss(x, w, t)]
    torch.cuda.synchronize()
    ws = eng.lib.dm0_vocab_loss_workspace(N, V, H)
    side = torch.cuda.Stream()
    for _ in range(5):
        blocks = [torch.empty(n, device="cuda", dtype=torch.uint8) for n in (ws, 4 * N, 4 * N)]
        for k in range(60):   # some milliseconds of writes
            for b in blocks:
                b.fill_(k)
        del b, blocks
        got = eng.vocab_loss(x, w, t, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_an_output_freed_by_its_reader_is_not_written_too_early(eng):  # noqa: F811
    """The current stream reads an output of another stream's call, which the program then drops: later calls there
    leave the memory alone until the reading is done."""
    g = rng(53)
    V, H, N = 500, 1024, 4000
    table = randn(g, V, H, dtype=BF16)
    ids = [torch.full((N,), k, device="cuda") for k in range(4)]
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    kept = []
    torch.cuda.synchronize()
    for k in range(4):
        out = eng.embed(table, ids[k], stream=side)
        here.wait_stream(side)
        late = torch.zeros_like(out)
        for _ in range(20):
            late.add_(1e-3)       # the read below waits behind these
        kept.append(out.clone())
        del out, late
    torch.cuda.synchronize()
    for k in range(4):
        assert torch.equal(kept[k], table[k].expand(N, H))


def test_a_captured_branch_on_its_own_stream(eng):  # noqa: F811
    """Inside a capture, on a stream that joined it: outputs and workspace belong to the graph, and replays agree while
    the program's own allocations go on."""
    N, V, H = 200, 3000, 128
    x, w, t = loss_case(rng(54), N, V, H)
    eng.vocab_loss(x, w, t)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        out = eng.vocab_loss(x, w, t, stream=side)
        here.wait_stream(side)
    x.mul_(0.5)
    want = eng.vocab_loss(x, w, t)
    for _ in range(3):
        others = [torch.full((n,), float("nan"), device="cuda") for n in [2 ** k for k in range(7, 20)] * 4]
        for v in out:
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        del others
    del graph
