"""The language-side operators, as cases that can be timed and compared: token embedding rows and their
gradient, the norms on both sides of a block with its gate and residual, and the softmax cross entropy over a
vocabulary, each with its backward pass.

`listed()` names fixed cases, `draw(rng)` gives others of the same ranges, `prepare(case, seed)` makes the
tensors a program has before the call, and `run(state)` makes one pass: with `own` false in plain torch
operations in 32 bits, with `own` true through vla_dual_expert_b200.Engine.  `exact(case, seed)` evaluates the
same definition in 64 bits.
"""
from __future__ import annotations

import functools
import math
import types

import torch

own = False

EPS = 1e-6   # of the norms (rms_eps of the model configuration)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token of one observation: latency
        dict(name="embed_one", op="embed", batch=1, tokens=1, skip=0, vocab=32003, hidden=2048, out="bf16", wide_ids=True),
        # the text rows of a batch of prompts, written behind 768 image rows of each sample's prefix
        dict(name="embed_text_rows", op="embed", batch=16, tokens=48, skip=768, vocab=131072, hidden=2048, out="bf16",
             wide_ids=True),
        # whole prompts of a training batch
        dict(name="embed_prompts", op="embed", batch=16, tokens=2048, skip=0, vocab=131072, hidden=2048, out="bf16",
             wide_ids=False),
        # a small table's gradient from the text rows of a batch, fp32 gradients of the residual stream
        dict(name="embed_grad_text_rows", op="embed_grad", batch=16, tokens=48, skip=768, vocab=32003, hidden=1024,
             dout="f32", wide_ids=True),
        # the gradient of a large table from whole prompts: frequent tokens thousands of times, most never
        dict(name="embed_grad_prompts", op="embed_grad", batch=16, tokens=2048, skip=0, vocab=131072, hidden=2048,
             dout="bf16", wide_ids=True),
        # one observation's 50 action tokens: gate and time modulation, latency
        dict(name="norm_chunk", op="norm", batch=1, tokens=50, hidden=1024, h="f32", y="bf16", post=False, gate="sample",
             mod=True, pre=False, scale=1.0),
        # the prefix pass of 16 observations with norms on both sides of the block
        dict(name="norm_prefix", op="norm", batch=16, tokens=2048, hidden=2048, h="f32", y="bf16", post=True, gate="none",
             mod=False, pre=True, scale=1.0),
        # a training batch of action chunks: gate and modulation per sample
        dict(name="norm_grad_chunks", op="norm_grad", batch=16, tokens=50, hidden=1024, h="f32", y="f32", post=False,
             gate="sample", mod=True, pre=True, scale=1.0),
        # a training batch of prefixes, norms on both sides, one learned gate for every row, a scaled residual
        dict(name="norm_grad_prefix", op="norm_grad", batch=16, tokens=2048, hidden=2048, h="f32", y="bf16", post=True,
             gate="shared", mod=False, pre=True, scale=0.5),
        # the log probabilities of a few tokens of an answer: the weights are read once
        dict(name="loss_score", op="loss", tokens=7, vocab=131072, hidden=2048, wide_ids=True),
        # a training batch's loss
        dict(name="loss_train", op="loss", tokens=4096, vocab=131072, hidden=2048, wide_ids=True),
        # a training batch's gradients, mean over the tokens with a target
        dict(name="loss_grad_train", op="loss_grad", tokens=8192, vocab=131072, hidden=2048, weights="mean", wide_ids=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "loss", "loss_grad"])
    wide = rng.random() < 0.5
    if op in ("embed", "embed_grad"):
        batch = rng.randint(1, 16)
        tokens = _log(rng, 1, 2048)
        c = dict(op=op, batch=batch, tokens=tokens, skip=rng.choice([0, 0, 1, 256, 768]), vocab=_log(rng, 1000, 131072),
                 hidden=8 * _log(rng, 16, 256), wide_ids=wide)
        c["out" if op == "embed" else "dout"] = rng.choice(["bf16", "f32"]) if tokens <= 1024 else "bf16"
        return c
    if op in ("norm", "norm_grad"):
        return dict(op=op, batch=rng.randint(1, 16), tokens=_log(rng, 1, 2000), hidden=8 * _log(rng, 16, 256),
                    h=rng.choice(["f32", "f32", "bf16"]), y=rng.choice(["bf16", "bf16", "f32"]) if op == "norm" else "bf16",
                    post=rng.random() < 0.5, gate=rng.choice(["none", "shared", "sample"]), mod=rng.random() < 0.5,
                    pre=rng.random() < 0.7, scale=rng.choice([1.0, 0.5]))
    hidden = 64 * _log(rng, 2, 32)
    vocab = _log(rng, 1000, 131072)
    c = dict(op=op, tokens=_log(rng, 1, 4096 if op == "loss" else 8192), vocab=vocab, hidden=hidden, wide_ids=wide)
    if op == "loss_grad":
        c["weights"] = rng.choice(["mean", "each"])
    return c


# ----------------------------------------------------------------------------------------------- inputs
def _ids(g, shape, vocab, missing, wide):
    """Token ids with a few very frequent ones, and a share of -1 (no token, no target)."""
    u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
    v = (vocab * u ** 4).long().clamp_(max=vocab - 1)
    gone = torch.rand(shape, generator=g, device="cuda") < missing
    v = torch.where(gone, torch.full_like(v, -1), v)
    return v if wide else v.int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)

    def rand(*shape, dtype="f32", std=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(DT[dtype])

    op, H = case["op"], case["hidden"]
    if op in ("embed", "embed_grad"):
        B, T, skip = case["batch"], case["tokens"], case["skip"]
        s["factor"] = math.sqrt(H)
        s["ids"] = _ids(g, (B, T), case["vocab"], 0.05, case["wide_ids"])
        if op == "embed":
            s["table"] = rand(case["vocab"], H, dtype="bf16", std=0.02)
            s["out_rows"] = torch.zeros(B, skip + T, H, device="cuda", dtype=DT[case["out"]])[:, skip:]
        else:
            s["dout_rows"] = rand(B, skip + T, H, dtype=case["dout"], std=1e-3)[:, skip:]
        return s
    if op in ("norm", "norm_grad"):
        B, T = case["batch"], case["tokens"]
        s["h_in" if op == "norm" else "h_out"] = rand(B, T, H, dtype=case["h"], std=2.0)
        s["y_in"] = rand(B, T, H, dtype=case["y"], std=0.7)
        s["post_gain"] = 1 + rand(H, std=0.1) if case["post"] else None
        s["pre_gain"] = 1 + rand(H, std=0.1) if case["pre"] else None
        s["gate_v"] = None if case["gate"] == "none" else rand(H, std=0.5) if case["gate"] == "shared" else rand(B, H, std=0.5)
        s["mod_scale"] = rand(B, H, std=0.1) if case["mod"] else None
        s["mod_shift"] = rand(B, H, std=0.1) if case["mod"] else None
        if op == "norm_grad":
            s["dn"] = rand(B, T, H, dtype="bf16", std=1e-3)
            s["dh_out"] = rand(B, T, H, dtype=case["h"], std=1e-3)
            s["r_pre"] = torch.rsqrt(s["h_out"].float().square().mean(-1) + EPS)
            s["r_post"] = torch.rsqrt(s["y_in"].float().square().mean(-1) + EPS) if case["post"] else None
        return s
    N, V = case["tokens"], case["vocab"]
    s["weight"] = rand(V, H, dtype="bf16", std=0.02)
    s["targets"] = _ids(g, (N,), V, 0.1, case["wide_ids"])
    # hidden states that know their target to different degrees: probabilities from 1/V to nearly 1
    at = s["weight"][s["targets"].long().clamp(min=0)].float()
    know = torch.rand((N, 1), generator=g, device="cuda") * 22 / (0.02 * math.sqrt(H)) * 0.9
    s["hidden_rows"] = (rand(N, H) + know * at / at.norm(dim=1, keepdim=True)).to(torch.bfloat16)
    if op == "loss_grad":
        x, parts = s["hidden_rows"].float(), []
        for v0 in range(0, V, 16384):
            parts.append(torch.logsumexp(x @ s["weight"][v0:v0 + 16384].float().T, 1))
        s["lse"] = torch.logsumexp(torch.stack(parts), 0)
        if case["weights"] == "mean":
            s["dloss"] = torch.ones(N, device="cuda") / (s["targets"] >= 0).sum().clamp(min=1)
        else:
            s["dloss"] = torch.rand(N, generator=g, device="cuda") / N
    return s


# ----------------------------------------------------------------------------------------- plain forms
def _embed(s):
    ids = s["ids"].long()
    rows = s["table"][ids.clamp(min=0)].float() * s["factor"]
    s["out_rows"].copy_(torch.where((ids >= 0)[..., None], rows, torch.zeros((), device="cuda")))
    return s["out_rows"]


def _embed_grad(s):
    ids = s["ids"].long()
    rows = torch.where((ids >= 0)[..., None], s["dout_rows"].float() * s["factor"], torch.zeros((), device="cuda"))
    grad = torch.zeros(s["vocab"], s["hidden"], device="cuda")
    return grad.index_add_(0, ids.clamp(min=0).flatten(), rows.flatten(0, 1))


def _per_row(v):
    """[H] for every row, or [B][H] for the rows of each sample."""
    return v if v is None or v.dim() == 1 else v[:, None, :]


def _norm(s):
    h, y = s["h_in"].float(), s["y_in"].float()
    out = {}
    if s["post_gain"] is not None:
        out["r_post"] = torch.rsqrt((y * y).mean(-1) + EPS)
        y = y * out["r_post"][..., None] * s["post_gain"]
    if s["gate_v"] is not None:
        y = y * _per_row(s["gate_v"])
    h = h * s["scale"] + y
    out["r_pre"] = torch.rsqrt((h * h).mean(-1) + EPS)
    n = h * out["r_pre"][..., None]
    if s["pre_gain"] is not None:
        n = n * s["pre_gain"]
    if s["mod_scale"] is not None:
        n = n * (1 + _per_row(s["mod_scale"])) + _per_row(s["mod_shift"])
    out["h"] = h.to(DT[s["h"]])
    out["n"] = n.to(torch.bfloat16)
    return out


def _norm_grad(s):
    h, y, dn = s["h_out"].float(), s["y_in"].float(), s["dn"].float()
    x = h * s["r_pre"][..., None]
    gain = torch.ones(s["hidden"], device="cuda") if s["pre_gain"] is None else s["pre_gain"]
    modul = torch.ones_like(gain) if s["mod_scale"] is None else 1 + _per_row(s["mod_scale"])
    out = {}
    if s["mod_scale"] is not None:
        out["mod_scale"] = (dn * x * gain).sum(1)
        out["mod_shift"] = dn.sum(1)
    if s["pre_gain"] is not None:
        out["pre_gain"] = (dn * x * modul).sum((0, 1))
    dx = dn * gain * modul
    dh = s["dh_out"].float() + s["r_pre"][..., None] * (dx - x * (dx * x).mean(-1, keepdim=True))
    out["h"] = (dh * s["scale"]).to(DT[s["h"]])
    u = y if s["post_gain"] is None else y * s["r_post"][..., None] * s["post_gain"]
    du = dh
    if s["gate_v"] is not None:
        out["gate"] = (dh * u).sum(1 if s["gate_v"].dim() == 2 else (0, 1))
        du = dh * _per_row(s["gate_v"])
    if s["post_gain"] is not None:
        z = y * s["r_post"][..., None]
        out["post_gain"] = (du * z).sum((0, 1))
        dz = du * s["post_gain"]
        du = s["r_post"][..., None] * (dz - z * (dz * z).mean(-1, keepdim=True))
    out["y"] = du.to(DT[s["y"]])
    return out


def _loss(s):
    t = s["targets"].long()
    logits = s["hidden_rows"].float() @ s["weight"].float().T
    top = logits.amax(1)
    lse = top + (logits - top[:, None]).exp().sum(1).log()
    picked = logits.gather(1, t.clamp(min=0)[:, None])[:, 0]
    return {"loss": torch.where(t >= 0, lse - picked, torch.zeros((), device="cuda")), "lse": lse}


def _loss_grad(s):
    t = s["targets"].long()
    x, w = s["hidden_rows"].float(), s["weight"].float()
    p = (x @ w.T - s["lse"][:, None]).exp_()
    p.scatter_add_(1, t.clamp(min=0)[:, None], torch.full((t.shape[0], 1), -1.0, device="cuda"))
    p *= torch.where(t >= 0, s["dloss"], torch.zeros((), device="cuda"))[:, None]
    return {"hidden": (p @ w).to(torch.bfloat16), "weight": (p.T @ x).to(torch.bfloat16)}


_PLAIN = dict(embed=_embed, embed_grad=_embed_grad, norm=_norm, norm_grad=_norm_grad, loss=_loss, loss_grad=_loss_grad)


# ---------------------------------------------------------------------------------- the framework's calls
@functools.lru_cache(maxsize=None)
def _engine():
    """A context; these operators take their sizes from their tensors, so a small model's context does."""
    from vla_dual_expert_b200 import Engine
    dims = types.SimpleNamespace(layers=1, hidden_v=128, inter_v=128, hidden_a=128, inter_a=128, n_q=4, n_kv=2,
                                 head_dim=32, chunk=4, action_dim=8, rope_theta=1e6, rms_eps=EPS)
    return Engine(dims, 1, 16)


def _own_run(s):
    eng, op = _engine(), s["op"]
    if op == "embed":
        return eng.embed(s["table"], s["ids"], scale=s["factor"], out=s["out_rows"])
    if op == "embed_grad":
        return eng.embed_grad(s["ids"], s["dout_rows"], s["vocab"], scale=s["factor"])
    if op == "norm":
        h, n, r_post, r_pre = eng.residual_norm(s["h_in"], s["y_in"], post_gain=s["post_gain"], gate=s["gate_v"],
                                                scale=s["scale"], pre_gain=s["pre_gain"], mod_scale=s["mod_scale"],
                                                mod_shift=s["mod_shift"])
        return {"h": h, "n": n, "r_pre": r_pre} | ({"r_post": r_post} if r_post is not None else {})
    if op == "norm_grad":
        return eng.residual_norm_grad(s["dn"], s["dh_out"], s["h_out"], s["y_in"], s["r_post"], s["r_pre"],
                                      post_gain=s["post_gain"], gate=s["gate_v"], scale=s["scale"],
                                      pre_gain=s["pre_gain"], mod_scale=s["mod_scale"], mod_shift=s["mod_shift"])
    if op == "loss":
        loss, lse = eng.vocab_loss(s["hidden_rows"], s["weight"], s["targets"])
        return {"loss": loss, "lse": lse}
    dh, dw = eng.vocab_loss_grad(s["hidden_rows"], s["weight"], s["targets"], s["lse"], s["dloss"])
    return {"hidden": dh, "weight": dw}


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------- work and exactness
def work(case):
    op, H = case["op"], case["hidden"]
    size = {"bf16": 2, "f32": 4}
    if op in ("embed", "embed_grad"):
        n = case["batch"] * case["tokens"]
        idb = n * (8 if case["wide_ids"] else 4)
        if op == "embed":
            return {"bytes": idb + n * H * (2 + size[case["out"]]), "flops": n * H}
        return {"bytes": idb + n * H * size[case["dout"]] + case["vocab"] * H * 4, "flops": 2 * n * H}
    if op in ("norm", "norm_grad"):
        n = case["batch"] * case["tokens"] * H
        h, y = size[case["h"]], size[case["y"]]
        if op == "norm":
            return {"bytes": n * (2 * h + y + 2), "flops": 10 * n}
        return {"bytes": n * (3 * h + 2 * y + 2), "flops": 24 * n}
    N, V = case["tokens"], case["vocab"]
    idb = N * (8 if case["wide_ids"] else 4)
    if op == "loss":
        return {"bytes": idb + 2 * H * (N + V) + 8 * N, "flops": 2 * N * V * H}
    return {"bytes": idb + 2 * 2 * H * (N + V) + 8 * N, "flops": 6 * N * V * H}


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()
         if k not in ("table", "weight")}
    op, H = case["op"], case["hidden"]
    if op == "embed":
        flat = s["ids"].long().reshape(-1)
        out = torch.zeros(flat.numel(), H, device="cuda", dtype=torch.float64)
        held = (flat >= 0).nonzero()[:, 0]
        out[held] = math.sqrt(H) * s["table"].index_select(0, flat[held]).double()
        return out.view(case["batch"], case["tokens"], H)
    if op == "embed_grad":
        flat = s["ids"].long().reshape(-1)
        held = (flat >= 0).nonzero()[:, 0]
        rows = d["dout_rows"].reshape(-1, H)[held]
        grad = torch.zeros(case["vocab"], H, device="cuda", dtype=torch.float64)
        grad.index_put_((flat[held],), rows * math.sqrt(H), accumulate=True)
        return grad
    if op == "norm":
        out = {}
        u = d["y_in"]
        if case["post"]:
            out["r_post"] = 1 / (u.pow(2).sum(-1) / H + EPS).sqrt()
            u = torch.einsum("bth,bt,h->bth", u, out["r_post"], d["post_gain"])
        if case["gate"] != "none":
            u = u * (d["gate_v"] if case["gate"] == "shared" else d["gate_v"].unsqueeze(1))
        h = case["scale"] * d["h_in"] + u
        out["h"] = h
        out["r_pre"] = 1 / (h.pow(2).sum(-1) / H + EPS).sqrt()
        n = torch.einsum("bth,bt->bth", h, out["r_pre"])
        n = n * d["pre_gain"] if case["pre"] else n
        out["n"] = n * (1 + d["mod_scale"]).unsqueeze(1) + d["mod_shift"].unsqueeze(1) if case["mod"] else n
        return out
    if op == "norm_grad":
        # every gradient by automatic differentiation of the definition, the saved 1/rms values as functions
        # of what they were saved from
        y = d["y_in"].clone().requires_grad_()
        h = d["h_out"].clone().requires_grad_()
        names = {"pre_gain": "pre_gain", "mod_scale": "mod_scale", "mod_shift": "mod_shift"}
        par = {k: d[v].clone().requires_grad_() for k, v in names.items() if d[v] is not None}
        n = h / (h.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        n = n * par["pre_gain"] if "pre_gain" in par else n
        n = n * (1 + par["mod_scale"][:, None]) + par["mod_shift"][:, None] if "mod_scale" in par else n
        got = torch.autograd.grad(n, [h, *par.values()], d["dn"])
        dh = got[0] + d["dh_out"]
        out = dict(zip(par, got[1:]))
        out["h"] = case["scale"] * dh
        par = {k: d[v].clone().requires_grad_() for k, v in {"post_gain": "post_gain", "gate": "gate_v"}.items()
               if d[v] is not None}
        u = y
        if case["post"]:
            u = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * par["post_gain"]
        if case["gate"] != "none":
            u = u * (par["gate"] if case["gate"] == "shared" else par["gate"][:, None])
        got = torch.autograd.grad(u, [y, *par.values()], dh)
        out["y"] = got[0]
        out.update(zip(par, got[1:]))
        return out
    N, V = case["tokens"], case["vocab"]
    t = s["targets"].long()
    held = (t >= 0).nonzero()[:, 0]
    step = max(1, (1 << 27) // N)
    if op == "loss":
        parts = torch.stack([torch.logsumexp(d["hidden_rows"] @ s["weight"][v:v + step].double().T, 1)
                             for v in range(0, V, step)])
        lse = torch.logsumexp(parts, 0)
        loss = torch.zeros_like(lse)
        loss[held] = lse[held] - (d["hidden_rows"][held] * s["weight"][t[held]].double()).sum(1)
        return {"loss": loss, "lse": lse}
    row = torch.zeros(N, 1, device="cuda", dtype=torch.float64)
    row[held, 0] = d["dloss"][held]
    dh, dw = torch.zeros(N, H, device="cuda", dtype=torch.float64), []
    for v in range(0, V, step):
        w = s["weight"][v:v + step].double()
        p = row * torch.exp(d["hidden_rows"] @ w.T - d["lse"][:, None])
        here = held[(t[held] >= v) & (t[held] < v + step)]
        p[here, t[here] - v] -= row[here, 0]
        dh += p @ w
        dw.append((p.T @ d["hidden_rows"]).to(torch.float32))
    return {"hidden": dh, "weight": torch.cat(dw)}
