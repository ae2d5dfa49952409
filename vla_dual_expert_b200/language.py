"""The language operators of Engine: token embedding, the norms around a block, the vocabulary loss, and their
gradients (include/dm0.h has their definitions).

Marshalling only, as the rest of the binding, and written for short calls: a single token's call is bound by
the host, so each tensor is checked by a few attribute reads and torch is bound once, with the first Engine.
"""
from __future__ import annotations

import ctypes

from ._abi import Dm0Norm, Dm0NormGrads

torch = None   # bound by the first Engine: building and packing need none
F32 = BF16 = None
_INTS = _FLOATS = ()


def _bind():
    global torch, F32, BF16, _INTS, _FLOATS
    if torch is None:
        import torch as t
        torch, F32, BF16 = t, t.float32, t.bfloat16
        _INTS, _FLOATS = (t.int64, t.int32), (t.bfloat16, t.float32)


def _check(t, device, dtypes, shape, name):
    """A contiguous tensor of `shape` and one of `dtypes` on CUDA device `device`; its address."""
    if t.dtype in dtypes and t.get_device() == device and t.is_contiguous() and t.shape == shape:
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise TypeError(f"{name} must be a contiguous tensor on cuda:{device} of {' or '.join(map(str, dtypes))}")


def _check_rows(t, device, shape, name):
    """As _check for [T][H] or [B][T][H] rows that are contiguous but may lie apart: (batch stride, row stride)."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in _FLOATS or t.get_device() != device:
        raise TypeError(f"{name} must be a bf16 or fp32 tensor on cuda:{device}")
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    # the stride of a dimension of one says nothing
    return (st[0] if len(st) == 3 and shape[0] > 1 else 0), (st[-2] if shape[-2] > 1 else shape[-1])


class LanguageOps:
    """Mixed into Engine, whose context handle, library and status check it uses."""

    def _open_language(self):
        _bind()
        self.device = torch.cuda.current_device()   # the context's: the tensors of these operators live there
        # the raw handle of the current stream, without building a Stream object around it
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._place = torch.device("cuda", self.device)

    def _on(self, stream):
        if stream is None:
            return self._raw_stream(self.device)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def _scratch(self, nbytes: int, stream):
        """Workspace of one call, from torch's allocator, which keeps it from others until the call's stream is past
        it."""
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=self._place)
        if stream is not None:
            ws.record_stream(stream if isinstance(stream, torch.cuda.Stream) else
                             torch.cuda.ExternalStream(self._on(stream), self.device))
        return ws

    def _ids(self, ids):
        shape = ids.shape
        if len(shape) != 1 and len(shape) != 2:
            raise ValueError("ids must be [T] or [B][T]")
        return _check(ids, self.device, _INTS, shape, "ids"), ids.dtype == torch.int64, shape

    def embed(self, table, ids, scale: float = 1.0, out=None, stream=None):
        """scale * table[ids] (dm0_embed), a zero row where an id is negative.

        table: CUDA bf16 [vocab][hidden]; ids: int32 or int64 [T] or [B][T]; out (bf16, made if not given, or fp32):
        [T][hidden] or [B][T][hidden], whose rows are contiguous but may lie apart, as the text rows behind the
        image rows of a prefix do: out=prefix_emb[:, image_rows:]."""
        ip, wide, shape = self._ids(ids)
        tshape = table.shape
        if len(tshape) != 2:
            raise ValueError("table must be [vocab][hidden]")
        V, H = tshape
        tp = _check(table, self.device, (BF16,), tshape, "table")
        oshape = (*shape, H)
        if out is None:
            out = torch.empty(*oshape, dtype=BF16, device=self._place)
        bs, rs = _check_rows(out, self.device, oshape, "out")
        st = self.lib.dm0_embed(self.h, tp, ip, wide, 1 if len(shape) == 1 else shape[0], shape[-1], V, H, scale,
                                out.data_ptr(), out.dtype == F32, bs, rs, self._on(stream))
        if st:
            self._chk(st)
        return out

    def prefill_tokens(self, image_emb, table, ids, scale: float = 1.0):
        """Prefix pass over [image rows; text rows] on the current stream: image_emb CUDA bf16 [B][Ti][hidden_v], and
        the table's rows of ids [B][Tt] behind them.  Returns the prefix it passed to prefill, [B][Ti + Tt][hidden_v]."""
        B, Ti, H = image_emb.shape
        _check_rows(image_emb, self.device, (B, Ti, H), "image_emb")
        prefix = torch.empty(B, Ti + ids.shape[-1], H, dtype=BF16, device=self._place)
        prefix[:, :Ti] = image_emb
        self.embed(table, ids, scale, out=prefix[:, Ti:])
        self.prefill(prefix)
        return prefix

    def embed_grad(self, ids, dout, vocab: int, scale: float = 1.0, grad=None, accumulate: bool = False, stream=None):
        """Gradient of embed with respect to its table (dm0_embed_grad): f32 [vocab][hidden].

        dout: bf16 or fp32 rows as embed's out.  accumulate adds to `grad`, e.g. to the weight gradient that
        vocab_loss_grad left there when the loss's weights are the table."""
        ip, wide, shape = self._ids(ids)
        H = dout.shape[-1]
        bs, rs = _check_rows(dout, self.device, (*shape, H), "dout")
        if grad is None:
            if accumulate:
                raise ValueError("accumulate needs grad")
            grad = torch.empty(vocab, H, dtype=F32, device=self._place)
        gp = _check(grad, self.device, (F32,), (vocab, H), "grad")
        B, T = 1 if len(shape) == 1 else shape[0], shape[-1]
        n = self.lib.dm0_embed_grad_workspace(B, T, vocab, H)
        ws = self._scratch(n, stream)
        st = self.lib.dm0_embed_grad(self.h, ip, wide, B, T, vocab, H, scale, dout.data_ptr(), dout.dtype == F32, bs, rs,
                                     gp, accumulate, ws.data_ptr(), n, self._on(stream))
        if st:
            self._chk(st)
        return grad

    def _vector(self, v, B, H, name):
        """Address and sample stride (0: one row for all) of a per-sample vector."""
        if v is None:
            return None, 0
        shape, st = v.shape, v.stride()
        if v.dtype != F32 or v.get_device() != self.device or st[-1] != 1:
            raise TypeError(f"{name} must be an fp32 tensor on cuda:{self.device} with contiguous rows")
        if shape == (H,) or (B == 1 and shape == (1, H)):
            return v.data_ptr(), 0
        if shape != (B, H):
            raise ValueError(f"{name} has shape {tuple(shape)}, expected {(H,)} or {(B, H)}")
        if st[0] < H:
            raise ValueError(f"the rows of {name} overlap")
        return v.data_ptr(), st[0]

    def _norm(self, h, y, post_gain, gate, scale, pre_gain, mod_scale, mod_shift):
        """The dm0_norm of a call, and the addresses of h and y."""
        dev, shape = self.device, h.shape
        if len(shape) == 3:
            B, T, H = shape
        elif len(shape) == 2:
            B, (T, H) = 1, shape
        else:
            raise ValueError("the residual stream must be [T][hidden] or [B][T][hidden]")
        hp = _check(h, dev, _FLOATS, shape, "the residual stream")
        yp = None if y is None else _check(y, dev, _FLOATS, shape, "y")
        post = None if post_gain is None else _check(post_gain, dev, (F32,), (H,), "post_gain")
        pre = None if pre_gain is None else _check(pre_gain, dev, (F32,), (H,), "pre_gain")
        gp, gs = self._vector(gate, B, H, "gate")
        sp, ss = self._vector(mod_scale, B, H, "mod_scale")
        tp, ts = self._vector(mod_shift, B, H, "mod_shift")
        if sp is not None and tp is not None and ss != ts:
            raise ValueError("mod_scale and mod_shift must be laid out alike")
        return Dm0Norm(B, T, H, h.dtype == F32, y is not None and y.dtype == F32, scale, post, gp, gs, pre, sp, tp,
                       ss or ts), hp, yp

    def residual_norm(self, h, y=None, post_gain=None, gate=None, scale: float = 1.0, pre_gain=None, mod_scale=None,
                      mod_shift=None, h_out=None, n_out=None, stream=None):
        """The boundary behind a block (dm0_residual_norm): norm of its output y, gate, scaled residual and the next
        block's norm, in one pass.

        h, y: bf16 or fp32 [T][hidden] or [B][T][hidden]; gains f32 [hidden]; gate, mod_scale, mod_shift f32 [hidden]
        or [B][hidden].  Returns (h_out, n_out bf16, r_post or None, r_pre); the last two are the rows' 1 / rms for
        residual_norm_grad."""
        a, hp, yp = self._norm(h, y, post_gain, gate, scale, pre_gain, mod_scale, mod_shift)
        shape = h.shape
        if h_out is None:
            h_out = torch.empty_like(h)
        if n_out is None:
            n_out = torch.empty_like(h, dtype=BF16)
        r_pre = torch.empty(*shape[:-1], dtype=F32, device=self._place)
        r_post = None if post_gain is None else torch.empty_like(r_pre)
        st = self.lib.dm0_residual_norm(self.h, ctypes.byref(a), hp, yp,
                                        _check(h_out, self.device, (h.dtype,), shape, "h_out"),
                                        _check(n_out, self.device, (BF16,), shape, "n_out"),
                                        None if r_post is None else r_post.data_ptr(), r_pre.data_ptr(), self._on(stream))
        if st:
            self._chk(st)
        return h_out, n_out, r_post, r_pre

    def residual_norm_grad(self, dn, dh_out, h_out, y, r_post, r_pre, post_gain=None, gate=None, scale: float = 1.0,
                           pre_gain=None, mod_scale=None, mod_shift=None, stream=None) -> dict:
        """Adjoint of residual_norm (dm0_residual_norm_grad), from its outputs and the gradients dn (bf16 or fp32) of
        n_out and dh_out (the residual's type, or None) of h_out.

        Returns a dict: "h", "y" (their types) and, for each vector that was given, its f32 gradient ("post_gain",
        "gate", "pre_gain", "mod_scale", "mod_shift"), of the vector's shape."""
        a, hp, yp = self._norm(h_out, y, post_gain, gate, scale, pre_gain, mod_scale, mod_shift)
        dev, shape = self.device, h_out.shape
        np_ = _check(dn, dev, _FLOATS, shape, "dn")
        up = None if dh_out is None else _check(dh_out, dev, (h_out.dtype,), shape, "dh_out")
        rp = _check(r_pre, dev, (F32,), shape[:-1], "r_pre")
        rq = None if r_post is None else _check(r_post, dev, (F32,), shape[:-1], "r_post")
        out = {"h": torch.empty_like(h_out)}
        dy = None
        if y is not None:
            out["y"] = torch.empty_like(y)
            dy = out["y"].data_ptr()
        ptrs = []
        for name, v in (("post_gain", post_gain), ("gate", gate), ("pre_gain", pre_gain), ("mod_scale", mod_scale),
                        ("mod_shift", mod_shift)):
            if v is None:
                ptrs.append(None)
            else:
                out[name] = t = torch.empty_like(v)   # dense: rows that lie apart are not copied in their strides
                ptrs.append(t.data_ptr())
        g = Dm0NormGrads(*ptrs)
        n = self.lib.dm0_residual_norm_grad_workspace(ctypes.byref(a))
        ws = self._scratch(n, stream)
        st = self.lib.dm0_residual_norm_grad(self.h, ctypes.byref(a), np_, dn.dtype == F32, up, hp, yp, rq, rp,
                                             out["h"].data_ptr(), dy, ctypes.byref(g), ws.data_ptr(), ws.numel(),
                                             self._on(stream))
        if st:
            self._chk(st)
        return out

    def _vocab(self, hidden, weight, targets):
        hs, wsh = hidden.shape, weight.shape
        if len(hs) != 2 or len(wsh) != 2 or wsh[1] != hs[1]:
            raise ValueError("hidden must be [tokens][H] and weight [vocab][H]")
        dev = self.device
        return (hs[0], wsh[0], hs[1], _check(hidden, dev, (BF16,), hs, "hidden"),
                _check(weight, dev, (BF16,), wsh, "weight"), _check(targets, dev, _INTS, hs[:1], "targets"),
                targets.dtype == torch.int64)

    def vocab_loss(self, hidden, weight, targets, stream=None):
        """Softmax cross entropy of hidden @ weight.T against targets without keeping the logits (dm0_vocab_loss).

        hidden: bf16 [tokens][H]; weight: bf16 [vocab][H]; targets: int32 or int64 [tokens], negative: no target.
        Returns (loss, lse), f32 [tokens]; -loss is the target's log probability, lse is for vocab_loss_grad."""
        N, V, H, hp, wp, tp, wide = self._vocab(hidden, weight, targets)
        loss = torch.empty(N, dtype=F32, device=self._place)
        lse = torch.empty_like(loss)
        n = self.lib.dm0_vocab_loss_workspace(N, V, H)
        ws = self._scratch(n, stream)
        st = self.lib.dm0_vocab_loss(self.h, hp, wp, tp, wide, N, V, H, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                                     n, self._on(stream))
        if st:
            self._chk(st)
        return loss, lse

    def vocab_loss_grad(self, hidden, weight, targets, lse, dloss, dhidden=None, dweight=None,
                        accumulate: bool = False, stream=None):
        """Gradients of sum(dloss * loss) of vocab_loss with respect to hidden and weight (dm0_vocab_loss_grad).

        lse, dloss: f32 [tokens].  dhidden [tokens][H] and dweight [vocab][H] are bf16 unless an fp32 tensor is
        given; False leaves that gradient out.  accumulate adds to an fp32 dweight.  Returns (dhidden, dweight)."""
        N, V, H, hp, wp, tp, wide = self._vocab(hidden, weight, targets)
        if accumulate and not isinstance(dweight, torch.Tensor):
            raise ValueError("accumulate needs dweight")
        dh, dw = (torch.empty_like(like) if t is None else None if t is False else t
                  for t, like in ((dhidden, hidden), (dweight, weight)))
        n = self.lib.dm0_vocab_loss_grad_workspace(N, V, H)
        ws = self._scratch(n, stream)
        st = self.lib.dm0_vocab_loss_grad(
            self.h, hp, wp, tp, wide, _check(lse, self.device, (F32,), (N,), "lse"),
            _check(dloss, self.device, (F32,), (N,), "dloss"), N, V, H,
            None if dh is None else _check(dh, self.device, _FLOATS, (N, H), "dhidden"), dh is not None and dh.dtype == F32,
            None if dw is None else _check(dw, self.device, _FLOATS, (V, H), "dweight"), dw is not None and dw.dtype == F32,
            accumulate, ws.data_ptr(), n, self._on(stream))
        if st:
            self._chk(st)
        return dh, dw
