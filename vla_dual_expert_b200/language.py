"""The language operators of Engine: token embedding, the norms around a block, the vocabulary loss, and their
gradients (include/dm0.h has their definitions).

Marshalling only, as the rest of the binding.  Calls on a few tokens are bound by the host, so the tensors are
checked and the outputs and workspaces made in native code (csrc/binding.cpp, built beside libdm0.so): TypeError
for a tensor of another type, device or layout, ValueError for another shape, Dm0Error for what the C ABI refuses.
`stream` is a torch stream or a cudaStream_t handle; None is torch's current stream.  A call on another stream waits
for nothing on the current one: its inputs, and an output that is given, have to be ready there and are the caller's
to keep.  Its outputs and workspace come from that stream's pool; outputs are kept until both streams are past them,
and a third stream that uses one is recorded by the caller (Tensor.record_stream), as with any tensor of torch's.
"""
from __future__ import annotations


class _Unbound:
    """In place of the native module until an operator is called: an Engine's other calls need neither it nor torch."""

    def __getattr__(self, name):
        _bind()
        return getattr(_C, name)


_C = _Unbound()


def _bind():
    global _C
    if isinstance(_C, _Unbound):
        import torch  # noqa: F401  (before the native module, which links against its libraries)
        try:
            from . import _language
        except ImportError as e:
            raise ImportError(f"_language.so did not load ({e}); run `python -m vla_dual_expert_b200.build`") from e
        _C = _language


def _handle(stream):
    return None if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class LanguageOps:
    """Mixed into Engine, whose context handle, device and status check it uses."""

    def _done(self, r):
        """The native call's outputs; a status instead of them raises."""
        if r.__class__ is int:
            self._chk(r)
        return r

    def embed(self, table, ids, scale: float = 1.0, out=None, stream=None):
        """scale * table[ids] (dm0_embed), a zero row where an id is negative.

        table: CUDA bf16 [vocab][hidden]; ids: int32 or int64 [T] or [B][T]; out (bf16, made if not given, or fp32):
        [T][hidden] or [B][T][hidden], whose rows are contiguous but may lie apart, as the text rows behind the
        image rows of a prefix do: out=prefix_emb[:, image_rows:]."""
        return self._done(_C.embed(self.h.value or 0, self.device, table, ids, scale, out, _handle(stream)))

    def prefill_tokens(self, image_emb, table, ids, scale: float = 1.0):
        """Prefix pass over [image rows; text rows] on the current stream: image_emb CUDA bf16 [B][Ti][hidden_v], and
        the table's rows of ids [B][Tt] behind them.  Returns the prefix it passed to prefill, [B][Ti + Tt][hidden_v].
        The image rows are copied there; a program that makes them in its own prefix tensor has no copy with
        embed(table, ids, out=prefix[:, Ti:]) and prefill(prefix)."""
        import torch
        B, Ti, H = image_emb.shape
        if ids.dim() != 2 or ids.shape[0] != B:
            raise ValueError(f"ids has shape {tuple(ids.shape)}, expected [{B}][Tt]")
        if not image_emb.is_cuda or image_emb.dtype != torch.bfloat16:
            raise TypeError("image_emb must be a CUDA torch.bfloat16 tensor")
        prefix = torch.empty(B, Ti + ids.shape[1], H, dtype=torch.bfloat16, device=image_emb.device)
        prefix[:, :Ti] = image_emb
        self.embed(table, ids, scale, out=prefix[:, Ti:])
        self.prefill(prefix)
        return prefix

    def embed_grad(self, ids, dout, vocab: int, scale: float = 1.0, grad=None, accumulate: bool = False, stream=None):
        """Gradient of embed with respect to its table (dm0_embed_grad): f32 [vocab][hidden].

        dout: bf16 or fp32 rows as embed's out.  accumulate adds to `grad`, e.g. to the weight gradient that
        vocab_loss_grad left there when the loss's weights are the table."""
        return self._done(_C.embed_grad(self.h.value or 0, self.device, ids, dout, vocab, scale, grad, accumulate,
                                        _handle(stream)))

    def residual_norm(self, h, y=None, post_gain=None, gate=None, scale: float = 1.0, pre_gain=None, mod_scale=None,
                      mod_shift=None, h_out=None, n_out=None, stream=None):
        """The boundary behind a block (dm0_residual_norm): norm of its output y, gate, scaled residual and the next
        block's norm, in one pass.

        h, y: bf16 or fp32 [T][hidden] or [B][T][hidden]; gains f32 [hidden]; gate, mod_scale, mod_shift f32 [hidden]
        or [B][hidden].  Returns (h_out, n_out bf16, r_post or None, r_pre); the last two are the rows' 1 / rms for
        residual_norm_grad."""
        return self._done(_C.residual_norm(self.h.value or 0, self.device, h, y, post_gain, gate, scale, pre_gain,
                                           mod_scale, mod_shift, h_out, n_out, _handle(stream)))

    def residual_norm_grad(self, dn, dh_out, h_out, y, r_post, r_pre, post_gain=None, gate=None, scale: float = 1.0,
                           pre_gain=None, mod_scale=None, mod_shift=None, stream=None) -> dict:
        """Adjoint of residual_norm (dm0_residual_norm_grad), from its outputs and the gradients dn (bf16 or fp32) of
        n_out and dh_out (the residual's type, or None) of h_out.

        Returns a dict: "h", "y" (their types) and, for each vector that was given, its f32 gradient ("post_gain",
        "gate", "pre_gain", "mod_scale", "mod_shift"), of the vector's shape."""
        return self._done(_C.residual_norm_grad(self.h.value or 0, self.device, dn, dh_out, h_out, y, r_post, r_pre,
                                                post_gain, gate, scale, pre_gain, mod_scale, mod_shift,
                                                _handle(stream)))

    def vocab_loss(self, hidden, weight, targets, stream=None):
        """Softmax cross entropy of hidden @ weight.T against targets without keeping the logits (dm0_vocab_loss).

        hidden: bf16 [tokens][H]; weight: bf16 [vocab][H]; targets: int32 or int64 [tokens], negative: no target.
        Returns (loss, lse), f32 [tokens]; -loss is the target's log probability, lse is for vocab_loss_grad."""
        return self._done(_C.vocab_loss(self.h.value or 0, self.device, hidden, weight, targets, _handle(stream)))

    def vocab_loss_grad(self, hidden, weight, targets, lse, dloss, dhidden=None, dweight=None,
                        accumulate: bool = False, stream=None):
        """Gradients of sum(dloss * loss) of vocab_loss with respect to hidden and weight (dm0_vocab_loss_grad).

        lse, dloss: f32 [tokens].  dhidden [tokens][H] and dweight [vocab][H] are bf16 unless an fp32 tensor is
        given; False leaves that gradient out.  accumulate adds to an fp32 dweight.  The hidden states of tokens without
        a target have to be finite (dweight takes them times zero).  Returns (dhidden, dweight)."""
        return self._done(_C.vocab_loss_grad(self.h.value or 0, self.device, hidden, weight, targets, lse, dloss,
                                             dhidden, dweight, accumulate, _handle(stream)))
