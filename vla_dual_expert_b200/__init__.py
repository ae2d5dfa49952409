"""DM0 dual-expert merged-attention inference on B200 (sm_100a).

Python face of the C ABI in include/dm0.h.  `Engine` owns one dm0_ctx and
takes torch CUDA tensors (or host numpy arrays for `infer_host`); it only
passes their pointers, sizes and the current CUDA stream to the library.
"""
from __future__ import annotations

import ctypes

import numpy as np

from ._abi import (EXPORTS, LIB_PATH, SITES, Dm0Config, Dm0Error, Dm0Norm, Dm0NormGrads,  # noqa: F401
                   load_library, make_config, pack_weights)

__all__ = ["Engine", "Dm0Error", "pack_weights", "pack_e4m3_rows", "load_library", "EXPORTS", "LIB_PATH"]


c_int_t = ctypes.c_int


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check_cuda(t, dtype, shape, name):
    import torch
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous CUDA {dtype} tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_on(t, device, dtypes, shape, name):
    """A contiguous tensor of `shape` and one of `dtypes` on CUDA device `device` (the context's)."""
    if not (t.is_cuda and t.get_device() == device and t.dtype in dtypes and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous tensor on cuda:{device} of {' or '.join(map(str, dtypes))}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_rows(t, device, dtypes, shape, name):
    """As _check_on for [T][H] or [B][T][H] rows that are contiguous themselves: (batch stride, row stride)."""
    if not (t.is_cuda and t.get_device() == device and t.dtype in dtypes):
        raise TypeError(f"{name} must be a tensor on cuda:{device} of {' or '.join(map(str, dtypes))}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.stride(-1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    # the stride of a dimension of one says nothing
    return (t.stride(0) if t.dim() == 3 and t.shape[0] > 1 else 0), (t.stride(-2) if t.shape[-2] > 1 else t.shape[-1])


def pack_e4m3_rows(x: np.ndarray):
    """FP8 E4M3 codes (uint8, OCP bit patterns) and one fp32 scale per row of a 2-D array, through
    dm0_pack_e4m3_rows (host code; no GPU needed)."""
    lib = load_library()
    a = np.ascontiguousarray(x, np.float32)
    if a.ndim != 2:
        raise ValueError("pack_e4m3_rows expects a 2-D array")
    codes = np.empty(a.shape, np.uint8)
    scales = np.empty(a.shape[0], np.float32)
    st = lib.dm0_pack_e4m3_rows(a.ctypes.data, a.shape[0], a.shape[1], codes.ctypes.data, scales.ctypes.data)
    if st != 0:
        raise Dm0Error(st, "dm0_pack_e4m3_rows")
    return codes, scales


class Engine:
    """One dm0_ctx on the current CUDA device."""

    def __init__(self, dims, max_batch: int, max_prefix: int, time_mod: bool = False):
        """time_mod: the time-modulated action expert (DM0.5 page, section 5.2) instead of the DM0 one."""
        self.lib = load_library()
        self.dims = dims
        self.time_mod = bool(time_mod)
        self.cfg = make_config(dims, max_batch, max_prefix, self.time_mod)
        h = ctypes.c_void_p()
        st = self.lib.dm0_create(ctypes.byref(self.cfg), ctypes.byref(h))
        if st != 0 or not h.value:
            raise Dm0Error(st, "dm0_create failed (configuration or device allocation)")
        self.h = h
        import torch
        self.device = torch.cuda.current_device()   # the context's: tensors of the language operators live there

    # ------------------------------------------------------------------ helpers
    def _chk(self, st: int):
        if st != 0:
            raise Dm0Error(st, self.lib.dm0_last_error(self.h).decode())

    def close(self):
        if getattr(self, "h", None) is not None and self.h.value:
            self.lib.dm0_destroy(self.h)
            self.h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ API
    def weights_bytes(self) -> int:
        return int(self.lib.dm0_weights_bytes(ctypes.byref(self.cfg)))

    def load_weights(self, blob: np.ndarray):
        blob = np.ascontiguousarray(blob, dtype=np.uint8)
        self._chk(self.lib.dm0_load_weights(self.h, blob.ctypes.data_as(ctypes.c_void_p), blob.nbytes))

    def load_from(self, provider):
        self.load_weights(pack_weights(provider, self.dims.layers, self.time_mod))

    def prefill(self, prefix_emb, stream=None):
        import torch
        B, P = prefix_emb.shape[:2]
        _check_cuda(prefix_emb, torch.bfloat16, (B, P, self.dims.hidden_v), "prefix_emb")
        self._chk(self.lib.dm0_prefill(self.h, _ptr(prefix_emb), B, P, _stream(stream)))

    def prepare(self, B: int, P: int, steps: int):
        """Capture ahead of time what dm0_denoise needs for (B, P, steps) (dm0_prepare)."""
        self._chk(self.lib.dm0_prepare(self.h, B, P, steps))

    def kv_view(self):
        k, v = ctypes.c_void_p(), ctypes.c_void_p()
        self._chk(self.lib.dm0_kv_view(self.h, ctypes.byref(k), ctypes.byref(v)))
        return k.value, v.value

    def kv_commit(self, B: int, P: int):
        self._chk(self.lib.dm0_kv_commit(self.h, B, P))

    def denoise(self, noise, steps: int, actions=None, velocities=None, stream=None):
        import torch
        _check_cuda(noise, torch.float32, noise.shape, "noise")
        if actions is None:
            actions = torch.empty_like(noise)
        _check_cuda(actions, torch.float32, noise.shape, "actions")
        if velocities is not None:
            _check_cuda(velocities, torch.float32, (steps,) + tuple(noise.shape), "velocities")
        self._chk(self.lib.dm0_denoise(self.h, _ptr(noise), steps, _ptr(actions), _ptr(velocities),
                                       _stream(stream)))
        return actions

    def infer_host(self, prefix_bits: np.ndarray, noise: np.ndarray, steps: int, actions: np.ndarray = None,
                   stream=None) -> np.ndarray:
        """prefix_bits: host uint16 bf16 bit patterns [B][P][Hv]; noise: host f32 [B][S][A]."""
        B, P = prefix_bits.shape[:2]
        if actions is None:
            actions = np.empty_like(noise, dtype=np.float32)
        self._chk(self.lib.dm0_infer_host(self.h, prefix_bits.ctypes.data_as(ctypes.c_void_p),
                                          noise.ctypes.data_as(ctypes.c_void_p), B, P, steps,
                                          actions.ctypes.data_as(ctypes.c_void_p), _stream(stream)))
        return actions

    def merged_layer(self, layer, h_prefix, h_suffix, out_prefix, out_suffix, k_out, v_out, stream=None):
        import torch
        d = self.dims
        B, P = h_prefix.shape[:2]
        _check_cuda(h_prefix, torch.float32, (B, P, d.hidden_v), "h_prefix")
        _check_cuda(h_suffix, torch.float32, (B, d.chunk, d.hidden_a), "h_suffix")
        _check_cuda(out_prefix, torch.float32, (B, P, d.hidden_v), "out_prefix")
        _check_cuda(out_suffix, torch.float32, (B, d.chunk, d.hidden_a), "out_suffix")
        _check_cuda(k_out, torch.bfloat16, (B, d.n_kv, P, d.head_dim), "k_out")
        _check_cuda(v_out, torch.bfloat16, (B, d.n_kv, P, d.head_dim), "v_out")
        self._chk(self.lib.dm0_merged_layer(self.h, layer, _ptr(h_prefix), _ptr(h_suffix), B, P, _ptr(out_prefix),
                                            _ptr(out_suffix), _ptr(k_out), _ptr(v_out), _stream(stream)))

    def op_gemm(self, A, B, C, swap=0, splits=1, stream=None):
        import torch
        M, K = A.shape
        N = B.shape[0]
        _check_cuda(A, torch.bfloat16, (M, K), "A")
        _check_cuda(B, torch.bfloat16, (N, K), "B")
        _check_cuda(C, torch.float32, (N, M) if swap else (M, N), "C")
        self._chk(self.lib.dm0_op_gemm(self.h, _ptr(A), _ptr(B), _ptr(C), M, N, K, swap, splits, _stream(stream)))

    def grad_floats(self) -> int:
        return int(self.lib.dm0_grad_floats(ctypes.byref(self.cfg)))

    def train_step(self, a, eps, t, mask, grads=None, kv_grads=None, stream=None):
        """One flow-matching training step (dm0_train_step) over the context's prefix cache.

        a, eps: CUDA f32 [B][chunk][A]; t: CUDA f32 [B]; mask: CUDA uint8 [B][chunk][A].  Returns (loss
        [1], grads [grad_floats]) as CUDA f32 tensors; kv_grads, when given, is CUDA f32
        [2][layers][B][n_kv][P][head_dim] and receives the cache gradients."""
        import torch
        B = a.shape[0]
        d = self.dims
        shape = (B, d.chunk, d.action_dim)
        _check_cuda(a, torch.float32, shape, "a")
        _check_cuda(eps, torch.float32, shape, "eps")
        _check_cuda(t, torch.float32, (B,), "t")
        _check_cuda(mask, torch.uint8, shape, "mask")
        if grads is None:
            grads = torch.empty(self.grad_floats(), device=a.device, dtype=torch.float32)
        _check_cuda(grads, torch.float32, (self.grad_floats(),), "grads")
        loss = torch.empty(1, device=a.device, dtype=torch.float32)
        self._chk(self.lib.dm0_train_step(self.h, _ptr(a), _ptr(eps), _ptr(t), _ptr(mask), _ptr(loss), _ptr(grads),
                                          _ptr(kv_grads), _stream(stream)))
        return loss, grads

    def set_prefix_fp8(self, enable: bool = True, stream=None):
        """Run the VLM MLP's gate/up and down GEMMs in FP8 E4M3 (dm0_set_prefix_fp8)."""
        self._chk(self.lib.dm0_set_prefix_fp8(self.h, 1 if enable else 0, _stream(stream)))

    def op_quant_e4m3(self, x, codes, scales, gain=None, ssq=None, stream=None):
        import torch
        rows, cols = x.shape
        f32 = x.dtype == torch.float32
        _check_cuda(x, torch.float32 if f32 else torch.bfloat16, (rows, cols), "x")
        _check_cuda(codes, torch.uint8, (rows, cols), "codes")
        _check_cuda(scales, torch.float32, (rows,), "scales")
        if gain is not None:
            _check_cuda(gain, torch.float32, (cols,), "gain")
        if ssq is not None:
            _check_cuda(ssq, torch.float32, (rows,), "ssq")
        self._chk(self.lib.dm0_op_quant_e4m3(self.h, _ptr(x), int(f32), rows, cols, _ptr(gain), _ptr(ssq),
                                             _ptr(codes), _ptr(scales), _stream(stream)))

    def op_gemm_e4m3(self, A, sa, B, sb, C, stream=None):
        import torch
        M, K = A.shape
        N = B.shape[0]
        _check_cuda(A, torch.uint8, (M, K), "A")
        _check_cuda(B, torch.uint8, (N, K), "B")
        _check_cuda(sa, torch.float32, (M,), "sa")
        _check_cuda(sb, torch.float32, (N,), "sb")
        _check_cuda(C, torch.float32, (M, N), "C")
        self._chk(self.lib.dm0_op_gemm_e4m3(self.h, _ptr(A), _ptr(sa), _ptr(B), _ptr(sb), _ptr(C), M, N, K,
                                            _stream(stream)))

    def op_attention(self, q, ka, va, kb, vb, o, splits=1, stream=None):
        import torch
        for t, nm in ((q, "q"), (ka, "ka"), (va, "va"), (kb, "kb"), (vb, "vb"), (o, "o")):
            if t is not None:
                _check_cuda(t, torch.bfloat16, t.shape, nm)
        B, Tq = q.shape[:2]
        Ta = ka.shape[2]
        Tb = 0 if kb is None else kb.shape[2]
        self._chk(self.lib.dm0_op_attention(self.h, _ptr(q), _ptr(ka), _ptr(va), Ta, _ptr(kb), _ptr(vb), Tb,
                                            _ptr(o), B, Tq, splits, _stream(stream)))

    # ------------------------------------------------------------------ language side
    def _ids(self, ids, name):
        import torch
        if ids.dim() not in (1, 2):
            raise ValueError(f"{name} must be [T] or [B][T]")
        _check_on(ids, self.device, (torch.int64, torch.int32), ids.shape, name)
        return ids.dtype == torch.int64, (1 if ids.dim() == 1 else ids.shape[0]), ids.shape[-1]

    def embed(self, table, ids, scale: float = 1.0, out=None, stream=None):
        """scale * table[ids] (dm0_embed), a zero row where an id is negative.

        table: CUDA bf16 [vocab][hidden]; ids: int32 or int64 [T] or [B][T]; out (bf16, made if not given, or fp32):
        [T][hidden] or [B][T][hidden], whose rows are contiguous but may lie apart, as the text rows behind the
        image rows of a prefix do: out=prefix_emb[:, image_rows:]."""
        import torch
        wide, B, T = self._ids(ids, "ids")
        if table.dim() != 2:
            raise ValueError("table must be [vocab][hidden]")
        V, H = table.shape
        _check_on(table, self.device, (torch.bfloat16,), table.shape, "table")
        shape = (*ids.shape, H)
        if out is None:
            out = torch.empty(shape, device=table.device, dtype=torch.bfloat16)
        bs, rs = _check_rows(out, self.device, (torch.bfloat16, torch.float32), shape, "out")
        self._chk(self.lib.dm0_embed(self.h, _ptr(table), _ptr(ids), wide, B, T, V, H, scale, _ptr(out),
                                     out.dtype == torch.float32, bs, rs, _stream(stream)))
        return out

    def embed_grad(self, ids, dout, vocab: int, scale: float = 1.0, grad=None, accumulate: bool = False, stream=None):
        """Gradient of embed with respect to its table (dm0_embed_grad): f32 [vocab][hidden].

        dout: bf16 or fp32 rows as embed's out.  accumulate adds to `grad`, e.g. to the weight gradient that
        vocab_loss_grad left there when the loss's weights are the table."""
        import torch
        wide, B, T = self._ids(ids, "ids")
        H = dout.shape[-1]
        bs, rs = _check_rows(dout, self.device, (torch.bfloat16, torch.float32), (*ids.shape, H), "dout")
        if grad is None:
            if accumulate:
                raise ValueError("accumulate needs grad")
            grad = torch.empty((vocab, H), device=dout.device, dtype=torch.float32)
        _check_on(grad, self.device, (torch.float32,), (vocab, H), "grad")
        ws = self._workspace(self.lib.dm0_embed_grad_workspace(B, T, vocab, H), stream)
        self._chk(self.lib.dm0_embed_grad(self.h, _ptr(ids), wide, B, T, vocab, H, scale, _ptr(dout),
                                          dout.dtype == torch.float32, bs, rs, _ptr(grad), accumulate, _ptr(ws),
                                          ws.numel(), _stream(stream)))
        return grad

    def _workspace(self, nbytes: int, stream):
        """Scratch of one call, from torch's allocator, which keeps it from others until the call's stream is past it."""
        import torch
        ws = torch.empty(max(nbytes, 16), device=f"cuda:{self.device}", dtype=torch.uint8)
        if stream is not None:
            ws.record_stream(stream if isinstance(stream, torch.cuda.Stream) else
                             torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), self.device))
        return ws

    def _norm(self, h, y, post_gain, gate, scale, pre_gain, mod_scale, mod_shift):
        import torch
        two = (torch.float32, torch.bfloat16)
        if h.dim() not in (2, 3):
            raise ValueError("the residual stream must be [T][hidden] or [B][T][hidden]")
        B, T, H = (1, *h.shape) if h.dim() == 2 else h.shape
        _check_on(h, self.device, two, h.shape, "the residual stream")
        if y is not None:
            _check_on(y, self.device, two, h.shape, "y")
        for v, name in ((post_gain, "post_gain"), (pre_gain, "pre_gain")):
            if v is not None:
                _check_on(v, self.device, (torch.float32,), (H,), name)
        strides = {}
        for v, name in ((gate, "gate"), (mod_scale, "mod_scale"), (mod_shift, "mod_shift")):
            strides[name] = 0
            if v is None:
                continue
            if not (v.is_cuda and v.get_device() == self.device and v.dtype == torch.float32 and v.stride(-1) == 1):
                raise TypeError(f"{name} must be an fp32 tensor on cuda:{self.device} with contiguous rows")
            if v.shape != (H,) and v.shape != (B, H):
                raise ValueError(f"{name} has shape {tuple(v.shape)}, expected {(H,)} or {(B, H)}")
            strides[name] = v.stride(0) if v.dim() == 2 and B > 1 else 0
            if v.dim() == 2 and B > 1 and v.stride(0) < H:
                raise ValueError(f"the rows of {name} overlap")
        if mod_scale is not None and mod_shift is not None and strides["mod_scale"] != strides["mod_shift"]:
            raise ValueError("mod_scale and mod_shift must be laid out alike")
        return Dm0Norm(B, T, H, h.dtype == torch.float32, y is not None and y.dtype == torch.float32, scale,
                       _ptr(post_gain), _ptr(gate), strides["gate"], _ptr(pre_gain), _ptr(mod_scale),
                       _ptr(mod_shift), max(strides["mod_scale"], strides["mod_shift"]))

    def residual_norm(self, h, y=None, post_gain=None, gate=None, scale: float = 1.0, pre_gain=None, mod_scale=None,
                      mod_shift=None, h_out=None, n_out=None, stream=None):
        """The boundary behind a block (dm0_residual_norm): norm of its output y, gate, scaled residual and the next
        block's norm, in one pass.

        h, y: bf16 or fp32 [T][hidden] or [B][T][hidden]; gains f32 [hidden]; gate, mod_scale, mod_shift f32 [hidden]
        or [B][hidden].  Returns (h_out, n_out bf16, r_post or None, r_pre); the last two are the rows' 1 / rms for
        residual_norm_grad."""
        import torch
        a = self._norm(h, y, post_gain, gate, scale, pre_gain, mod_scale, mod_shift)
        if h_out is None:
            h_out = torch.empty_like(h)
        if n_out is None:
            n_out = torch.empty_like(h, dtype=torch.bfloat16)
        _check_on(h_out, self.device, (h.dtype,), h.shape, "h_out")
        _check_on(n_out, self.device, (torch.bfloat16,), h.shape, "n_out")
        r_pre = torch.empty(h.shape[:-1], device=h.device, dtype=torch.float32)
        r_post = torch.empty_like(r_pre) if post_gain is not None else None
        self._chk(self.lib.dm0_residual_norm(self.h, ctypes.byref(a), _ptr(h), _ptr(y), _ptr(h_out), _ptr(n_out),
                                             _ptr(r_post), _ptr(r_pre), _stream(stream)))
        return h_out, n_out, r_post, r_pre

    def residual_norm_grad(self, dn, dh_out, h_out, y, r_post, r_pre, post_gain=None, gate=None, scale: float = 1.0,
                           pre_gain=None, mod_scale=None, mod_shift=None, stream=None) -> dict:
        """Adjoint of residual_norm (dm0_residual_norm_grad), from its outputs and the gradients dn (bf16 or fp32) of
        n_out and dh_out (the residual's type, or None) of h_out.

        Returns a dict: "h", "y" (their types) and, for each vector that was given, its f32 gradient ("post_gain",
        "gate", "pre_gain", "mod_scale", "mod_shift"), of the vector's shape."""
        import torch
        a = self._norm(h_out, y, post_gain, gate, scale, pre_gain, mod_scale, mod_shift)
        _check_on(dn, self.device, (torch.bfloat16, torch.float32), h_out.shape, "dn")
        if dh_out is not None:
            _check_on(dh_out, self.device, (h_out.dtype,), h_out.shape, "dh_out")
        for r, name in ((r_pre, "r_pre"), (r_post, "r_post")):
            if r is not None:
                _check_on(r, self.device, (torch.float32,), h_out.shape[:-1], name)
        out = {"h": torch.empty_like(h_out)}
        if y is not None:
            out["y"] = torch.empty_like(y)
        vecs = {"post_gain": post_gain, "gate": gate, "pre_gain": pre_gain, "mod_scale": mod_scale,
                "mod_shift": mod_shift}
        out.update((k, torch.empty(v.shape, device=v.device, dtype=torch.float32)) for k, v in vecs.items()
                   if v is not None)
        g = Dm0NormGrads(*(_ptr(out.get(k)) for k in vecs))
        ws = self._workspace(self.lib.dm0_residual_norm_grad_workspace(ctypes.byref(a)), stream)
        self._chk(self.lib.dm0_residual_norm_grad(
            self.h, ctypes.byref(a), _ptr(dn), dn.dtype == torch.float32, _ptr(dh_out), _ptr(h_out), _ptr(y),
            _ptr(r_post), _ptr(r_pre), _ptr(out["h"]), _ptr(out.get("y")), ctypes.byref(g), _ptr(ws), ws.numel(),
            _stream(stream)))
        return out

    def _vocab(self, hidden, weight, targets):
        import torch
        if hidden.dim() != 2 or weight.dim() != 2 or targets.dim() != 1:
            raise ValueError("hidden must be [tokens][H], weight [vocab][H] and targets [tokens]")
        N, H = hidden.shape
        V = weight.shape[0]
        _check_on(hidden, self.device, (torch.bfloat16,), (N, H), "hidden")
        _check_on(weight, self.device, (torch.bfloat16,), (V, H), "weight")
        _check_on(targets, self.device, (torch.int64, torch.int32), (N,), "targets")
        return N, V, H, targets.dtype == torch.int64

    def vocab_loss(self, hidden, weight, targets, stream=None):
        """Softmax cross entropy of hidden @ weight.T against targets without keeping the logits (dm0_vocab_loss).

        hidden: bf16 [tokens][H]; weight: bf16 [vocab][H]; targets: int32 or int64 [tokens], negative: no target.
        Returns (loss, lse), f32 [tokens]; -loss is the target's log probability, lse is for vocab_loss_grad."""
        import torch
        N, V, H, wide = self._vocab(hidden, weight, targets)
        out = torch.empty((2, N), device=hidden.device, dtype=torch.float32)
        loss, lse = out[0], out[1]
        ws = self._workspace(self.lib.dm0_vocab_loss_workspace(N, V, H), stream)
        self._chk(self.lib.dm0_vocab_loss(self.h, _ptr(hidden), _ptr(weight), _ptr(targets), wide, N, V, H, _ptr(loss),
                                          _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))
        return loss, lse

    def vocab_loss_grad(self, hidden, weight, targets, lse, dloss, dhidden=None, dweight=None,
                        accumulate: bool = False, stream=None):
        """Gradients of sum(dloss * loss) of vocab_loss with respect to hidden and weight (dm0_vocab_loss_grad).

        lse, dloss: f32 [tokens].  dhidden [tokens][H] and dweight [vocab][H] are bf16 unless an fp32 tensor is
        given; False leaves that gradient out.  accumulate adds to an fp32 dweight.  Returns (dhidden, dweight)."""
        import torch
        N, V, H, wide = self._vocab(hidden, weight, targets)
        _check_on(lse, self.device, (torch.float32,), (N,), "lse")
        _check_on(dloss, self.device, (torch.float32,), (N,), "dloss")
        if accumulate and not isinstance(dweight, torch.Tensor):
            raise ValueError("accumulate needs dweight")
        grads = []
        for t, like, name in ((dhidden, hidden, "dhidden"), (dweight, weight, "dweight")):
            if t is None:
                t = torch.empty_like(like)
            elif t is False:
                t = None
            if t is not None:
                _check_on(t, self.device, (torch.bfloat16, torch.float32), like.shape, name)
            grads.append(t)
        dh, dw = grads
        ws = self._workspace(self.lib.dm0_vocab_loss_grad_workspace(N, V, H), stream)
        self._chk(self.lib.dm0_vocab_loss_grad(
            self.h, _ptr(hidden), _ptr(weight), _ptr(targets), wide, _ptr(lse), _ptr(dloss), N, V, H, _ptr(dh),
            dh is not None and dh.dtype == torch.float32, _ptr(dw), dw is not None and dw.dtype == torch.float32,
            accumulate, _ptr(ws), ws.numel(), _stream(stream)))
        return dh, dw

    def debug_view(self, name: str) -> int:
        """Device address of an internal activation buffer (see dm0_debug_view)."""
        p = ctypes.c_void_p()
        self._chk(self.lib.dm0_debug_view(self.h, name.encode(), ctypes.byref(p)))
        return p.value

    def launch_count(self) -> int:
        return int(self.lib.dm0_launch_count(self.h))

    def probe(self, site_mask: int):
        self._chk(self.lib.dm0_probe(self.h, site_mask))

    def probe_read(self, site: int):
        n, ms = c_int_t(), ctypes.c_double()
        self._chk(self.lib.dm0_probe_read(self.h, site, ctypes.byref(n), ctypes.byref(ms)))
        return n.value, ms.value

    def selftest_timeout(self, limit_us: int = 20000, stream=None):
        self._chk(self.lib.dm0_selftest_timeout(self.h, limit_us, _stream(stream)))

    def sync(self, stream=None):
        self._chk(self.lib.dm0_sync(self.h, _stream(stream)))

    def device_error(self) -> int:
        return int(self.lib.dm0_device_error(self.h))

    def clear_error(self):
        self._chk(self.lib.dm0_clear_error(self.h))
