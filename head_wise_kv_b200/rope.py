"""Rotary positions: a host-side plan of the angles and the kernel call that
rotates queries and keys (duo_rope_apply), with its gradient for autograd."""
from __future__ import annotations

import torch

from . import _lib as L
from . import _binding as _b

_DTYPE = {torch.bfloat16: L.DUO_BF16, torch.float16: L.DUO_FP16, torch.float32: L.DUO_FP32}
_LAYOUT = {"half": L.DUO_ROPE_HALF, "interleaved": L.DUO_ROPE_INTERLEAVED}
_SCALING = {"none": L.DUO_ROPE_NONE, "linear": L.DUO_ROPE_LINEAR, "ntk": L.DUO_ROPE_NTK, "yarn": L.DUO_ROPE_YARN,
            "bands": L.DUO_ROPE_BANDS, "factors": L.DUO_ROPE_FACTORS}


class Rope:
    """Rotary positions of heads of ``head_dim`` (64 or 128) elements.

    rot_dim: elements that rotate, the first ones (a multiple of 16; default
    all).  layout: pairs "half" (i, i + rot_dim / 2) or "interleaved" (2i,
    2i + 1).  scaling, for contexts beyond the one trained on: "none",
    "linear", "ntk", "yarn", "bands" or "factors" (pair_factors, one per
    pair); factor, original_len, low, high and magnitude as in duo_rope_desc.
    """

    def __init__(self, head_dim, theta=10000.0, rot_dim=None, layout="half", scaling="none", factor=1.0,
                 original_len=0, low=0.0, high=0.0, magnitude=0.0, pair_factors=None):
        if layout not in _LAYOUT:
            raise ValueError(f"layout must be one of {sorted(_LAYOUT)}")
        if scaling not in _SCALING:
            raise ValueError(f"scaling must be one of {sorted(_SCALING)}")
        self.handle = None
        self.d = int(head_dim)
        self.rot_dim = self.d if rot_dim is None else int(rot_dim)
        if pair_factors is not None and len(pair_factors) != self.rot_dim // 2:
            raise ValueError(f"pair_factors: {len(pair_factors)} values, expected {self.rot_dim // 2}")
        desc, _keep = L.make_rope_desc(self.d, self.rot_dim, _LAYOUT[layout], _SCALING[scaling], float(theta),
                                       float(factor), float(original_len), float(low), float(high), float(magnitude),
                                       pair_factors)
        self.handle = L.duo_rope_create(desc)

    def close(self):
        if getattr(self, "handle", None):
            L.duo_rope_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def frequencies(self):
        """(angles per position in radians [rot_dim / 2], magnitude)."""
        return L.duo_rope_frequencies(self.handle, self.rot_dim)

    # ------------------------------------------------------------------ the call
    def _entry(self, x, out, rotate=1):
        if x.dim() != 4 or x.shape[3] != self.d:
            raise ValueError(f"shape {tuple(x.shape)}, expected [batch][heads][tokens][{self.d}]")
        if out.shape != x.shape or out.dtype != x.dtype or out.device != x.device:
            raise ValueError("out must have the input's shape, dtype and device")
        if x.stride(3) != 1 or out.stride(3) != 1:
            raise ValueError("the elements of a head must be contiguous")
        # a dimension of one entry has no stride that matters
        xs, os = ([t.stride(i) if t.shape[i] > 1 else 0 for i in range(3)] for t in (x, out))
        return L.duo_rope_tensor(x.data_ptr(), out.data_ptr(), x.shape[1], rotate, (L._I64 * 3)(*xs),
                                 (L._I64 * 3)(*os))

    def launch(self, tensors, positions, n_new=None, transpose=False):
        """Rotate (or, with False in third place, only lay out) up to three
        tensors of one batch in one launch: tensors = [(x, out, rotate)], each
        [batch][heads][tokens][d] by strides, the same dtype and device."""
        x0 = tensors[0][0]
        dt = _DTYPE.get(x0.dtype)
        if dt is None:
            raise TypeError(f"dtype {x0.dtype}, expected bfloat16, float16 or float32")
        dev, B, n = x0.device, x0.shape[0], x0.shape[2]
        if dev.type != "cuda":
            raise ValueError("the tensors must be on a CUDA device")
        for x, _, _ in tensors[1:]:
            if x.dtype != x0.dtype or x.device != dev or x.shape[0] != B or x.shape[2] != n:
                raise ValueError("tensors of one launch share dtype, device, batch and tokens")
        per_token = positions.dim() == 2
        if positions.dtype != torch.int32 or positions.device != dev or not positions.is_contiguous():
            raise ValueError("positions must be contiguous int32 on the tensors' device")
        if tuple(positions.shape) != ((B, n) if per_token else (B,)):
            raise ValueError(f"positions: shape {tuple(positions.shape)}, expected ({B},) or ({B}, {n})")
        if n_new is not None and (n_new.dtype != torch.int32 or n_new.device != dev or tuple(n_new.shape) != (B,)
                                  or not n_new.is_contiguous()):
            raise ValueError(f"n_new must be contiguous int32 [{B}] on the tensors' device")
        arr = (L.duo_rope_tensor * len(tensors))(*[self._entry(x, o, int(bool(r))) for x, o, r in tensors])
        if torch.cuda.current_device() == dev.index:
            self._call(dt, transpose, B, n, arr, positions, per_token, n_new, dev)
        else:
            with torch.cuda.device(dev):
                self._call(dt, transpose, B, n, arr, positions, per_token, n_new, dev)

    def _call(self, dt, transpose, B, n, arr, positions, per_token, n_new, dev):
        L.duo_rope_apply(self.handle, dt, int(bool(transpose)), B, n, arr, positions.data_ptr(), int(per_token),
                         n_new.data_ptr() if n_new is not None else None, torch.cuda.current_stream(dev).cuda_stream)

    def apply(self, x, positions, n_new=None, transpose=False, out=None):
        """Rotate x ([batch][heads][tokens][d], any strides with contiguous
        heads; bf16, fp16 or fp32).  positions: int32 [batch] (token i at
        positions[b] + i) or [batch][tokens].  n_new: int32 [batch], only so
        many tokens of each sequence; the rest of out stays as it was (zero
        where out is new).  transpose: the transposed map, i.e. the gradient.
        out may be x (in place).  Differentiable in x where out is not given."""
        if x.requires_grad and torch.is_grad_enabled():
            if out is not None:
                raise ValueError("out cannot be given where a gradient is recorded")
            _b.check_capture(x)
            return _RopeFunction.apply(x, positions, n_new, self, bool(transpose))
        return self._apply(x, positions, n_new, transpose, out)

    def _apply(self, x, positions, n_new, transpose, out):
        return _b.rope_apply(self.handle or 0, self.d, x, positions, n_new, transpose, out)


class _RopeFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, n_new, rope, transpose):
        ctx.rope, ctx.transposed, ctx.has_count = rope, transpose, n_new is not None
        ctx.save_for_backward(positions, *([n_new] if n_new is not None else []))
        return rope._apply(x, positions, n_new, transpose, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        positions, *rest = ctx.saved_tensors
        if grad.stride(3) != 1 or any(s * grad.element_size() % 16 for s in grad.stride()[:3]) or \
                grad.data_ptr() % 16:
            grad = grad.contiguous()
        return ctx.rope._apply(grad, positions, rest[0] if ctx.has_count else None, not ctx.transposed,
                               None), None, None, None, None
