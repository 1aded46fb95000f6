"""Rotary positions: a host-side plan of the angles and the kernel call that
rotates queries and keys (duo_rope_apply), with its gradient for autograd."""
from __future__ import annotations

import torch

from . import _lib as L
from . import _binding as _b

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
        pair_factors = None if pair_factors is None else [float(x) for x in pair_factors]
        self._made_of = (head_dim, theta, rot_dim, layout, scaling, factor, original_len, low, high, magnitude, pair_factors)
        self.d = int(head_dim)
        self.rot_dim = self.d if rot_dim is None else int(rot_dim)
        if pair_factors is not None and len(pair_factors) != self.rot_dim // 2:
            raise ValueError(f"pair_factors: {len(pair_factors)} values, expected {self.rot_dim // 2}")
        desc, _keep = L.make_rope_desc(self.d, self.rot_dim, _LAYOUT[layout], _SCALING[scaling], float(theta),
                                       float(factor), float(original_len), float(low), float(high), float(magnitude),
                                       pair_factors)
        self.handle = L.duo_rope_create(desc)

    def __reduce__(self):
        # a copy has a plan of its own: this one's is freed once
        return type(self), self._made_of

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
    def launch(self, tensors, positions, n_new=None, transpose=False):
        """Rotate (or, with False in third place, only lay out) up to three
        tensors of one batch in one launch: tensors = [(x, out, rotate)], each
        [batch][heads][tokens][d] by strides, the same dtype and device.  An
        out may be its x; otherwise results lie apart from each other and
        from what is read."""
        _b.rope_launch(self.handle or 0, self.d, [(x, o, bool(r)) for x, o, r in tensors], positions, n_new,
                       bool(transpose))

    def apply(self, x, positions, n_new=None, transpose=False, out=None):
        """Rotate x ([batch][heads][tokens][d], any strides in steps of 16
        bytes with contiguous heads; bf16, fp16 or fp32).  positions: int32 [batch] (token i at
        positions[b] + i) or [batch][tokens].  n_new: int32 [batch], only so
        many tokens of each sequence; the rest of out stays as it was (zero
        where out is new).  transpose: the transposed map, i.e. the gradient.
        out may be x (in place).  Differentiable in x (backward mode) where
        out is not given."""
        if (x.requires_grad or out is not None and out.requires_grad) and torch.is_grad_enabled():
            _b.check_recorded(x)
            if out is not None:
                _b.check_recorded(out)
                raise ValueError("out cannot be given where a gradient is recorded")
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
        _b.check_captured_backward(grad)
        positions, *rest = ctx.saved_tensors
        if grad.stride(3) != 1 or any(s * grad.element_size() % 16 for s in grad.stride()[:3]) or \
                grad.data_ptr() % 16:
            grad = grad.clone(memory_format=torch.contiguous_format)     # also where it is contiguous but starts askew
        return ctx.rope._apply(grad, positions, rest[0] if ctx.has_count else None, not ctx.transposed,
                               None), None, None, None, None
