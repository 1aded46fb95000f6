"""Causal attention of whole sequences with a sliding window and sinks, and
its gradient (duo_window_attn, duo_window_attn_grad): the two branches of the
gated forward in which retrieval heads are told from streaming ones."""
from __future__ import annotations

import torch

from . import _lib as L
from .cache import _on, _stream

_DTYPE = {torch.bfloat16: L.DUO_BF16, torch.float16: L.DUO_FP16}
_status: dict = {}      # device -> int32 word of the status bits


def _status_word(device):
    word = _status.get(device)
    if word is None:
        word = _status[device] = torch.zeros(1, dtype=torch.int32, device=device)
    return word


def window_attention_status(device="cuda", clear=True) -> int:
    """Status bits (DUO_STATUS_WAIT_TIMEOUT) of the calls on a device so far;
    waits for the device's current stream."""
    device = torch.device(device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    word = _status_word(device)
    bits = int(word.item())
    if clear:
        word.zero_()
    return bits


def _usable(x):
    """x, or a copy of it that the kernels can read: contiguous heads, strides in 16-byte steps, none of them 0."""
    if x.stride(3) != 1 or x.data_ptr() % 16 or any(s % 8 or s < x.shape[3] for s, n in zip(x.stride(), x.shape[:3])
                                                    if n > 1):
        return x.contiguous()
    return x


def _like(x):
    """A new dense tensor with x's shape and order of dimensions (a token-major view gives a token-major one)."""
    order = sorted(range(3), key=lambda i: -x.stride(i)) if x.numel() else [0, 1, 2]
    y = torch.empty([x.shape[i] for i in order] + [x.shape[3]], dtype=x.dtype, device=x.device)
    return y.permute(*[order.index(i) for i in range(3)], 3)


def _heads(x):
    s = x.stride()
    return L.duo_heads(x.data_ptr(), s[0], s[1], s[2])


def _desc(q, k, sink, window, scale, lengths):
    return L.duo_window_attn_desc(_DTYPE[q.dtype], q.shape[0], q.shape[1], k.shape[1], q.shape[3], q.shape[2], sink,
                                  window, scale, lengths.data_ptr() if lengths is not None else None)


class _WindowAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lengths, sink, window, scale):
        q, k, v = _usable(q), _usable(k), _usable(v)
        desc = _desc(q, k, sink, window, scale, lengths)
        out = _like(q)
        with _on(q.device):
            stats = torch.empty(L.duo_window_attn_stats_bytes(desc) // 4, dtype=torch.float32, device=q.device)
            L.duo_window_attn(desc, _heads(q), _heads(k), _heads(v), _heads(out), stats.data_ptr(),
                              _status_word(q.device).data_ptr(), _stream(q.device))
        ctx.save_for_backward(q, k, v, out, stats, lengths)
        ctx.args = sink, window, scale
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        q, k, v, out, stats, lengths = ctx.saved_tensors
        grad = _usable(grad)
        desc = _desc(q, k, *ctx.args, lengths)
        dq, dk, dv = _like(q), _like(k), _like(v)
        with _on(q.device):
            n = L.duo_window_attn_workspace_bytes(desc)
            ws = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
            L.duo_window_attn_grad(desc, _heads(q), _heads(k), _heads(v), _heads(out), _heads(grad), stats.data_ptr(),
                                   _heads(dq), _heads(dk), _heads(dv), ws.data_ptr(), ws.numel(),
                                   _status_word(q.device).data_ptr(), _stream(q.device))
        need = ctx.needs_input_grad
        return dq if need[0] else None, dk if need[1] else None, dv if need[2] else None, None, None, None, None


def window_attention(q, k, v, sink=0, window=None, lengths=None, scale=None):
    """Causal attention of whole sequences, differentiable in q, k and v.

    q: [batch][query heads][tokens][128], k, v: [batch][key heads][tokens][128],
    bf16 or fp16, any strides (a token-major projection's output is read as
    the view that it is; tensors whose heads are not contiguous, not aligned
    to 16 bytes or expanded are copied).  Row i sees the keys j <= i with
    j < sink or j > i - window; window None: all of them.  lengths: int32
    [batch], tokens of each sequence (default all); results behind them are
    zero, and what the inputs hold there does not matter.  scale: default
    128 ** -0.5.  The result has q's order of dimensions; gradients have their
    inputs'.  See duo_window_attn."""
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype not in _DTYPE or t.dtype != q.dtype:
            raise TypeError(f"{name}: dtype {t.dtype}, expected bfloat16 or float16, the same for q, k and v")
        if t.device.type != "cuda" or t.device != q.device:
            raise ValueError(f"{name}: on {t.device}, expected one CUDA device for q, k and v")
        if t.dim() != 4:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [batch][heads][tokens][128]")
    B, hq, T, d = q.shape
    if k.shape != v.shape or (k.shape[0], k.shape[2], k.shape[3]) != (B, T, d):
        raise ValueError(f"k, v: shapes {tuple(k.shape)}, {tuple(v.shape)}, expected ({B}, key heads, {T}, {d})")
    if d != 128:
        raise ValueError(f"heads of {d} elements, expected 128")
    if k.shape[1] < 1 or hq % k.shape[1] or hq < 1:
        raise ValueError(f"{hq} query heads over {k.shape[1]} key heads")
    if sink < 0 or (window is not None and window < 1):
        raise ValueError("sink must be at least 0 and window at least 1 (or None)")
    if lengths is not None and (lengths.dtype != torch.int32 or lengths.device != q.device or
                                tuple(lengths.shape) != (B,) or not lengths.is_contiguous()):
        raise ValueError(f"lengths must be contiguous int32 [{B}] on the tensors' device")
    scale = d ** -0.5 if scale is None else float(scale)
    if not 0 < scale < 1e30:
        raise ValueError("scale must be above 0")
    top = 2 ** 31 - 1
    return _WindowAttention.apply(q, k, v, lengths, min(int(sink), top), 0 if window is None else min(int(window), top),
                                  scale)
