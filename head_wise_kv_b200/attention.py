"""Causal attention of whole sequences with a sliding window and sinks, and
its gradient (duo_window_attn, duo_window_attn_grad): the two branches of the
gated forward in which retrieval heads are told from streaming ones."""
from __future__ import annotations

import torch

from . import _lib as L  # noqa: F401  (raises ImportError where the library is missing)
from . import _binding as _b


def window_attention(q, k, v, sink=0, window=None, lengths=None, scale=None):
    """Causal attention of whole sequences, differentiable in q, k and v.

    q: [batch][query heads][tokens][128], k, v: [batch][key heads][tokens][128],
    bf16 or fp16, any strides (a token-major projection's output is read as
    the view that it is; tensors whose heads are not contiguous, not aligned
    to 16 bytes or expanded are copied).  Row i sees the keys j <= i with
    j < sink or j > i - window; window None: all of them.  lengths: int32
    [batch], tokens of each sequence (default all); results behind them are
    zero, and what the inputs hold there does not matter.  scale: default
    128 ** -0.5; scores, scale |q.k|, stay below 2^23.  The result has q's
    order of dimensions; gradients have their inputs'.  Differentiable once,
    in backward mode.  To capture a backward pass into a graph, capture its
    forward pass with it.  See duo_window_attn."""
    return _b.window_attention(q, k, v, sink, window, lengths, scale)


def window_attention_status(device="cuda", clear=True) -> int:
    """Status bits (DUO_STATUS_WAIT_TIMEOUT) of the calls on a device so far;
    waits for the device's current stream."""
    device = torch.device(device)
    return _b.window_attention_status(torch.cuda.current_device() if device.index is None else device.index, clear)
