"""Windowed attention and its gradient on the GPU against the fp64 oracle.

Bounds, element by element, worked out in fp64 beside the reference.  u is
half a step of the type (2^-8 for bf16, 2^-11 for fp16).

* Scores: 128 exact products summed in fp32, at most 2^-23 of the sum of
  magnitudes per addition, so es = scale 2^-16 max sum |q k|, and a softmax
  weight is off by at most ep = 2 es + 2^-18 of itself (the fast exponential
  2^-22 relative for arguments up to 2^4, the sum's roundings).
* out: weights rounded once (u p), the result once (u |out|):
    Eo = (u + ep) p|v| + u |out|.
* dv: Ev = (u + ep) p^T|g| + u |dv|.
* ds = p (g.v - D): D is the dot of g with the rounded out, so
    Es = p (2^-16 |g|.|v| + |g|.Eo) + (u + ep) |ds|;
  dq, dk: scale Es |k|, scale Es^T |q| (and 2^-16 of the magnitudes for the
  fp32 sums), plus u of the result.
fp16 has a smallest step: 2^-24 for each rounded weight, ds and result.
"""
import numpy as np
import pytest
import torch

from oracle import duo_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _reference(q, k, v, g, sees, scale, dtype):
    """(values, bounds) of (out, dq, dk, dv) for one head of fp64 arrays."""
    u = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0
    n = int(sees.any(1).sum())
    q, k, v, g = (np.where(np.arange(len(x))[:, None] < n, x, 0.0) for x in (q, k, v, g))
    out, p = O.window_attention(q, k, v, sees, scale)
    dq, dk, dv = O.window_attention_grad(q, k, v, g, sees, scale)
    aq, ak, av, ag = (np.abs(x) for x in (q, k, v, g))
    ep = 2 * scale * 2.0 ** -16 * float((aq @ ak.T).max()) + 2.0 ** -18
    seen = sees.astype(np.float64)
    eo = (u + ep) * (p @ av) + u * np.abs(out) + tiny * (1 + seen @ av)
    ev = (u + ep) * (p.T @ ag) + u * np.abs(dv) + tiny * (1 + seen.T @ ag)
    ds = p * (g @ v.T - (g * out).sum(1, keepdims=True))
    es = p * (2.0 ** -16 * (ag @ av.T) + (ag * eo).sum(1, keepdims=True)) + (u + ep) * np.abs(ds) + tiny * seen
    mag = 2.0 ** -16 * np.abs(ds)
    eq = scale * (es + mag) @ ak + u * np.abs(dq) + tiny
    ek = scale * (es + mag).T @ aq + u * np.abs(dk) + tiny
    return (out, dq, dk, dv), (eo, eq, ek, ev)


def _check(q, k, v, g, got, sink, window, lengths, scale, heads=None):
    """got: (out, dq, dk, dv) tensors."""
    B, hq, T, _ = q.shape
    n_kv = k.shape[1]
    G = hq // n_kv
    x64 = [x.detach().double().cpu().numpy() for x in (q, k, v, g)]
    res = [x.detach().double().cpu().numpy() for x in got]
    assert all(np.isfinite(x).all() for x in res)
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        sees = O.window_visible(T, sink, window or 0, n)
        for kv in range(n_kv):
            dk = dv = ek = ev = 0.0
            for h in range(kv * G, kv * G + G):
                (out, dq, a, c), (eo, eq, ea, ec) = _reference(x64[0][b, h], x64[1][b, kv], x64[2][b, kv], x64[3][b, h],
                                                               sees, scale, q.dtype)
                dk, dv, ek, ev = dk + a, dv + c, ek + ea, ev + ec
                for name, y, ref, bound in (("out", res[0], out, eo), ("dq", res[1], dq, eq)):
                    _within(f"{name} b{b} h{h}", y[b, h], ref, bound, n)
            for name, y, ref, bound in (("dk", res[2], dk, ek), ("dv", res[3], dv, ev)):
                _within(f"{name} b{b} kv{kv}", y[b, kv], ref, bound, n)


def _within(name, y, ref, bound, n):
    assert not y[n:].any(), f"{name}: not zero behind the sequence"
    err = np.abs(y - ref)
    worst = (err / np.maximum(bound, 1e-30))[err > 0].max() if (err > 0).any() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} bounds at {np.unravel_index((err - bound).argmax(), err.shape)}"


def _make(B, hq, n_kv, T, dtype, token_major, seed):
    gen = torch.Generator().manual_seed(seed)
    out = []
    for h in (hq, n_kv, n_kv, hq):
        x = torch.randn(*((B, T, h) if token_major else (B, h, T)), 128, generator=gen).to(dtype).to(DEV)
        out.append(x.transpose(1, 2) if token_major else x)
    return out


def _run(q, k, v, g, sink, window, lengths=None, scale=None):
    from head_wise_kv_b200 import window_attention
    x = [t.detach().requires_grad_() for t in (q, k, v)]
    le = torch.tensor(lengths, dtype=torch.int32, device=DEV) if lengths is not None else None
    out = window_attention(*x, sink, window, lengths=le, scale=scale)
    return (out, *torch.autograd.grad(out, x, g))


CASES = [   # B, hq, n_kv, T, sink, window, lengths
    (1, 1, 1, 1, 0, None, None), (2, 2, 1, 1, 3, 1, [0, 1]), (1, 2, 2, 127, 0, 1, None), (1, 2, 1, 128, 4, 16, None),
    (2, 4, 2, 129, 0, None, None), (2, 4, 4, 257, 16, 64, [257, 129]), (3, 2, 1, 300, 4, 33, [0, 1, 128]),
    (1, 3, 1, 511, 0, 128, [400]), (1, 8, 1, 700, 64, 256, None), (1, 2, 1, 901, 200, 33, [-5]),
    (1, 2, 1, 901, 200, 33, [5000]), (1, 2, 2, 640, 0, None, [555]), (1, 1, 1, 640, 5000, 7, None),
    (2, 2, 1, 385, 0, 5000, None), (1, 1, 1, 1500, 130, 400, None),
]


@pytest.mark.parametrize("B,hq,n_kv,T,sink,window,lengths", CASES)
@pytest.mark.parametrize("dtype,token_major", [(torch.bfloat16, True), (torch.float16, False)])
def test_values_and_gradients(B, hq, n_kv, T, sink, window, lengths, dtype, token_major):
    from head_wise_kv_b200 import window_attention_status
    q, k, v, g = _make(B, hq, n_kv, T, dtype, token_major, T)
    got = _run(q, k, v, g, sink, window, lengths)
    assert window_attention_status(DEV) == 0
    assert [t.stride() for t in got] == [t.stride() for t in (q, q, k, v)] or T == 1 or B == 1 or 1 in (hq, n_kv)
    _check(q, k, v, g, got, sink, window, lengths, 128 ** -0.5)


def _marks(B, h, T, scale=1.0):
    """Row j holds `scale` at element j mod 128: a sum over tokens keeps those of every residue apart."""
    x = torch.zeros(B, h, T, 128, dtype=torch.bfloat16, device=DEV)
    t = torch.arange(T, device=DEV)
    x[:, :, t, t % 128] = scale
    return x


@pytest.mark.parametrize("T,sink,window", [(385, 0, None), (700, 64, 256), (901, 200, 33), (1100, 130, 128), (600, 0, 129),
                                           (640, 1, 1)])
def test_every_pair_counts_once(T, sink, window):
    """Uniform weights and marked tokens: one pair too many or too few moves a sum of at most T / 128 + 1 terms."""
    q, k, v, g = _make(1, 2, 1, T, torch.bfloat16, False, 3)
    marks_q, marks_kv = _marks(1, 2, T), _marks(1, 1, T)
    for x in ((torch.zeros_like(q), marks_kv, marks_kv, g), (marks_q, torch.zeros_like(k), v, marks_q),
              (torch.zeros_like(q), marks_kv, v, marks_q)):
        _check(*x, _run(*x, sink, window), sink, window, None, 128 ** -0.5)


@pytest.mark.parametrize("hq,n_kv,T,sink,window", [(8, 1, 2200, 64, 256), (4, 2, 2050, 0, None), (16, 1, 1300, 300, 200)])
def test_key_tiles_in_pieces(hq, n_kv, T, sink, window):
    """Few key heads and many rows: the lists of the key tiles are shared out and joined."""
    q, k, v, g = _make(1, hq, n_kv, T, torch.bfloat16, True, 5)
    _check(q, k, v, g, _run(q, k, v, g, sink, window, [T - 3]), sink, window, [T - 3], 128 ** -0.5)


def test_what_lies_behind_a_sequence_does_not_matter():
    B, T = 3, 300
    lengths = [300, 131, 0]
    q, k, v, g = _make(B, 4, 2, T, torch.bfloat16, True, 8)
    for window in (None, 40):
        clean = _run(q, k, v, g, 4, window, lengths)
        bad = [x.clone() for x in (q, k, v, g)]
        for i, x in enumerate(bad):
            for b, n in enumerate(lengths):
                x[b, :, n:] = (float("nan"), float("inf"), float("-inf"), float("nan"))[i]
        assert all(torch.equal(a, b) for a, b in zip(clean, _run(*bad, 4, window, lengths)))


def test_large_scores_and_a_given_scale():
    q, k, v, g = _make(1, 2, 1, 260, torch.bfloat16, False, 9)
    q = q * 30          # weights close to one-hot, maxima that grow along the row
    got = _run(q, k, v, g, 2, 70, scale=0.125)
    _check(q, k, v, g, got, 2, 70, None, 0.125)


def test_views_expanded_and_misaligned_inputs():
    from head_wise_kv_b200 import window_attention
    B, T, hq, n_kv = 2, 150, 4, 2
    gen = torch.Generator().manual_seed(10)
    qkv = torch.randn(B, T, hq + 2 * n_kv, 128, generator=gen).to(torch.bfloat16).to(DEV).requires_grad_()
    g = torch.randn(B, T, hq, 128, generator=gen).to(torch.bfloat16).to(DEV).transpose(1, 2)
    q, k, v = (t.transpose(1, 2) for t in qkv.split([hq, n_kv, n_kv], 2))       # parts of one projection
    out = window_attention(q, k, v, 4, 30)
    grad, = torch.autograd.grad(out, qkv, g)
    grads = [t.transpose(1, 2) for t in grad.split([hq, n_kv, n_kv], 2)]
    _check(q, k, v, g, (out, *grads), 4, 30, None, 128 ** -0.5)
    # one sequence's keys for the whole batch (the gradient adds up), and a gradient of a sum (expanded)
    k1, v1 = (t[:1].detach().contiguous().requires_grad_() for t in (k, v))
    out = window_attention(q.detach(), k1.expand(B, -1, -1, -1), v1.expand(B, -1, -1, -1), 4, 30)
    gk, gv = torch.autograd.grad(out.sum(), (k1, v1))
    ones = torch.ones_like(out)
    want = _run(q, k1.expand(B, -1, -1, -1).contiguous(), v1.expand(B, -1, -1, -1).contiguous(), ones, 4, 30)
    assert torch.equal(out, want[0])
    for a, b in ((gk, want[2]), (gv, want[3])):
        assert torch.equal(a, b.sum(0, keepdim=True))
    # storage that no 16-byte load may start at, and heads that are not contiguous
    pad = torch.randn(B, hq, T, 132, generator=gen).to(torch.bfloat16).to(DEV)[..., 2:130]
    flip = torch.randn(B, hq, 128, T, generator=gen).to(torch.bfloat16).to(DEV).transpose(2, 3)
    for x in (pad, flip):
        assert torch.equal(window_attention(x, k, v, 4, 30), window_attention(x.contiguous(), k, v, 4, 30))


def test_gradients_only_where_asked_and_no_grad():
    from head_wise_kv_b200 import window_attention
    q, k, v, g = _make(1, 2, 1, 140, torch.bfloat16, False, 12)
    want = _run(q, k, v, g, 0, None)
    kk = k.clone().requires_grad_()
    out = window_attention(q, kk, v)
    out.backward(g)
    assert torch.equal(kk.grad, want[2]) and torch.equal(out, want[0])
    assert not window_attention(q, k, v).requires_grad


def test_differences():
    """The gradient along a direction against the oracle's difference of the loss."""
    T, scale, h = 200, 128 ** -0.5, 2.0 ** -12
    q, k, v, g = _make(1, 1, 1, T, torch.bfloat16, False, 13)
    got = _run(q, k, v, g, 4, 50)
    x64 = [x[0, 0].double().cpu().numpy() for x in (q, k, v)]
    g64 = g[0, 0].double().cpu().numpy()
    sees = O.window_visible(T, 4, 50)
    _, bounds = _reference(*x64, g64, sees, scale, torch.bfloat16)
    rng = np.random.default_rng(0)
    for i in range(3):
        u = rng.standard_normal((T, 128))
        f = [(O.window_attention(*[x + s * h * u if j == i else x for j, x in enumerate(x64)], sees, scale)[0] * g64).sum()
             for s in (1, -1)]
        slope = (got[1 + i][0, 0].double().cpu().numpy() * u).sum()
        # the bounds of the gradient, and h^2 / 6 times a third derivative below 2^16
        assert abs((f[0] - f[1]) / (2 * h) - slope) <= (bounds[1 + i] * np.abs(u)).sum() + h * h / 6 * 2 ** 16


def test_same_bits_again_on_another_stream_and_in_a_graph():
    from head_wise_kv_b200 import window_attention
    q, k, v, g = _make(2, 8, 2, 700, torch.bfloat16, True, 14)
    want = _run(q, k, v, g, 64, 128)
    assert all(torch.equal(a, b) for a, b in zip(want, _run(q, k, v, g, 64, 128)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _run(q, k, v, g, 64, 128)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # forward and backward captured together, with leaves of the capture's own, replayed on new inputs
    x = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    gg = g.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = window_attention(*x, 64, 128)
        res = (out, *torch.autograd.grad(out, x, gg))
    for seed in (15, 16):
        new = _make(2, 8, 2, 700, torch.bfloat16, True, seed)
        with torch.no_grad():
            for a, b in zip((*x, gg), new):
                a.copy_(b)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(res, _run(*new, 64, 128)))


def test_second_derivatives_and_foreign_captures_are_refused():
    from head_wise_kv_b200 import Rope, window_attention
    x = [t.detach().requires_grad_() for t in _make(1, 2, 1, 40, torch.bfloat16, False, 18)[:3]]
    out = window_attention(*x, 2, 9)
    gq, gk, gv = torch.autograd.grad(out.float().sum(), x, create_graph=True)
    assert gq.requires_grad
    with pytest.raises(RuntimeError, match="once"):
        (gq.float() ** 2).sum().backward()
    # the eager graph of these leaves lives: a capture with the same leaves is refused, one with its own is not
    keep = window_attention(*x, 2, 9)
    rope, pos = Rope(128), torch.zeros(1, dtype=torch.int32, device=DEV)
    for call in (lambda: window_attention(*x, 2, 9), lambda: rope.apply(x[0], pos)):
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(ValueError, match="eager graph"):
            with torch.cuda.graph(graph):
                call()
    torch.cuda.synchronize()
    y = [t.detach().requires_grad_() for t in x]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(window_attention(*y, 2, 9).float().sum(), y)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, torch.autograd.grad(keep.float().sum(), x)))


def test_empty_and_refusals():
    from head_wise_kv_b200 import window_attention, window_attention_status
    q, k, v, g = _make(2, 4, 2, 20, torch.bfloat16, False, 17)
    assert window_attention(q[:0], k[:0], v[:0]).shape == (0, 4, 20, 128)
    got = _run(q[:, :, :0], k[:, :, :0], v[:, :, :0], g[:, :, :0], 0, 3)
    assert [t.shape[2] for t in got] == [0, 0, 0, 0]
    le = torch.zeros(2, dtype=torch.int32, device=DEV)
    for bad in (lambda: window_attention(q, k[:, :, :10], v), lambda: window_attention(q, k, v[:, :1]),
                lambda: window_attention(q[:, :3], k, v), lambda: window_attention(q[0], k, v),
                lambda: window_attention(q, k, v, -1), lambda: window_attention(q, k, v, 0, 0),
                lambda: window_attention(q, k, v, lengths=le[:1]), lambda: window_attention(q, k, v, lengths=le.cpu()),
                lambda: window_attention(q, k, v, lengths=le.long()), lambda: window_attention(q, k, v, scale=0.0),
                lambda: window_attention(q[..., :64], k[..., :64], v[..., :64]), lambda: window_attention(q, k.cpu(), v)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: window_attention(q.float(), k.float(), v.float()), lambda: window_attention(q, k.half(), v)):
        with pytest.raises(TypeError):
            bad()
    assert window_attention_status(DEV) == 0


def test_gated_branches_with_rotary_positions():
    """The layer in which heads are told apart: rotate, both branches, gate; gradients of the projection and the gate."""
    from head_wise_kv_b200 import Rope, window_attention
    B, T, hq, n_kv, S, W = 2, 260, 4, 2, 8, 48
    gen = torch.Generator().manual_seed(20)
    qkv = torch.randn(B, T, hq + 2 * n_kv, 128, generator=gen).to(torch.bfloat16).to(DEV).requires_grad_()
    alpha = torch.rand(hq, generator=gen).to(DEV).requires_grad_()
    w = torch.randn(B, hq, T, 128, generator=gen).to(DEV)
    rope = Rope(128)
    pos = torch.zeros(B, dtype=torch.int32, device=DEV)
    q, k, v = (t.transpose(1, 2) for t in qkv.split([hq, n_kv, n_kv], 2))
    q, k = rope.apply(q, pos), rope.apply(k, pos)
    gate = alpha[None, :, None, None]
    full, stream = window_attention(q, k, v), window_attention(q, k, v, S, W)
    loss = ((gate * full.float() + (1 - gate) * stream.float()) * w).sum()
    g_qkv, g_alpha = torch.autograd.grad(loss, (qkv, alpha))
    # the same in fp64, from the definition
    x = qkv.detach().double().requires_grad_()
    a64 = alpha.detach().double().requires_grad_()
    f, _ = rope.frequencies()
    ang = torch.arange(T, device=DEV).double()[:, None] * torch.tensor(f, dtype=torch.float64, device=DEV)

    def turn(t):
        y, z = t[..., :64], t[..., 64:]
        return torch.cat([y * ang.cos() - z * ang.sin(), z * ang.cos() + y * ang.sin()], -1)
    qd, kd, vd = (t.transpose(1, 2) for t in x.split([hq, n_kv, n_kv], 2))
    qd, kd = turn(qd), turn(kd).repeat_interleave(hq // n_kv, 1)
    vd = vd.repeat_interleave(hq // n_kv, 1)

    def branch(s, win):
        sees = torch.from_numpy(O.window_visible(T, s, win)).to(DEV)
        return torch.softmax((qd @ kd.transpose(2, 3) * 128 ** -0.5).masked_fill(~sees, -torch.inf), -1) @ vd
    g64 = a64[None, :, None, None]
    ref = ((g64 * branch(0, 0) + (1 - g64) * branch(S, W)) * w.double()).sum()
    r_qkv, r_alpha = torch.autograd.grad(ref, (x, a64))
    # a chain of four bf16 roundings on each path (rotated input, weights, ds or branch, result) and the backward's
    # rotation: rms 2^-8 / sqrt(3) each, independent, at most eight of them
    rel = float((g_qkv.double() - r_qkv).norm() / r_qkv.norm())
    assert rel <= 2.0 ** -8 * (8 / 3) ** 0.5, rel
    # the gate's gradient: 2 T B 128 terms |w| |branch| with errors of rms 2^-8 of the branches' size
    scale = float((w.double() ** 2 * (branch(0, 0).detach() ** 2 + branch(S, W).detach() ** 2)).sum((0, 2, 3)).sqrt().max())
    assert float((g_alpha.double() - r_alpha).abs().max()) <= 4 * 2.0 ** -8 * scale


_FIRST_IN_CAPTURE = """
import torch
from head_wise_kv_b200 import window_attention, window_attention_status
x = [torch.randn(1, 2, 40, 128, device="cuda:0", dtype=torch.bfloat16) for _ in range(3)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = window_attention(*x, 2, 9)
assert window_attention_status("cuda:0") == 0
from head_wise_kv_b200 import _binding
word = _binding.status_word(0)
word.fill_(64)
graph.replay()
assert window_attention_status("cuda:0") == 64
assert torch.equal(got, window_attention(*x, 2, 9)) and window_attention_status("cuda:0") == 0
"""


def test_status_outlives_a_graph_captured_first():
    """The first call of a process inside a capture: replays leave the status bits of other calls."""
    import subprocess
    import sys
    done = subprocess.run([sys.executable, "-c", _FIRST_IN_CAPTURE], capture_output=True, text=True, timeout=240)
    assert done.returncode == 0, done.stderr[-2000:]


def test_a_dimension_of_one_entry_has_any_stride():
    from head_wise_kv_b200 import window_attention
    x = [torch.randn(1, 1, 50, 128, device=DEV, dtype=torch.bfloat16) for _ in range(3)]
    want = window_attention(*x, 1, 7)
    odd = [t.as_strided(t.shape, (3, 5, 128, 1)) for t in x]
    assert torch.equal(window_attention(*odd, 1, 7), want)
    g = torch.randn_like(want)
    a, b = ([t.detach().requires_grad_() for t in y] for y in (x, odd))
    ga = torch.autograd.grad(window_attention(*a, 1, 7), a, g)
    gb = torch.autograd.grad(window_attention(*b, 1, 7), b, g)
    assert all(torch.equal(s, t) for s, t in zip(ga, gb))


# enough heads that the forward takes two query tiles to a CTA (the cases above are small: one each), or
# two for the first and one for the last of them
MANY = [   # B, hq, n_kv, T, sink, window, lengths
    (3, 14, 2, 400, 0, None, [400, 129, 257]), (1, 32, 8, 600, 0, None, None), (2, 26, 2, 385, 16, 64, [385, 200]),
    (4, 44, 4, 130, 4, 33, [130, 0, 129, 1]), (1, 80, 8, 513, 200, 150, [400]),
]


@pytest.mark.parametrize("B,hq,n_kv,T,sink,window,lengths", MANY)
@pytest.mark.parametrize("dtype,token_major", [(torch.bfloat16, True), (torch.float16, False)])
def test_many_heads(B, hq, n_kv, T, sink, window, lengths, dtype, token_major):
    """Values and gradients; and each head alone, whose tiles go one to a CTA, gives the same bits."""
    from head_wise_kv_b200 import window_attention, window_attention_status
    q, k, v, g = _make(B, hq, n_kv, T, dtype, token_major, T + 1)
    got = _run(q, k, v, g, sink, window, lengths)
    _check(q, k, v, g, got, sink, window, lengths, 128 ** -0.5)
    le = torch.tensor(lengths, dtype=torch.int32, device=DEV) if lengths is not None else None
    G = hq // n_kv
    for h in range(0, hq, 5):
        one = window_attention(q[:, h:h + 1], k[:, h // G:h // G + 1], v[:, h // G:h // G + 1], sink, window, lengths=le)
        assert torch.equal(one, got[0][:, h:h + 1])
    assert window_attention_status(DEV) == 0


@pytest.mark.parametrize("B,hq,n_kv,T,sink,window", [(4, 44, 4, 130, 4, 33), (2, 26, 2, 385, 0, None)])
def test_garbage_behind_sequences_of_many_heads(B, hq, n_kv, T, sink, window):
    q, k, v, g = _make(B, hq, n_kv, T, torch.bfloat16, False, 5)
    lengths = [max(T - 61 * b, 0) for b in range(B)]
    clean = _run(q, k, v, g, sink, window, lengths)
    for x in (q, k, v, g):
        for b, n in enumerate(lengths):
            x[b, :, n:] = float("nan")
    assert all(torch.equal(a, b) for a, b in zip(clean, _run(q, k, v, g, sink, window, lengths)))


# fp16 holds 11 bits from 2^-14 to 65504 only.  Weights and ds are held times powers of two, so beside half a step of
# each (u = 2^-11) there remain, absolute: 2^-32 of the row's largest weight in the forward (2^-25, the weights held
# times 2^7, and the running maximum never above the last), 2^-39 of a weight in the backward (2^-25, times 2^14), and
# 2^-39 M of ds with M = max |g_i| max |v_j| over the heads that share a key head (2^-25 / f, f >= 2^14 / M).  The
# result's own rounding has a smallest half step of 2^-25.
def _reference_fp16(q, k, v, g, sees, scale, M):
    u = 2.0 ** -11
    out, p = O.window_attention(q, k, v, sees, scale)
    dq, dk, dv = O.window_attention_grad(q, k, v, g, sees, scale)
    aq, ak, av, ag = (np.abs(x) for x in (q, k, v, g))
    ep = 2 * scale * 2.0 ** -16 * float((aq @ ak.T).max()) + 2.0 ** -18
    seen = sees.astype(np.float64)
    step = 2.0 ** -25
    top = p.max(1, keepdims=True)
    eo = (u + ep) * (p @ av) + 2.0 ** -32 * top * (seen @ av) + u * np.abs(out) + step
    ev = (u + ep) * (p.T @ ag) + 2.0 ** -39 * (seen.T @ ag) + u * np.abs(dv) + step
    ds = p * (g @ v.T - (g * out).sum(1, keepdims=True))
    es = p * (2.0 ** -16 * (ag @ av.T) + (ag * eo).sum(1, keepdims=True)) + (u + ep + 2.0 ** -16) * np.abs(ds) + \
        2.0 ** -39 * M * seen
    eq = scale * es @ ak + u * np.abs(dq) + step
    ek = scale * es.T @ aq + u * np.abs(dk) + step
    return (out, dq, dk, dv), (eo, eq, ek, ev)


def _within_fp16(name, y, ref, bound):
    """A result from 65520 on rounds to infinity in fp16, and only such a one may."""
    big = np.abs(ref) - bound >= 65520
    assert np.array_equal(y[big], np.sign(ref[big]) * np.inf), name
    may = np.isinf(y) & (np.abs(ref) + bound >= 65520) & (np.sign(y) == np.sign(ref))
    _within(name, np.where(big | may, ref, y), ref, bound, len(y))


def _check_fp16(x, got, sink, window):
    q, k, v, g = (t.detach().double().cpu().numpy()[0] for t in x)
    res = [t.detach().double().cpu().numpy()[0] for t in got]
    T, G = q.shape[1], len(q) // len(k)
    sees = O.window_visible(T, sink, window or 0)
    for kv in range(len(k)):
        group = range(kv * G, kv * G + G)
        M = max(np.linalg.norm(g[h], axis=1).max() for h in group) * np.linalg.norm(v[kv], axis=1).max()
        refs = [_reference_fp16(q[h], k[kv], v[kv], g[h], sees, 128 ** -0.5, M) for h in group]
        for h, (ref, bound) in zip(group, refs):
            _within_fp16(f"out h{h}", res[0][h], ref[0], bound[0])
            _within_fp16(f"dq h{h}", res[1][h], ref[1], bound[1])
        for i, name in ((2, "dk"), (3, "dv")):
            _within_fp16(f"{name} kv{kv}", res[i][kv], sum(r[0][i] for r in refs), sum(r[1][i] for r in refs))


@pytest.mark.parametrize("T,size,sink,window", [(900, 2.0 ** -22, 0, None), (2300, 2.0 ** -20, 0, None), (700, 2.0 ** -24, 70, 300),
                                                (130, 2.0 ** -8, 0, None), (60, 512.0, 0, None), (200, 4096.0, 3, 50)])
@pytest.mark.parametrize("hq,n_kv", [(2, 1), (2, 2)])
def test_fp16_gradients_of_any_size(T, size, sink, window, hq, n_kv):
    """ds from far below fp16's smallest step to above its largest value, all of a key's with one sign.

    Values are plus or minus one pattern, gradients the pattern times `size`, so g.v = +- 128 size |v|.  Keys hold the
    value's sign in a dimension that queries leave out and queries a one in another that keys leave out: sums over ds
    add up to gradients of a size that fp16 holds."""
    gen = torch.Generator().manual_seed(T)
    pattern = torch.where(torch.rand(128, generator=gen) < 0.5, -1.0, 1.0)
    sign = torch.where(torch.rand(n_kv, T, 1, generator=gen) < 0.5, -1.0, 1.0)
    large = size >= 1           # then small queries and keys, and rows of either sign: what comes out has to fit
    v_size, other = (64.0, 2.0 ** -6 * 512 / size) if large else (1.0, 1.0)
    unit = other / 4 if large else (8.0 if size < 2.0 ** -15 else 1.0)
    q = other * torch.randn(1, hq, T, 128, generator=gen)
    k = other * torch.randn(1, n_kv, T, 128, generator=gen)
    q[..., 0], k[..., 1] = 0, 0
    q[..., 1], k[..., 0] = unit, unit * sign[..., 0]
    v = (v_size * pattern * sign)[None]
    g = size * (pattern * (1 + torch.arange(hq)[:, None, None] % 2)).expand(1, hq, T, 128)
    if large:
        g = g * torch.where(torch.rand(1, hq, T, 1, generator=gen) < 0.5, -1.0, 1.0)
    x = [t.to(torch.float16).to(DEV) for t in (q, k, v, g)]
    got = _run(*x, sink, window)
    assert float(got[1][..., T // 2:, 0].abs().min()) > 0 and float(got[2][..., 1].abs().max()) > 0
    _check_fp16(x, got, sink, window)


@pytest.mark.parametrize("T,gap", [(1500, 20), (1500, 26), (300, 30)])
def test_fp16_weights_far_below_the_largest(T, gap):
    """One key of weight nearly 1, the others 2^-gap of it each: their share of out and their dv."""
    gen = torch.Generator().manual_seed(gap)
    q, k, v, g = (torch.zeros(1, 1, T, 128) for _ in range(4))
    q[..., 0], k[0, 0, 0, 0] = 16.0, gap * 0.6931471805599453 * 128 ** 0.5 / 16
    v[..., 1:] = 64 * torch.rand(1, 1, T, 127, generator=gen)
    v[0, 0, 0] = 0
    g[:] = 64 * torch.rand(1, 1, T, 128, generator=gen)
    x = [t.to(torch.float16).to(DEV) for t in (q, k, v, g)]
    got = _run(*x, 0, None)
    # 1500 rows, gap 20: D_i = g.out is about 127 x 32 x 32 x 2^-20 i = 0.12 i, and dk of the first key
    # -16 x 128^-0.5 x (the sum of D_i: 1.4e5) = -2e5, which fp16 holds as -inf
    _check_fp16(x, got, 0, None)
    assert float(got[3][0, 0, 1, 5].abs()) > 0


def test_fp16_rows_of_very_different_gradients():
    """Most of a sequence gets no gradient or a small one, and each head its own scale."""
    q, k, v, g = _make(1, 4, 2, 600, torch.float16, False, 31)
    size = torch.exp2(-torch.randint(0, 24, (1, 4, 600, 1), generator=torch.Generator().manual_seed(1)).float()).to(DEV)
    size[:, :, ::7] = 0
    g = (g * size).to(torch.float16)
    x = [q, k, v, g]
    _check_fp16(x, _run(*x, 16, 200), 16, 200)
    zero = torch.zeros_like(g)
    assert not any(t.any() for t in _run(q, k, v, zero, 16, 200)[1:])


def test_fp16_gradient_captured_and_replayed():
    """The factor of ds is that of each replay's gradients."""
    from head_wise_kv_b200 import window_attention
    q, k, v, g = _make(1, 4, 2, 300, torch.float16, True, 32)
    x = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    gg = g.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = torch.autograd.grad(window_attention(*x, 8, 60), x, gg)
    for size in (2.0 ** -20, 256.0, 2.0 ** -12):
        gg.copy_(g * size)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(res, _run(q, k, v, gg, 8, 60)[1:]))


_FIRST_IN_INFERENCE = """
import torch
from head_wise_kv_b200 import window_attention, window_attention_status
x = [torch.randn(1, 2, 40, 128, device="cuda:0", dtype=torch.bfloat16) for _ in range(3)]
with torch.inference_mode():
    got = window_attention(*x, 2, 9)
    assert window_attention_status("cuda:0") == 0
assert window_attention_status("cuda:0") == 0
y = [t.clone().requires_grad_() for t in x]
out = window_attention(*y, 2, 9)
out.sum().backward()
assert torch.equal(got, out) and window_attention_status("cuda:0") == 0
"""


def test_status_outlives_the_inference_mode_of_the_first_call():
    import subprocess
    import sys
    done = subprocess.run([sys.executable, "-c", _FIRST_IN_INFERENCE], capture_output=True, text=True, timeout=240)
    assert done.returncode == 0, done.stderr[-2000:]


_LEAF_FURTHER_UP = """
import sys
import torch
from head_wise_kv_b200 import Rope, window_attention
rope, pos = Rope(128), torch.zeros(1, dtype=torch.int32, device="cuda:0")
w = torch.randn(1, 40, 6, 128, device="cuda:0").to(torch.bfloat16).requires_grad_()

def attend(w):
    return window_attention(*[t.transpose(1, 2) for t in w.split([2, 2, 2], 2)], 2, 9)

def rotate(w):
    return rope.apply(w.transpose(1, 2), pos)

for f in (attend, rotate):
    keep = f(w)                     # an eager graph of the leaf
    for take in (lambda y: torch.autograd.grad(y.float().sum(), w), lambda y: y.float().sum().backward()):
        graph = torch.cuda.CUDAGraph()
        try:
            with torch.cuda.graph(graph):
                take(f(w))
        except ValueError as e:
            assert "eager graph" in str(e), e
        else:
            sys.exit("captured")
        torch.cuda.synchronize()
    # the forward pass alone may be captured, and so may both with a leaf of the capture's own
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f(w)
    graph.replay()
    assert torch.equal(out, keep)
    own = w.detach().clone().requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, = torch.autograd.grad(f(own).float().sum(), own)
    graph.replay()
    assert torch.equal(got, torch.autograd.grad(keep.float().sum(), w)[0])
    del keep, out
print("done")
"""


def test_captured_backward_that_would_meet_an_eager_graphs_leaf_further_up():
    import subprocess
    import sys
    done = subprocess.run([sys.executable, "-c", _LEAF_FURTHER_UP], capture_output=True, text=True, timeout=240)
    assert done.returncode == 0 and done.stdout.endswith("done\n"), (done.returncode, done.stderr[-2000:])


def test_d_comes_from_the_unrounded_result():
    """Two keys of one weight whose values are one step apart: the result lies half a step between them, and what its
    rounding takes away is as large as ds itself.

    v = 1 and 1 + 2e (e half a step, 2^-8 for bf16): out = 1 + e rounds to 1 (to even).  With g = 1 and 128 dims
    D = 128 (1 + e), ds = -+ 64 e; from the rounded result D = 128 would give 0 and 128 e.  Everything is exact up to
    the fast exponential (p = 1/2 within 2^-18, so D within 2^-10 and ds within 2^-10) and the rounding of ds."""
    for dtype in (torch.bfloat16, torch.float16):
        e = torch.finfo(dtype).eps / 2
        q, k, v = (torch.zeros(1, 1, 2, 128, dtype=dtype, device=DEV) for _ in range(3))
        q[..., 1] = 1                       # what dk = scale ds^T q shows
        k[0, 0, 0, 0], k[0, 0, 1, 1] = 1, 0  # what dq = scale ds k shows
        v[0, 0, 0], v[0, 0, 1] = 1, 1 + 2 * e
        got = _run(q, k, v, torch.ones_like(q), 0, None, scale=1.0)
        assert (got[0][0, 0, 1] == 1).all()
        ds = [float(got[2][0, 0, 0, 1]), float(got[2][0, 0, 1, 1]), float(got[1][0, 0, 1, 0])]
        # ds, its rounding and the result's: 64 e is 0.25 or 2^-5, and 2^-10 is 1/256 or 1/32 of it
        for y, want in zip(ds, (-64 * e, 64 * e, -64 * e)):
            assert abs(y - want) <= 2.0 ** -10 + 2 * e * 64 * e, (dtype, ds)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scores_far_from_zero(sign, dtype):
    """Every scaled score of a row about +- 2^22, the edge of what is taken: only their differences count.

    127 dims of 2^7 times +- 2^11, and a last one of 2^-1 times +- 2^11 + 16 d_j: fp32 holds the sums (below 2^25, in
    steps of 2).  Scaled by 2^-3 that is +- 2^22 + d_j.  In log2 units a row's rounding of the maximum is common to its
    weights, and what is left are differences below 2: weights are right to 2^-17 + u."""
    from head_wise_kv_b200 import window_attention, window_attention_status
    T = 300
    q = torch.full((1, 1, T, 128), 128.0, dtype=dtype, device=DEV)
    q[..., 127] = 0.5
    k = torch.full((1, 1, T, 128), sign * 2048.0, dtype=dtype, device=DEV)
    d = torch.arange(T, device=DEV) % 2
    k[0, 0, :, 127] = (sign * 2048.0 + d * 16).to(dtype)
    assert (k[0, 0, :, 127].double() == sign * 2048 + d * 16).all()
    v = torch.randn(1, 1, T, 128, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    got = window_attention(q, k, v, scale=0.125).double()[0, 0]
    s = (q[0, 0].double() @ k[0, 0].double().T) * 0.125
    p = torch.softmax(s.masked_fill(~torch.ones(T, T, dtype=torch.bool, device=DEV).tril(), -torch.inf), -1)
    want, u = p @ v[0, 0].double(), torch.finfo(dtype).eps / 2
    bound = (u + 2.0 ** -17) * (p @ v[0, 0].double().abs()) + u * want.abs() + 2.0 ** -24
    assert ((got - want).abs() <= bound).all() and window_attention_status(DEV) == 0


_CAPTURED_AFTER_WARM_UP = """
import torch
from torch import nn
from head_wise_kv_b200 import Rope, window_attention, window_attention_status

class Layer(nn.Module):
    def __init__(self):
        super().__init__()
        self.proj = nn.Linear(256, 8 * 128, bias=False, dtype=torch.bfloat16, device="cuda")
        self.rope = Rope(128)
        self.register_buffer("pos", torch.zeros(2, dtype=torch.int32, device="cuda"))

    def forward(self, x):
        q, k, v = (t.transpose(1, 2) for t in self.proj(x).view(2, -1, 8, 128).split([4, 2, 2], 2))
        return window_attention(self.rope.apply(q, self.pos), self.rope.apply(k, self.pos), v, 4, 50)

torch.manual_seed(0)
layer = Layer()
x = torch.randn(2, 130, 256, device="cuda", dtype=torch.bfloat16)

def step(f):
    f(x).float().square().sum().backward()
    grad, layer.proj.weight.grad = layer.proj.weight.grad, None
    return grad

want = step(layer)
# forward and backward captured apart, the warm-up's gradient nodes kept on a stream of its own
assert torch.equal(step(torch.cuda.make_graphed_callables(layer, (x.clone(),))), want)
del layer.forward
# a whole step, warmed up on a side stream whose last graph is kept
side = torch.cuda.Stream()
side.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(side):
    step(layer)
    keep = layer(x)
torch.cuda.current_stream().wait_stream(side)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    layer(x).float().square().sum().backward()
layer.proj.weight.grad.zero_()
graph.replay()
assert torch.equal(layer.proj.weight.grad, want) and window_attention_status("cuda") == 0
# a leaf as the call's own input
q, k, v = (torch.randn(1, 2, 40, 128, device="cuda").to(torch.bfloat16).requires_grad_() for _ in range(3))
with torch.cuda.stream(side):
    keep = window_attention(q, k, v, 2, 9)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = torch.autograd.grad(window_attention(q, k, v, 2, 9).float().square().sum(), (q, k, v))
graph.replay()
assert all(torch.equal(a, b) for a, b in zip(got, torch.autograd.grad(keep.float().square().sum(), (q, k, v))))
print("done")
"""


def test_captures_after_a_warm_up_on_another_stream():
    import subprocess
    import sys
    done = subprocess.run([sys.executable, "-c", _CAPTURED_AFTER_WARM_UP], capture_output=True, text=True, timeout=240)
    assert done.returncode == 0 and done.stdout.endswith("done\n"), (done.returncode, done.stderr[-2000:])
