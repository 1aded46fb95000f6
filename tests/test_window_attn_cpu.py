"""The oracle's windowed attention against its definition and against
differences, and the refusals that need no device."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import duo_oracle as O


def test_visible_is_the_rule():
    for T, S, W, n in ((9, 2, 3, None), (9, 0, 1, 5), (9, 4, 0, 7), (5, 9, 9, 0)):
        got = O.window_visible(T, S, W, n)
        for i in range(T):
            for j in range(T):
                sees = j <= i and (W == 0 or j < S or j > i - W) and i < (T if n is None else n)
                assert got[i, j] == sees
        if S + W:       # the same rule as a decode step's keep set
            last = T - 1 if n is None else n - 1
            if W and last >= 0:
                assert list(np.nonzero(got[last])[0]) == list(O.keep_set(last, S, W))


@pytest.mark.parametrize("S,W", [(0, 0), (2, 3), (0, 1)])
def test_gradients_against_differences(S, W):
    rng = np.random.default_rng(1)
    T, d = 11, 6
    q, k, v, g = (rng.standard_normal((T, d)) for _ in range(4))
    see = O.window_visible(T, S, W, 9)
    grads = O.window_attention_grad(q, k, v, g, see, 0.3)

    def f(*x):
        return (O.window_attention(*x, see, 0.3)[0] * g).sum()
    h = 1e-5
    for i, dx in enumerate(grads):
        for _ in range(4):
            u = rng.standard_normal((T, d))
            up, down = ([x + s * h * u if j == i else x for j, x in enumerate((q, k, v))] for s in (1, -1))
            # second-order remainder h^2 times third derivatives of order 10, and 2^-52 / h of cancellation
            assert abs((f(*up) - f(*down)) / (2 * h) - (dx * u).sum()) < 1e-7


def test_masked_places_do_not_matter():
    rng = np.random.default_rng(2)
    q, k, v, g = (rng.standard_normal((8, 4)) for _ in range(4))
    see = O.window_visible(8, 1, 3, 5)
    clean = O.window_attention_grad(q, k, v, g, see, 1.0)
    for x in (q, k, v, g):
        x[5:] = np.nan
    assert all(np.array_equal(a, b) for a, b in zip(clean, O.window_attention_grad(q, k, v, g, see, 1.0)))


def _desc(L, **kw):
    a = dict(dtype=0, batch=2, hq=4, n_kv=2, d=128, tokens=9, sink=1, window=3, scale=0.1, lengths=None)
    a.update(kw)
    return L.duo_window_attn_desc(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -2), (dict(dtype=9), -2), (dict(d=64), -2), (dict(batch=-1), -1), (dict(tokens=-1), -1),
    (dict(hq=0), -1), (dict(n_kv=0), -1), (dict(hq=5), -1), (dict(sink=-1), -1), (dict(window=-1), -1),
    (dict(scale=0.0), -1), (dict(scale=-0.1), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(lengths=2), -6), (dict(tokens=1 << 27), -2), (dict(tokens=1 << 26, hq=256, n_kv=256), -2),
])
def test_description_refusals(kw, code):
    from head_wise_kv_b200 import _lib as L
    h = L.duo_heads(256, 128 * 64, 128, 512)
    n = ctypes.c_size_t(0)
    d = _desc(L, **kw)
    for call in (lambda: L._check(L._c_win_stats(ctypes.byref(d), ctypes.byref(n)), "stats"),
                 lambda: L._check(L._c_win_ws(ctypes.byref(d), ctypes.byref(n)), "workspace"),
                 lambda: L.duo_window_attn(d, h, h, h, h, 256, None, None),
                 lambda: L.duo_window_attn_grad(d, h, h, h, h, h, 256, h, h, h, 256, 1 << 20, None, None)):
        with pytest.raises(L.DuoError) as e:
            call()
        assert e.value.code == code


@pytest.mark.parametrize("heads,code", [
    ((0, 8192, 128, 512), -1), ((264, 8192, 128, 512), -6), ((256, 8196, 128, 512), -6), ((256, 8192, 132, 512), -6),
    ((256, 8192, 128, 514), -6), ((256, 8192, 64, 512), -1), ((256, 0, 128, 512), -1), ((256, 8192, 128, -512), -1),
    ((256, 1 << 39, 128, 512), -1),
])
def test_tensor_refusals(heads, code):
    from head_wise_kv_b200 import _lib as L
    good, bad, d = L.duo_heads(256, 8192, 128, 512), L.duo_heads(*heads), _desc(L)
    calls = [lambda a=a: L.duo_window_attn(d, *[bad if i == a else good for i in range(4)], 256, None, None)
             for a in range(4)]
    for a in range(8):
        t = [bad if i == a else good for i in range(8)]
        calls.append(lambda t=t: L.duo_window_attn_grad(d, *t[:5], 256, *t[5:], 256, 1 << 20, None, None))
    for call in calls:
        with pytest.raises(L.DuoError) as e:
            call()
        assert e.value.code == code


def test_pointer_refusals_and_empty_calls():
    from head_wise_kv_b200 import _lib as L
    h, d = L.duo_heads(256, 8192, 128, 512), _desc(L)
    for call, code in ((lambda: L.duo_window_attn(None, h, h, h, h, 256, None, None), -1),
                       (lambda: L.duo_window_attn(d, h, h, h, h, None, None, None), -1),
                       (lambda: L.duo_window_attn(d, h, h, h, h, 260, None, None), -6),
                       (lambda: L.duo_window_attn(d, h, h, h, h, 256, 258, None), -6),
                       (lambda: L.duo_window_attn_grad(d, h, h, h, h, h, 256, h, h, h, None, 0, None, None), -1),
                       (lambda: L.duo_window_attn_grad(d, h, h, h, h, h, 256, h, h, h, 128, 0, None, None), -6)):
        with pytest.raises(L.DuoError) as e:
            call()
        assert e.value.code == code
    for kw in (dict(batch=0), dict(tokens=0)):      # nothing to do
        L.duo_window_attn(_desc(L, **kw), None, None, None, None, None, None, None)
        L.duo_window_attn_grad(_desc(L, **kw), *[None] * 5, None, *[None] * 4, 0, None, None)
    assert L.duo_window_attn_stats_bytes(_desc(L)) == 2 * 4 * 128 * (4 + 128)


def test_python_refusals():
    from head_wise_kv_b200 import window_attention
    x = torch.zeros(1, 2, 3, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        window_attention(x, x, x)                   # not on a CUDA device
    with pytest.raises(TypeError):
        window_attention(x.float(), x, x)
    with pytest.raises(TypeError):
        window_attention([1], x, x)


def test_tangents_and_traces_are_refused():
    """A result that reads memory alone would lose a forward-mode tangent, and a trace would record nothing."""
    import torch.autograd.forward_ad as fwAD
    from head_wise_kv_b200 import Rope, window_attention
    rope, pos = Rope(128), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 3, 128, dtype=torch.bfloat16)
    with fwAD.dual_level():
        dual = fwAD.make_dual(x, torch.ones_like(x))
        for call in (lambda: window_attention(dual, x, x), lambda: window_attention(x, x, dual), lambda: rope.apply(dual, pos),
                     lambda: rope.apply(dual.requires_grad_(), pos), lambda: rope.apply(x, pos, out=dual),
                     lambda: rope.launch([(x, x, True), (dual, x, False)], pos)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
            window_attention(dual, x, x)
    for call in (lambda t: window_attention(t, t, t), lambda t: rope.apply(t, pos)):
        for t in (x, x.clone().requires_grad_()):
            with pytest.raises(NotImplementedError, match="trace"):
                torch.jit.trace(call, (t,))
    with pytest.raises(ValueError):     # not refused for either: on the CPU
        window_attention(x, x, x)
