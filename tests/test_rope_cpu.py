"""Rotary positions and page tables without a GPU: the library's angles
against the oracle's formulas, the oracle's rotation against its definition,
the oracle's page tables on hand-made cases, and the refusals that need no
device."""
import ctypes
import itertools
import random
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import duo_oracle as O

CASES = [
    dict(scaling="none"), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="yarn", factor=8.0, original_len=4096), dict(scaling="yarn", factor=1.0, original_len=4096),
    dict(scaling="yarn", factor=16.0, original_len=2048, low=2.0, high=20.0),
    dict(scaling="bands", factor=8.0, original_len=8192),
    dict(scaling="bands", factor=32.0, original_len=8192, low=1.5, high=9.0),
]


def _rope(d=128, **kw):
    from head_wise_kv_b200 import Rope
    return Rope(d, **kw)


@pytest.mark.parametrize("d,rot", [(64, 16), (64, 64), (128, 64), (128, 96), (128, 128)])
@pytest.mark.parametrize("theta", [10000.0, 500000.0])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['scaling']}-{c.get('factor', 1)}")
def test_angles_follow_the_formulas(d, rot, theta, case):
    r = _rope(d, theta=theta, rot_dim=rot, **case)
    f, m = r.frequencies()
    ref, mag = O.rope_frequencies(rot, theta=theta, **case)
    # a dozen fp64 operations on each side, the largest amplification that of a ramp (a difference of terms up to
    # ~70 over a span of at least 0.001 of one): 2^-40 leaves a wide margin over 2^-53 and is far below any use
    assert np.allclose(f, ref, rtol=2.0 ** -40, atol=0)
    assert m == pytest.approx(mag, rel=1e-15)


def test_angles_of_pair_factors_and_given_magnitude():
    factors = np.linspace(1.0, 40.0, 32)
    f, m = _rope(64, scaling="factors", pair_factors=factors, magnitude=1.25).frequencies()
    ref, _ = O.rope_frequencies(64, scaling="factors", pair_factors=factors)
    assert np.allclose(f, ref, rtol=2.0 ** -50) and m == 1.25


def test_oracle_rotation_is_the_definition():
    rng = np.random.default_rng(3)
    f, _ = O.rope_frequencies(32)
    x = rng.standard_normal((5, 48))
    pos = np.array([0, 1, 7, -3, 1000])
    for layout in ("half", "interleaved"):
        y = O.rope_rotate(x, pos, f, 1.5, layout)
        for t in range(5):
            for i in range(16):
                a, b = (i, i + 16) if layout == "half" else (2 * i, 2 * i + 1)
                c, s = np.cos(pos[t] * f[i]), np.sin(pos[t] * f[i])
                assert y[t, a] == pytest.approx(1.5 * (x[t, a] * c - x[t, b] * s), abs=1e-12)
                assert y[t, b] == pytest.approx(1.5 * (x[t, b] * c + x[t, a] * s), abs=1e-12)
        assert np.array_equal(y[:, 32:], x[:, 32:])
        # the transposed map: <R x, g> = <x, R^T g>
        g = rng.standard_normal(x.shape)
        back = O.rope_rotate(g, pos, f, 1.5, layout, transpose=True)
        assert np.allclose((y * g).sum(-1), (x * back).sum(-1), atol=1e-11)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), -2), (dict(d=128, rot_dim=24), -2), (dict(d=128, rot_dim=144), -1), (dict(d=64, rot_dim=0), -1),
    (dict(theta=1.0), -1), (dict(theta=float("nan")), -1), (dict(theta=float("inf")), -1),
    (dict(scaling="linear", factor=0.5), -1), (dict(scaling="ntk", factor=float("nan")), -1),
    (dict(scaling="yarn", factor=4.0), -1), (dict(scaling="bands", factor=4.0, original_len=-1), -1),
    (dict(scaling="bands", factor=4.0, original_len=64, low=4.0, high=2.0), -1),
    (dict(scaling="yarn", factor=4.0, original_len=64, low=40.0), -1),
    (dict(scaling="factors"), -1), (dict(scaling="factors", pair_factors=[0.0] * 64), -1),
    (dict(magnitude=-1.0), -1), (dict(magnitude=float("nan")), -1),
])
def test_rope_refusals(kw, code):
    from head_wise_kv_b200 import DuoError
    kw = dict(kw)
    with pytest.raises(DuoError) as e:
        _rope(kw.pop("d", 128), **kw)
    assert e.value.code == code


def test_rope_refuses_unknown_names_and_counts():
    for kw in (dict(layout="rows"), dict(scaling="dynamic"), dict(scaling="factors", pair_factors=[1.0] * 3)):
        with pytest.raises(ValueError):
            _rope(128, **kw)


def _tensor(L, x=256, out=256, heads=4, rotate=1, ins=(512, 128, 64), outs=(512, 128, 64)):
    return L.duo_rope_tensor(x, out, heads, rotate, (ctypes.c_int64 * 3)(*ins), (ctypes.c_int64 * 3)(*outs))


def test_rope_apply_refusals_come_before_any_launch():
    from head_wise_kv_b200 import _lib as L
    r = _rope(64)

    def call(tensors=None, handle=r.handle, dtype=0, batch=1, n=1, positions=64, n_new=None):
        t = [_tensor(L)] if tensors is None else tensors
        L.duo_rope_apply(handle, dtype, 0, batch, n, (L.duo_rope_tensor * len(t))(*t), positions, 0, n_new, None)
    for kw, code in [(dict(handle=None), -1), (dict(dtype=3), -1), (dict(batch=-1), -1), (dict(n=-1), -1),
                     (dict(positions=None), -1), (dict(positions=66), -6), (dict(n_new=2), -6),
                     (dict(tensors=[]), -1), (dict(tensors=[_tensor(L)] * 4), -1),
                     (dict(tensors=[_tensor(L, heads=0)]), -1), (dict(tensors=[_tensor(L, x=None)]), -1),
                     (dict(tensors=[_tensor(L, out=None)]), -1), (dict(tensors=[_tensor(L, x=264)]), -6),
                     (dict(tensors=[_tensor(L, outs=(512, 128, 60))]), -6),
                     (dict(tensors=[_tensor(L, ins=(4, 128, 64))]), -6)]:
        with pytest.raises(L.DuoError) as e:
            call(**kw)
        assert e.value.code == code, kw
    call(batch=0)     # nothing to do: no launch, no error
    call(n=0)


def test_append_step_and_page_calls_refuse_without_a_handle():
    from head_wise_kv_b200 import _lib as L
    r = _rope(128)
    rows = L.duo_rows(256, 1024, 128)
    n, view = ctypes.c_size_t(0), L.duo_kv_pages_view()
    calls = [
        lambda: L.duo_kv_append_rope(None, 0, r.handle, rows, rows, rows, 64, None, None, 1, 256, None),
        lambda: L.duo_decode_step_rope(None, 0, r.handle, rows, rows, rows, 64, 64, 0.1, 256, 256, None, 256, 1 << 20,
                                       None),
        lambda: L.duo_decode_step_rope(None, 0, r.handle, None, rows, rows, 64, 64, 0.1, 256, 256, None, 256, 1 << 20,
                                       None),
        lambda: L._check(L._c_pages_bytes(None, 4, ctypes.byref(n)), "bytes"),
        lambda: L.duo_kv_pages_init(None, 4, 256, 1 << 20, None),
        lambda: L._check(L._c_pages_view(None, ctypes.byref(view)), "view"),
        lambda: L.duo_kv_reserve(None, 64, None, 0, 64, None, None, None, None, None),
    ]
    for call in calls:
        with pytest.raises(L.DuoError) as e:
            call()
        assert e.value.code == L.DUO_ERR_INVALID_ARG
    assert L._c_rope_free(None) == 0


# ------------------------------------------------------------ the oracle's page tables
def test_oracle_pages_lowest_free_first():
    t = O.PageTables(3, 8, 4, 4, 16)
    after, cu, seq, pos, slot, refused = t.reserve([0, 0, 0], [5, 0, 3], 10)
    assert after == [5, 0, 3] and cu == [0, 5, 5, 8] and not refused
    assert t.pages == [[0, 1], [], [2]]
    assert seq == [0] * 5 + [2] * 3 + [-1] * 2 and pos == [0, 1, 2, 3, 4, 0, 1, 2, -1, -1]
    assert slot == [0, 1, 2, 3, 4, 8, 9, 10, -1, -1]
    # sequence 0 leaves, a new request takes its slot; sequence 2 goes on into the lowest free page
    after, cu, seq, pos, slot, _ = t.reserve([0, 0, 3], [1, 9, 2], 12)
    assert t.pages == [[0], [1, 3, 4], [2, 5]] and after == [1, 9, 5]
    assert slot[-2:] == [2 * 4 + 3, 5 * 4]


def test_oracle_pages_refusals():
    t = O.PageTables(4, 3, 4, 4, 16)
    t.reserve([0] * 4, [4, 1, 0, 0])
    # 1 free page: sequence 0 needs one and gets it; 2 asks for two and is refused, and 3 behind it as well; 1 needs none
    after, cu, *_, refused = t.reserve([4, 1, 0, 0], [1, 3, 8, 1], 100)
    assert after == [5, 4, 0, 0] and refused == {"page"} and cu == [0, 1, 4, 4, 4]
    assert t.reserve([17, -1, 0, 0], [0, 0, 0, 0])[5] == {"length"}
    assert t.reserve([4, 4, 0, 0], [13, 0, 0, 0])[5] == {"capacity"}
    assert t.reserve([4, 1, 0, 0], [1, 1, 0, 0], 1)[5] == {"map"}


def test_oracle_fork_shares_full_pages():
    t = O.PageTables(3, 6, 4, 4, 16)
    t.reserve([0, 0, 0], [10, 0, 0])
    assert t.fork(0, 1, 10) and t.pages[1] == [0, 1, 3] and t.refs[:4] == [2, 2, 1, 1]
    assert t.fork(0, 2, 8) and t.pages[2] == [0, 1] and t.refs[0] == 3
    # the first owner leaves: shared pages stay, its own comes back
    t.reserve([0, 10, 8], [0, 0, 0])
    assert t.refs == [2, 2, 0, 1, 0, 0]
    # going back into a shared page is refused
    assert t.reserve([0, 10, 6], [0, 0, 1])[5] == {"shared"}
    assert not t.fork(1, 0, 16)          # the source holds fewer pages


# ------------------------------------------------------------ overlap of strided tensors
def _bytes_of(t):
    size, places = t.element_size(), set()
    for index in itertools.product(*[range(n) for n in t.shape]):
        at = t.data_ptr() + size * sum(i * s for i, s in zip(index, t.stride()))
        places.update(range(at, at + size))
    return places


def test_overlap_is_that_of_the_bytes():
    """Random strided tensors of two element sizes in one storage against the sets of their bytes."""
    from head_wise_kv_b200 import _binding
    rng = random.Random(0)
    base = torch.zeros(400)
    for _ in range(1500):
        x, y = (torch.as_strided(rng.choice([base, base.view(torch.bfloat16)]),
                                 [rng.choice([0, 1, 2, 3, 4, 4, 4]) if rng.random() < 0.1 else rng.randint(1, 4) for _ in range(3)],
                                 [rng.choice([0, 1, 2, 3, 4, 5, 6, 8, 12, 16, 24, 30, 37]) for _ in range(3)],
                                 rng.randint(0, 60)) for _ in range(2))
        bx, by = _bytes_of(x), _bytes_of(y)
        assert _binding.overlap(x, y) == _binding.overlap(y, x) == bool(bx & by), (x.shape, x.stride(), y.shape, y.stride())
        assert _binding.overlaps_itself(x) == (len(bx) < x.numel() * x.element_size()), (x.shape, x.stride())


def test_overlap_of_a_projections_parts():
    from head_wise_kv_b200 import _binding
    qkv = torch.zeros(2, 500, 12, 128, dtype=torch.bfloat16)
    q, k, v = qkv.split([8, 2, 2], 2)
    for a, b in ((q, k), (q, v), (k, v), (q.transpose(1, 2), k.transpose(1, 2)), (qkv[:, :200], qkv[:, 200:])):
        assert not _binding.overlap(a, b) and not _binding.overlap(b, a)
    flat = qkv.view(-1)
    inside = flat[12 * 128 * 3 + 5: 12 * 128 * 3 + 5 + 1024].view(8, 128)
    for a, b in ((qkv[:, :, :4], qkv[:, :, 1:5]), (qkv[:, :4], qkv[:, 1:5]), (q, inside), (q, flat[:1024]), (k, qkv)):
        assert _binding.overlap(a, b) and _binding.overlap(b, a)
    assert not _binding.overlap(k, flat[:1024]) and not _binding.overlap(k, flat[1280:1536])
    assert _binding.overlaps_itself(q.expand(2, 500, 8, 128)[:1, :1].expand(3, 4, 8, 128))
    assert not any(_binding.overlaps_itself(t) for t in (q, k, v, q.transpose(1, 2)))


_COPIES = """
import copy, pickle
from head_wise_kv_b200 import Rope
for r in (Rope(128), Rope(64, rot_dim=32, layout="interleaved", scaling="factors", pair_factors=[1.0 + i for i in range(16)]),
          Rope(128, 500000.0, scaling="yarn", factor=8.0, original_len=4096, low=2.0, high=20.0, magnitude=1.5)):
    same = [copy.copy(r), copy.deepcopy({"layer": [r]})["layer"][0], pickle.loads(pickle.dumps(r))]
    want = r.frequencies()
    for c in same:
        assert c.handle not in (None, r.handle) and c.frequencies() == want and (c.d, c.rot_dim) == (r.d, r.rot_dim)
    r.close()
    assert all(c.frequencies() == want for c in same)
    same.clear()
print("done")
"""


def test_copies_of_a_plan_are_plans_of_their_own():
    """A copied model's Rope: the plan is freed once each (in a process of its own: a second free ends it)."""
    done = subprocess.run([sys.executable, "-c", _COPIES], capture_output=True, text=True, timeout=240)
    assert done.returncode == 0 and done.stdout == "done\n", done.stderr[-2000:]
