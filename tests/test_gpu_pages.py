"""Block tables and slot maps built on the GPU (duo_kv_reserve, duo_kv_fork)
against the oracle that keeps them page by page: whole numbers, all equal."""
import numpy as np
import pytest
import torch

from oracle import duo_oracle as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _cache(B, num_pages, page_tokens=256, cap=4096, max_pages=None):
    from head_wise_kv_b200 import DuoKVCache
    c = DuoKVCache(1, B, 1, 1, 128, 0, 1, cap, [[1]], device=DEV, kv_dtype="int4", page_tokens=page_tokens,
                   num_pages=num_pages)
    c.manage_pages(max_pages)
    return c


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _status_of(refused):
    from head_wise_kv_b200 import _lib as L
    bits = {"length": L.DUO_STATUS_BAD_LENGTH, "capacity": L.DUO_STATUS_OVER_CAPACITY, "page": L.DUO_STATUS_NO_PAGE,
            "shared": L.DUO_STATUS_SHARED_PAGE, "map": L.DUO_STATUS_OVER_CAPACITY}
    out = 0
    for r in refused:
        out |= bits[r]
    return out


def _state_equal(c, o):
    st = c.page_state()
    assert np.array_equal(st["table"].cpu().numpy(), o.table())
    assert st["held"].tolist() == [len(p) for p in o.pages]
    assert st["refs"].tolist() == o.refs
    bits = st["free_bits"].cpu().numpy().view(np.uint32)
    free = [(int(bits[p // 32]) >> (p % 32)) & 1 for p in range(o.N)]
    assert free == [int(r == 0) for r in o.refs]
    assert not any(int(bits[p // 32]) >> (p % 32) & 1 for p in range(o.N, 32 * len(bits)))


def _step(c, o, before, new, map_tokens):
    from head_wise_kv_b200 import TokenMap
    want = o.reserve(before, new, map_tokens)
    if map_tokens is None:
        after = c.reserve(_i32(before), _i32(new))
        assert after.tolist() == want[0]
    else:
        m = TokenMap(o.B, map_tokens, DEV)
        assert c.reserve(_i32(before), _i32(new), m) is m
        for got, ref in zip((m.len_after, m.cu, m.seq, m.pos, m.slot), want):
            assert np.array_equal(got.cpu().numpy(), ref)
    assert c.status() == _status_of(want[5])
    _state_equal(c, o)
    return want


@pytest.mark.parametrize("B,pages,page_tokens,cap,steps,top", [
    (1, 1, 256, 256, 6, 300), (5, 33, 256, 2048, 30, 700), (64, 200, 256, 4096, 20, 900),
    (1025, 3000, 512, 4096, 6, 900), (2100, 40000, 256, 4096, 4, 4000),
])
def test_random_steps_and_forks(B, pages, page_tokens, cap, steps, top):
    rng = np.random.default_rng(B)
    c, o = _cache(B, pages, page_tokens, cap), O.PageTables(B, pages, page_tokens, -(-cap // page_tokens), cap)
    lens = [0] * B
    for s in range(steps):
        before = [0 if rng.random() < 0.15 else n for n in lens]
        if rng.random() < 0.5:
            before = [max(0, n - int(rng.integers(0, 2)) * int(rng.integers(0, 300))) for n in before]   # going back
        kind = rng.random(B)
        new = [1 if x < 0.6 else (0 if x < 0.7 else int(rng.integers(1, top))) for x in kind]
        if s % 5 == 4:                                      # lengths that are refused
            before[int(rng.integers(0, B))] = -1
            new[int(rng.integers(0, B))] = -3
            before[int(rng.integers(0, B))] = cap + 1
        total = sum(n for n in new if n > 0)
        T = [None, total + 17, max(total * 2 // 3, 1)][s % 3]
        want = _step(c, o, before, new, T)
        lens = [min(max(a, 0), cap) if -1 < a <= cap else 0 for a in want[0]]
        if B > 1 and s % 2:
            from head_wise_kv_b200 import _lib as L
            src, dst = (int(x) for x in rng.choice(B, 2, replace=False))
            n = int(rng.integers(0, lens[src] + 1))
            ok = o.fork(src, dst, n)
            c.fork(src, dst, n)
            assert c.status() & L.DUO_STATUS_NO_PAGE == (0 if ok else L.DUO_STATUS_NO_PAGE)
            _state_equal(c, o)
            lens[dst] = n if ok else 0


def test_one_token_each_by_default_and_same_call_again():
    c, o = _cache(3, 9), O.PageTables(3, 9, 256, 16, 4096)
    lens = [255, 0, 300]
    _step(c, o, [0, 0, 0], lens, None)
    for _ in range(2):      # a step that is asked for twice gets the same pages
        after = c.reserve(_i32(lens))
        assert after.tolist() == [256, 1, 301]
        o.reserve(lens, [1, 1, 1])
        _state_equal(c, o)
    assert c.reserve(_i32([256, 1, 301])).tolist() == [257, 2, 302]
    o.reserve([256, 1, 301], [1, 1, 1])
    _state_equal(c, o)


def test_contiguous_map_and_long_map():
    from head_wise_kv_b200 import DuoKVCache, TokenMap
    c = DuoKVCache(1, 3, 1, 1, 128, 0, 1, 5000, [[1]], device=DEV)
    # a short map, and one longer than a block writes, too short for the last sequence by 990 tokens
    for before, new, T, served in (([10, 0, 4990], [1, 0, 3], 6, [1, 0, 3]),
                                   ([10, 0, 0], [4990, 4000, 5000], 13000, [4990, 4000, 0])):
        m = TokenMap(3, T, DEV)
        c.reserve(_i32(before), _i32(new), m)
        want = np.array([(b, before[b] + i) for b in range(3) for i in range(served[b])])
        n = len(want)
        assert np.array_equal(m.seq.cpu().numpy()[:n], want[:, 0]) and np.array_equal(m.pos.cpu().numpy()[:n], want[:, 1])
        assert np.array_equal(m.slot.cpu().numpy()[:n], want[:, 0] * 5000 + want[:, 1])
        assert (m.seq[n:] == -1).all() and (m.pos[n:] == -1).all() and (m.slot[n:] == -1).all()
        assert m.len_after.tolist() == [x + y for x, y in zip(before, served)]
        assert (c.status() != 0) == (served != new)


def test_two_maps_of_one_cache_on_two_streams_in_order():
    """A captured step replayed between eager ones, on another stream, in order: state and map as if all were eager."""
    from head_wise_kv_b200 import TokenMap
    c, o = _cache(4, 40), O.PageTables(4, 40, 256, 16, 4096)
    lens = _i32([0, 0, 0, 0])
    n_new = _i32([100, 0, 1, 300])
    m = TokenMap(4, 500, DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.reserve(lens, n_new, m)
        lens.copy_(m.len_after)
    host = [0, 0, 0, 0]
    side = torch.cuda.Stream()
    for i in range(6):
        if i % 2:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                c.reserve(lens, n_new, m)
                lens.copy_(m.len_after)
            torch.cuda.current_stream().wait_stream(side)
        else:
            graph.replay()
        want = o.reserve(host, [100, 0, 1, 300], 500)
        host = want[0]
        for got, ref in zip((m.len_after, m.cu, m.seq, m.pos, m.slot), want):
            assert np.array_equal(got.cpu().numpy(), ref)
        _state_equal(c, o)
    assert c.status() == 0


def test_refusals():
    from head_wise_kv_b200 import DuoError, DuoKVCache, TokenMap
    plain = DuoKVCache(1, 2, 1, 1, 128, 0, 1, 512, [[1]], device=DEV)
    with pytest.raises(ValueError):
        plain.manage_pages()
    with pytest.raises(DuoError):
        plain.page_state()
    c = DuoKVCache(1, 2, 1, 1, 128, 0, 1, 512, [[1]], device=DEV, page_tokens=256, num_pages=4)
    z = _i32([0, 0])
    with pytest.raises(DuoError):
        c.reserve(z)                    # the caller keeps the table
    with pytest.raises(DuoError):
        c.manage_pages(0)
    c.manage_pages()
    for bad in (lambda: c.reserve(z[:1]), lambda: c.reserve(z, z[:1]), lambda: c.reserve(z, z, TokenMap(3, 4, DEV)),
                lambda: c.reserve(z.cpu())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        c.reserve(z.long())
    c.set_page_table(torch.zeros(2, 2, dtype=torch.int32, device=DEV))
    with pytest.raises(DuoError):
        c.reserve(z)
    with pytest.raises(ValueError):
        TokenMap(0, 4, DEV)


@pytest.mark.parametrize("B,paged", [(3, True), (5, False), (2100, True)])
def test_lengths_that_advance_in_place(B, paged):
    """len_before is the map's own len_after: short maps (written by the block) and long ones (a second launch)."""
    from head_wise_kv_b200 import DuoKVCache, TokenMap
    cap, pages = 4096, 4 * B + 60
    c = _cache(B, pages) if paged else DuoKVCache(1, B, 1, 1, 128, 0, 1, cap, [[1]], device=DEV)
    o = O.PageTables(B, pages, 256, 16, cap)
    rng = np.random.default_rng(B)
    host, state = [0] * B, None
    for step, top in enumerate((3, 1, 2000 if B < 9 else 5, 2, 1500 if B < 9 else 4)):
        new = [int(n) for n in rng.integers(0, top + 1, B)]
        T = max(sum(new) + 3, 1)
        m = TokenMap(B, T, DEV)
        if state is not None:
            m.len_after.copy_(state)
        want = o.reserve(host, new, T)
        assert c.reserve(m.len_after, _i32(new), m) is m
        assert not want[5] and c.status() == 0
        n = sum(new)
        for got, ref in zip((m.len_after, m.cu, m.seq, m.pos), want):
            assert np.array_equal(got.cpu().numpy(), ref)
        slots = want[4] if paged else [b * cap + p if b >= 0 else -1 for b, p in zip(want[2], want[3])]
        assert np.array_equal(m.slot.cpu().numpy(), slots) and (m.slot[n:] == -1).all()
        if paged:
            _state_equal(c, o)
        host, state = want[0], m.len_after
    # the counts in the array that the lengths go to
    m.len_after.fill_(1)
    c.reserve(_i32(host), m.len_after, m)
    assert m.len_after.tolist()[:2] == [h + 1 for h in host[:2]]


def test_arrays_that_overlap_in_another_way_are_refused():
    from head_wise_kv_b200 import DuoError, TokenMap
    c = _cache(3, 9)
    m, lens = TokenMap(3, 8, DEV), _i32([0, 0, 0])
    shifted = TokenMap(3, 8, DEV)
    both = _i32([0, 0, 0, 0])
    shifted.len_after = both[1:]
    for args in ((both[:3], None, shifted), (lens, both[:3], shifted), (m.cu[1:], None, m), (m.seq[2:5], None, m),
                 (lens, m.pos[:3], m), (lens, m.slot.view(torch.int32)[13:], m)):
        with pytest.raises(DuoError):
            c.reserve(*args)
    assert c.status() == 0 and c.page_state()["held"].tolist() == [0, 0, 0]


def test_the_longest_map():
    """2^31 - 1 entries: the number of blocks is worked out without passing 31 bits."""
    from head_wise_kv_b200 import TokenMap
    T = 2 ** 31 - 1
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 34 GB for the map")
    c, o = _cache(2, 20), O.PageTables(2, 20, 256, 16, 4096)
    m = TokenMap(2, T, DEV)
    m.seq[-3:] = 7
    c.reserve(_i32([0, 0]), _i32([300, 5]), m)
    want = o.reserve([0, 0], [300, 5], 400)
    for got, ref in zip((m.seq, m.pos, m.slot), want[2:5]):
        assert got[:400].tolist() == ref and (got[-1000:] == -1).all()
    assert m.len_after.tolist() == [300, 5] and c.status() == 0
    del m
    torch.cuda.empty_cache()
