"""Rotary append and decode step (duo_kv_append_rope, duo_decode_step_rope,
prefill_rope) on the GPU.

Each append runs on twin caches: one with append_rope, one with the oracle's
rotation worked out in fp64, rounded to bf16 and appended with duo_kv_append.
Values, positions and every row that a step must not touch have to be the
same bytes.  Keys and rotated queries are compared with the fp64 rotation:
fp32 arithmetic (2^-20 of the pair's magnitudes, see test_gpu_rope.py) and
one rounding: half a step of bf16 (2^-8), of E4M3 (2^-4 of the value, at
least half the smallest step 2^-10, times the scale) or of INT4 (half a code
times the scale).
"""
import numpy as np
import pytest
import torch

from _harness import assert_close
from oracle import duo_oracle as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
PAGE = 256
KINDS = ["bf16", "fp8", "int4", "paged_bf16", "paged_fp8", "paged_int4"]
SCALING = dict(scaling="bands", factor=8.0, original_len=2048)


class Setup:
    def __init__(self, kind, B=3, hq=8, n_kv=4, d=128, sink=4, window=33, cap=1500, rot=None, layout="half", caches=2,
                 mask=None, num_pages=None):
        from head_wise_kv_b200 import DuoKVCache, Rope
        self.kv = kind.replace("paged_", "")
        self.B, self.hq, self.n_kv, self.d, self.S, self.W = B, hq, n_kv, d, sink, window
        self.mask = np.array([g % 2 == 0 for g in range(n_kv)] if mask is None else mask, dtype=np.uint8)
        rng = np.random.default_rng(7)
        self.ks, self.vs = (rng.uniform(0.3, 0.6, (1, n_kv)).astype(np.float32) for _ in range(2))
        if self.kv == "bf16":
            self.ks = self.vs = np.ones((1, n_kv), dtype=np.float32)
        paged = kind.startswith("paged")
        per = -(-cap // PAGE)
        kw = dict(page_tokens=PAGE, num_pages=num_pages or B * per + 2) if paged else {}
        quant = {} if self.kv == "bf16" else dict(k_scale=self.ks, v_scale=self.vs)
        self.caches = [DuoKVCache(1, B, hq, n_kv, d, sink, window, cap, self.mask[None], device=DEV, kv_dtype=self.kv,
                                  **quant, **kw) for _ in range(caches)]
        for c in self.caches[1:]:
            c.buf.copy_(self.caches[0].buf)
        if paged:
            perm = rng.permutation(kw["num_pages"])[:B * per].reshape(B, per).astype(np.int32)
            for c in self.caches:
                c.set_page_table(torch.from_numpy(perm).to(DEV))
        self.rope = Rope(d, rot_dim=rot, layout=layout, **SCALING)
        self.freq, self.mag = O.rope_frequencies(rot or d, **SCALING)
        self.layout, self.rot = layout, rot or d

    def rotate(self, x, pos):
        """x [..., d] tensor, pos broadcast against x's leading shape."""
        x64 = x.double().cpu().numpy()
        return O.rope_rotate(x64, np.asarray(pos), self.freq, self.mag, self.layout)

    def slack(self, x):
        x64 = np.abs(x.double().cpu().numpy())
        pair = np.zeros_like(x64)
        a, b = (slice(0, self.rot // 2), slice(self.rot // 2, self.rot)) if self.layout == "half" else \
            (slice(0, self.rot, 2), slice(1, self.rot, 2))
        pair[..., a] = pair[..., b] = x64[..., a] + x64[..., b]
        return self.mag * pair * 2.0 ** -20

    def key_rounding(self, ref, g):
        s = float(self.ks[0, g])
        if self.kv == "bf16":
            return np.abs(ref) * 2.0 ** -8
        if self.kv == "fp8":
            return np.maximum(np.abs(ref) * 2.0 ** -4, s * 2.0 ** -10)
        return np.full(ref.shape, s / 2)

    def values(self, codes, g, ks=True):
        """Rows of a cache region as the values they stand for."""
        s = float((self.ks if ks else self.vs)[0, g])
        if self.kv == "bf16":
            return codes.double().cpu().numpy()
        c = codes.cpu().numpy()
        return O.dequantize_kv(c, s) if self.kv == "fp8" else O.dequantize_kv_int4(c, s)


def _qkv(st, T, seed, lead=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*(lead or (T,)), st.hq + 2 * st.n_kv, st.d, generator=g).to(torch.bfloat16).to(DEV)
    return x.split([st.hq, st.n_kv, st.n_kv], -2)


def _twin_append(st, cache, k, v, before, counts, n):
    """The same tokens through duo_kv_append: k, v [B][n][n_kv][d]."""
    pos = np.asarray(before)[:, None, None] + np.arange(n)[None, :, None]
    kr = torch.from_numpy(st.rotate(k, pos)).to(torch.bfloat16).to(DEV)
    cache.append(0, kr.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous(),
                 torch.tensor(before, dtype=torch.int32, device=DEV), torch.tensor(counts, dtype=torch.int32, device=DEV))


def _same(a, b):
    """The same bytes (rows never written may hold NaN patterns)."""
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _compare(st, k, before, counts):
    """caches[0] (append_rope) against caches[1] and the fp64 keys of this step."""
    a, b = (c.layer_views(0) for c in st.caches)
    assert st.caches[0].status() == st.caches[1].status() == 0
    for name in ("v_retrieval", "v_streaming", "positions"):
        assert _same(a[name], b[name]), name
    table = st.caches[0]._page_table
    seen = {n: torch.zeros(a[n].shape[:-1], dtype=torch.bool) for n in ("k_retrieval", "k_streaming")}
    for s, (lb, n) in enumerate(zip(before, counts)):
        for i in range(n):
            p = lb + i
            for g in range(st.n_kv):
                r = a["head_rank"][g]
                if st.mask[g]:
                    at = (int(table[s, p // PAGE]), r, p % PAGE) if table is not None else (s, r, p)
                    name = "k_retrieval"
                elif p < st.S or p >= lb + n - st.W:
                    at, name = (s, r, p if p < st.S else st.S + (p - st.S) % st.W), "k_streaming"
                else:
                    continue
                seen[name][at] = True
                if i % 7 == 0 or i >= n - 3:
                    ref = st.rotate(k[s, i, g], p)
                    err = np.abs(st.values(a[name][at], g) - ref)
                    if st.kv == "int4":
                        sc = float(st.ks[0, g])
                        ref = np.clip(ref, -8 * sc, 7 * sc)
                        err = np.abs(st.values(a[name][at], g) - ref)
                    assert np.all(err <= st.key_rounding(ref, g) * (1 + 2.0 ** -10) + st.slack(k[s, i, g])), (s, p, g)
    for name, m in seen.items():     # what the step does not write stays as it was
        assert _same(a[name][~m.to(DEV)], b[name][~m.to(DEV)]), name
        b[name].copy_(a[name])       # later steps start from the same bytes


@pytest.mark.parametrize("kind,layout,rot,d", [(kind, layout, rot, 128) for kind in KINDS for layout, rot in
                                               (("half", None), ("interleaved", 64))] + [("bf16", "half", 32, 64)])
def test_padded(kind, layout, rot, d):
    st = Setup(kind, d=d, rot=rot, layout=layout)
    lens = [0, 0, 0]
    for step, (n, counts) in enumerate([(70, [70, 1, 0]), (1, [1, 1, 1]), (300, [300, 255, 33]), (5, [0, 5, 2]),
                                        (37, [37, 36, 35])]):
        q, k, v = _qkv(st, 0, step, (st.B, n))
        out = torch.full((st.B, n, st.hq, st.d), 3.0, dtype=torch.bfloat16, device=DEV)
        bt = torch.tensor(lens, dtype=torch.int32, device=DEV)
        even = len(set(counts)) == 1 and counts[0] == n
        st.caches[0].append_rope(0, st.rope, q, k, v, bt, out=out,
                                 n_new=None if even else torch.tensor(counts, dtype=torch.int32, device=DEV))
        _twin_append(st, st.caches[1], k, v, lens, counts, n)
        for b, c in enumerate(counts):
            assert (out[b, c:] == 3).all()
            ref = st.rotate(q[b, :c], lens[b] + np.arange(c)[:, None])
            err = np.abs(out[b, :c].double().cpu().numpy() - ref)
            assert np.all(err <= np.abs(ref) * 2.0 ** -8 * (1 + 2.0 ** -10) + st.slack(q[b, :c]))
        _compare(st, k, lens, counts)
        lens = [a + b for a, b in zip(lens, counts)]


@pytest.mark.parametrize("kind", ["bf16", "paged_fp8"])
@pytest.mark.parametrize("with_slot", [True, False])
def test_ragged_equals_padded(kind, with_slot):
    """The same tokens as one ragged batch with padding rows, in an order that is not the sequences'."""
    st = Setup(kind)
    from head_wise_kv_b200 import TokenMap
    lens, counts, n = [0, 200, 40], [260, 1, 33], 260
    q0, k0, v0 = _qkv(st, 0, 3, (st.B, 200))
    for c in st.caches:
        c.append_rope(0, st.rope, None, k0, v0, torch.zeros(3, dtype=torch.int32, device=DEV),
                      n_new=torch.tensor(lens, dtype=torch.int32, device=DEV))
    q, k, v = _qkv(st, 0, 4, (st.B, n))
    T = sum(counts) + 9
    order = [(b, i) for b in (2, 0, 1) for i in range(counts[b])] + [(-1, 0)] * 9
    m = TokenMap(st.B, T, DEV)
    table = st.caches[0]._page_table
    seq = torch.tensor([b for b, _ in order], dtype=torch.int32)
    pos = torch.tensor([lens[b] + i if b >= 0 else -1 for b, i in order], dtype=torch.int32)
    if table is not None:
        slot = [int(table[b, (lens[b] + i) // PAGE]) * PAGE + (lens[b] + i) % PAGE if b >= 0 else -1 for b, i in order]
    else:
        slot = [b * 1500 + lens[b] + i if b >= 0 else -1 for b, i in order]
    m.seq.copy_(seq), m.pos.copy_(pos), m.slot.copy_(torch.tensor(slot))
    m.len_after.copy_(torch.tensor([a + b for a, b in zip(lens, counts)], dtype=torch.int32))
    at = torch.tensor([b for b, _ in order]), torch.tensor([i for _, i in order])
    before = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = torch.full((T, st.hq, st.d), 3.0, dtype=torch.bfloat16, device=DEV)
    rows = [t[at[0].to(DEV), at[1].to(DEV)].contiguous() for t in (q, k, v)]
    if not with_slot:
        m.slot = torch.zeros(0, dtype=torch.int64, device=DEV)      # a NULL pointer: read through the page table
        assert m.slot.data_ptr() == 0
    st.caches[0].append_rope(0, st.rope, *rows, before, m, out=out)
    want = st.caches[1].append_rope(0, st.rope, q, k, v, before,
                                    n_new=torch.tensor(counts, dtype=torch.int32, device=DEV))
    assert (out[-9:] == 3).all()
    assert torch.equal(out[:-9], want[at[0][:-9].to(DEV), at[1][:-9].to(DEV)])
    assert torch.equal(st.caches[0].buf, st.caches[1].buf)
    assert st.caches[0].status() == 0


def test_all_heads_of_one_kind_and_keys_only():
    for mask in ([1, 1, 1, 1], [0, 0, 0, 0]):
        st = Setup("bf16", mask=mask, window=1, sink=0)
        _, k, v = _qkv(st, 0, 11, (3, 10))
        counts = [10, 3, 0]
        assert st.caches[0].append_rope(0, st.rope, None, k, v, torch.zeros(3, dtype=torch.int32, device=DEV),
                                        n_new=torch.tensor(counts, dtype=torch.int32, device=DEV)) is None
        _twin_append(st, st.caches[1], k, v, [0, 0, 0], counts, 10)
        _compare(st, k, [0, 0, 0], counts)


def test_status_bits_and_untouched_rows():
    from head_wise_kv_b200 import TokenMap, _lib as L
    st = Setup("paged_bf16", caches=1)
    cache = st.caches[0]
    q, k, v = _qkv(st, 8, 5)
    start = cache.buf.clone()
    zero = torch.zeros(3, dtype=torch.int32, device=DEV)

    def run(seq, pos, slot):
        cache.buf.copy_(start)
        m = TokenMap(3, 8, DEV)
        m.seq[0], m.pos[0], m.slot[0] = seq, pos, slot
        m.len_after.fill_(pos + 1 if pos >= 0 else 0)
        cache.append_rope(0, st.rope, q, k, v, zero, m)
        return cache.status()
    assert run(3, 0, 0) == L.DUO_STATUS_BAD_LENGTH
    assert run(0, -2, 0) == L.DUO_STATUS_BAD_LENGTH
    assert run(0, 1500, 0) == L.DUO_STATUS_OVER_CAPACITY
    assert run(0, 5, -1) == L.DUO_STATUS_NO_PAGE
    assert run(0, 5, 20 * PAGE) == L.DUO_STATUS_NO_PAGE
    assert run(0, 5, 1 << 40) == L.DUO_STATUS_NO_PAGE
    assert run(-1, 0, 0) == 0
    # padded: a negative length and one beyond the capacity
    cache.append_rope(0, st.rope, None, *[t.view(3, 2, *t.shape[1:]) for t in (k[:6], v[:6])],
                      torch.tensor([-1, 0, 1499], dtype=torch.int32, device=DEV))
    assert cache.status() == L.DUO_STATUS_BAD_LENGTH | L.DUO_STATUS_OVER_CAPACITY


def test_refusals():
    from head_wise_kv_b200 import DuoError, Rope, TokenMap
    st = Setup("bf16", caches=1)
    c = st.caches[0]
    q, k, v = _qkv(st, 6, 5)
    zero = torch.zeros(3, dtype=torch.int32, device=DEV)
    m = TokenMap(3, 6, DEV)
    q2, k2, v2 = (t.reshape(3, 2, *t.shape[1:]) for t in (q, k, v))
    for bad in (lambda: c.append_rope(0, Rope(64), q, k, v, zero, m), lambda: c.append_rope(0, st.rope, q, k, v, zero),
                lambda: c.append_rope(0, st.rope, q, k, v, zero, TokenMap(4, 6, DEV)),
                lambda: c.append_rope(0, st.rope, q[:5], k, v, zero, m),
                lambda: c.append_rope(0, st.rope, q, k, v, zero, m, n_new=zero),
                lambda: c.append_rope(0, st.rope, q, k, v, zero[:2], m),
                lambda: c.append_rope(0, st.rope, q2.transpose(0, 1).contiguous().transpose(0, 1), k2, v2, zero),
                lambda: c.append_rope(0, st.rope, None, k, v, zero, m, out=q)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        c.append_rope(0, st.rope, q.float(), k, v, zero, m)
    off = torch.zeros(6, st.n_kv, st.d + 4, dtype=torch.bfloat16, device=DEV)[..., 4:]
    with pytest.raises(DuoError) as e:
        c.append_rope(0, st.rope, q, off, v, zero, m)
    assert e.value.code == -6
    with pytest.raises(DuoError):
        c.append_rope(1, st.rope, q, k, v, zero, m)
    page = Setup("paged_bf16", caches=1).caches[0]
    from head_wise_kv_b200 import DuoKVCache
    bare = DuoKVCache(1, 3, 8, 4, 128, 4, 33, 1500, st.mask[None], device=DEV, page_tokens=PAGE, num_pages=9)
    with pytest.raises(DuoError):        # no page table
        bare.append_rope(0, st.rope, None, k2, v2, zero)
    assert page.status() == 0


class _Rows:
    """Keys and values of every sequence as appended, for the oracle."""

    def __init__(self, st):
        self.st, self.k, self.v = st, [[] for _ in range(st.B)], [[] for _ in range(st.B)]

    def add(self, b, k, v, first):
        st = self.st
        for i in range(k.shape[0]):
            kk = torch.from_numpy(st.rotate(k[i], first + i)).to(torch.bfloat16).double().numpy()
            vv = v[i].double().cpu().numpy()
            if st.kv == "fp8":
                kk = np.stack([O.dequantize_kv(O.quantize_kv(kk[g], float(st.ks[0, g])), float(st.ks[0, g]))
                               for g in range(st.n_kv)])
                vv = np.stack([O.dequantize_kv(O.quantize_kv(vv[g], float(st.vs[0, g])), float(st.vs[0, g]))
                               for g in range(st.n_kv)])
            self.k[b].append(kk)
            self.v[b].append(vv)

    def hist(self, which, b, g):
        return np.stack([r[g] for r in which[b]])


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("paged_bf16", 128), ("fp8", 128), ("bf16", 64)])
def test_step_rope_equals_append_rope_then_decode(kind, d):
    st = Setup(kind, B=4, d=d, window=8, layout="interleaved", rot=64)
    lens = [0, 3, 700, 41]
    _, k0, v0 = _qkv(st, 0, 21, (4, 700))
    for c in st.caches:
        c.append_rope(0, st.rope, None, k0, v0, torch.zeros(4, dtype=torch.int32, device=DEV),
                      n_new=torch.tensor(lens, dtype=torch.int32, device=DEV))
    scale = d ** -0.5
    for step in range(12):
        q, k, v = _qkv(st, 4, 30 + step)
        before = torch.tensor(lens, dtype=torch.int32, device=DEV)
        grow = [1, 1, 1, 1] if step != 5 else [1, 0, 1, 1]      # a length that does not grow: waits for the append
        after = torch.tensor([max(a + g, 1) for a, g in zip(lens, grow)], dtype=torch.int32, device=DEV)
        q_rot = torch.empty_like(q.contiguous())
        got, lse = st.caches[0].step_rope(0, st.rope, q, k, v, before, after, scale, want_lse=True, q_rot=q_rot)
        qr = st.caches[1].append_rope(0, st.rope, q[:, None], k[:, None], v[:, None], before)[:, 0].contiguous()
        ref, ref_lse = st.caches[1].decode(0, qr, after, scale, want_lse=True)
        assert torch.equal(q_rot, qr) and torch.equal(got, ref) and torch.equal(lse, ref_lse)
        assert torch.equal(st.caches[0].buf, st.caches[1].buf)
        lens = [a + 1 for a in lens]
    assert st.caches[0].status() == 0


def test_run_of_prompt_chunks_and_steps_against_the_oracle():
    """prefill_rope in two ragged chunks, then steps: attention equals the oracle on rotated keys."""
    st = Setup("bf16", B=2, sink=4, window=40, caches=1)
    cache, rows, scale = st.caches[0], _Rows(st), st.d ** -0.5
    lens = [0, 0]
    for C, counts in ((150, [150, 90]), (70, [1, 70])):
        q, k, v = _qkv(st, 0, 50 + C, (2, C))
        out = cache.prefill_rope(0, st.rope, q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV), scale,
                                 n_new=torch.tensor(counts, dtype=torch.int32, device=DEV))
        for b, n in enumerate(counts):
            rows.add(b, k[b, :n], v[b, :n], lens[b])
            qr = torch.from_numpy(st.rotate(q[b, :n], lens[b] + np.arange(n)[:, None])).to(torch.bfloat16)
            ref = O.prefill_attention(qr.transpose(0, 1)[None].double().numpy(), lambda _, g: rows.hist(rows.k, b, g),
                                      lambda _, g: rows.hist(rows.v, b, g), [lens[b]], st.mask, st.S, st.W, scale)
            assert_close(out[b:b + 1, :, :n].double().cpu().numpy(), ref, f"chunk of {C}, sequence {b}")
        lens = [a + b for a, b in zip(lens, counts)]
    for step in range(3):
        q, k, v = _qkv(st, 2, 90 + step)
        out = cache.step_rope(0, st.rope, q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV),
                              torch.tensor([n + 1 for n in lens], dtype=torch.int32, device=DEV), scale)
        for b in range(2):
            rows.add(b, k[b:b + 1], v[b:b + 1], lens[b])
        qr = np.stack([torch.from_numpy(st.rotate(q[b], lens[b])).to(torch.bfloat16).double().numpy() for b in range(2)])
        lens = [n + 1 for n in lens]
        ref, _ = O.decode_attention(qr, lambda b, g: rows.hist(rows.k, b, g), lambda b, g: rows.hist(rows.v, b, g),
                                    lens, st.mask, st.S, st.W, scale)
        assert_close(out.double().cpu().numpy(), ref, f"step {step}")
    assert cache.status() == 0


def test_captured_steps():
    """reserve, append_rope and decode of a step captured once and replayed with lengths that grow on the device."""
    from head_wise_kv_b200 import TokenMap
    B = 4
    st = Setup("paged_bf16", B=B, window=8, cap=600, caches=2)
    scale = st.d ** -0.5
    for c in st.caches:
        c.manage_pages()
    q, k, v = (t.contiguous() for t in _qkv(st, B, 1))
    lens = torch.tensor([0, 250, 255, 10], dtype=torch.int32, device=DEV)
    _, k0, v0 = _qkv(st, 0, 2, (B, 255))
    for c in st.caches:
        c.reserve(torch.zeros_like(lens), lens)
        c.append_rope(0, st.rope, None, k0, v0, torch.zeros_like(lens), n_new=lens)
    tokens = TokenMap(B, B, DEV)
    out = torch.empty(B, st.hq, st.d, dtype=torch.float32, device=DEV)
    q_out = torch.empty_like(q)
    moving = lens.clone()

    def step():
        st.caches[0].reserve(moving, None, tokens)
        st.caches[0].append_rope(0, st.rope, q, k, v, moving, tokens, out=q_out)
        st.caches[0].decode(0, q_out, tokens.len_after, scale, out=out)
        moving.add_(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(8):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        after = st.caches[1].reserve(lens)
        ref = st.caches[1].step_rope(0, st.rope, q, k, v, lens, after, scale)
        lens = after
        assert torch.equal(out, ref) and torch.equal(tokens.len_after, after)
    assert st.caches[0].status() == st.caches[1].status() == 0
    assert torch.equal(st.caches[0].page_state()["table"], st.caches[1].page_state()["table"])


def test_rotated_queries_over_an_input_are_refused():
    st = Setup("bf16", B=2)
    c = st.caches[0]
    x = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pool = torch.zeros(2 * 12 * 128, dtype=torch.bfloat16, device=DEV)
    inside, over = pool[:1024].view(2, 1, 4, 128), pool[:2048].view(2, 1, 8, 128)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    for args in ((x, k, v, x), (x, inside, v, over), (x, k, inside, over)):
        with pytest.raises(ValueError):
            c.append_rope(0, st.rope, *args[:3], zero, out=args[3])


def test_lengths_that_advance_in_place():
    """reserve advances the map's own len_after and append_rope gets that: a request that starts over in a used slot
    leaves no position of the last one in the ring."""
    from head_wise_kv_b200 import TokenMap
    B = 3
    st = Setup("paged_bf16", B=B, window=9, caches=2)
    for c in st.caches:
        c.manage_pages()
    maps = [TokenMap(B, 60, DEV) for _ in range(2)]
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    for step, (new, over) in enumerate((([20, 5, 33], None), ([1, 1, 1], None), ([3, 1, 6], [0, 1, 2]), ([2, 0, 1], [1, 2]),
                                        ([40, 1, 0], [0]))):
        for b in over or []:        # a new request in this slot
            lens[b] = 0
            maps[0].len_after[b] = 0
        n = torch.tensor(new, dtype=torch.int32, device=DEV)
        q, k, v = _qkv(st, 60, 70 + step)
        st.caches[0].reserve(maps[0].len_after, n, maps[0])
        got = st.caches[0].append_rope(0, st.rope, q, k, v, maps[0].len_after, maps[0])
        st.caches[1].reserve(lens, n, maps[1])
        want = st.caches[1].append_rope(0, st.rope, q, k, v, lens, maps[1])
        lens = maps[1].len_after.clone()
        assert torch.equal(got, want) and torch.equal(maps[0].len_after, lens)
        a, b = (c.layer_views(0) for c in st.caches)
        # a slot whose request has not brought a token yet is not looked at before it does
        live = lens > 0
        assert torch.equal(a["positions"][live], b["positions"][live])
        for name in ("k_retrieval", "v_retrieval", "k_streaming", "v_streaming"):
            assert _same(a[name], b[name]), name
    assert st.caches[0].status() == st.caches[1].status() == 0


def test_rotated_queries_within_a_projection_are_refused():
    """q, k and v as parts of one projection, and an out inside its storage; beside it, it is accepted."""
    from head_wise_kv_b200 import TokenMap
    st = Setup("bf16", B=2, caches=1)
    c, heads = st.caches[0], st.hq + 2 * st.n_kv
    pool = torch.randn(60 * heads * 128, device=DEV).to(torch.bfloat16)
    keep, before = pool.clone(), c.buf.clone()
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    m = TokenMap(2, 10, DEV)
    m.seq[:3], m.len_after[0] = 0, 3
    m.pos[:3].copy_(torch.arange(3))
    q, k, v = pool[10 * 128: 10 * 128 + 10 * heads * 128].view(10, heads, 128).split([st.hq, st.n_kv, st.n_kv], 1)
    n = 10 * st.hq * 128
    for start in (0, 128 * 5, 10 * 128, 100 * 128):
        with pytest.raises(ValueError, match="apart"):
            c.append_rope(0, st.rope, q, k, v, zero, m, out=pool[start:start + n].view(10, st.hq, 128))
    q2, k2, v2 = pool[:20 * heads * 128].view(2, 10, heads, 128).split([st.hq, st.n_kv, st.n_kv], 2)
    with pytest.raises(ValueError, match="apart"):
        c.append_rope(0, st.rope, q2, k2, v2, zero, out=pool[n:3 * n].view(2, 10, st.hq, 128))
    assert torch.equal(pool, keep) and torch.equal(c.buf, before)
    start = 20 * heads * 128
    got = c.append_rope(0, st.rope, q, k, v, zero, m, out=pool[start:start + n].view(10, st.hq, 128))
    want = c.append_rope(0, st.rope, q, k, v, zero, m)
    assert torch.equal(got[:3], want[:3]) and torch.equal(got[3:].reshape(-1), keep[start + 3 * st.hq * 128:start + n])


def test_a_steps_results_over_its_inputs_are_refused():
    """q_rot over a part of the projection, or over out; rotating in place is accepted."""
    st = Setup("bf16", B=2)
    heads = st.hq + 2 * st.n_kv
    pool = torch.randn(2 * heads * 128 + 4096, device=DEV).to(torch.bfloat16)
    keep, before = pool.clone(), st.caches[0].buf.clone()
    q, k, v = pool[:2 * heads * 128].view(2, heads, 128).split([st.hq, st.n_kv, st.n_kv], 1)
    n = 2 * st.hq * 128
    zero, one = torch.zeros(2, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    scratch = torch.zeros(4 * n, device=DEV)

    def step(c, q, **kw):
        return c.step_rope(0, st.rope, q, k, v, zero, one, 0.1, **kw)
    rot, out = scratch[:n // 2].view(torch.bfloat16).view(2, st.hq, 128), scratch[:n].view(2, st.hq, 128)
    lse = scratch[n - 5:n - 5 + 2 * st.hq].view(2, st.hq)
    part = pool.view(torch.float32)[:n].view(2, st.hq, 128)
    for kw in (dict(q_rot=pool[:n].view(2, st.hq, 128)), dict(q_rot=pool[n:2 * n].view(2, st.hq, 128)), dict(out=part),
               dict(lse=part.view(-1)[400:400 + 2 * st.hq].view(2, st.hq)), dict(q_rot=rot, out=out), dict(out=out, lse=lse)):
        with pytest.raises(ValueError, match="apart"):
            step(st.caches[0], q, **kw)
    assert torch.equal(pool, keep) and torch.equal(st.caches[0].buf, before)
    dense = q.contiguous()
    want = step(st.caches[0], dense, q_rot=rot)
    assert torch.equal(step(st.caches[1], dense, q_rot=dense), want) and torch.equal(dense, rot)
    assert torch.equal(st.caches[0].buf, st.caches[1].buf)


def test_tangents_are_refused():
    import torch.autograd.forward_ad as fwAD
    st = Setup("bf16", B=2, caches=1)
    c = st.caches[0]
    before = c.buf.clone()
    q, k, v = (t.contiguous() for t in _qkv(st, 2, 5))
    zero, one = torch.zeros(2, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    with fwAD.dual_level():
        dual = [fwAD.make_dual(t, torch.ones_like(t)) for t in (q, k, v)]
        for i in range(3):
            x = [dual[j] if j == i else t for j, t in enumerate((q, k, v))]
            for call in (lambda: c.step_rope(0, st.rope, *x, zero, one, 0.1),
                         lambda: c.append_rope(0, st.rope, *[t[:, None] for t in x], zero),
                         lambda: c.prefill_rope(0, st.rope, *[t[:, None] for t in x], zero, 0.1)):
                with pytest.raises(NotImplementedError, match="forward-mode"):
                    call()
    assert torch.equal(c.buf, before)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("strided", [False, True])
def test_prefill_rope_caches_what_append_rope_does(kind, strided):
    """The same token has the same codes whichever call it came by: quantised from the fp32 rotated value."""
    st = Setup(kind, cap=800)
    scale = st.d ** -0.5
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    for C, counts in ((130, [130, 1, 77]), (1, [1, 1, 1]), (60, [33, 60, 2])):
        q, k, v = _qkv(st, 0, C, (3, C + (5 if strided else 0)))
        if strided:         # a part of a longer batch: sequences do not follow one another at the token stride
            q, k, v = (t[:, 3:3 + C] for t in (q, k, v))
        n = None if len(set(counts)) == 1 and counts[0] == C else torch.tensor(counts, dtype=torch.int32, device=DEV)
        st.caches[0].prefill_rope(0, st.rope, q, k, v, lens, scale, n_new=n)
        st.caches[1].append_rope(0, st.rope, None, k.contiguous(), v.contiguous(), lens, n_new=n)
        a, b = (c.layer_views(0) for c in st.caches)
        for name in ("k_retrieval", "v_retrieval", "k_streaming", "v_streaming", "positions"):
            assert _same(a[name], b[name]), name
        lens = lens + torch.tensor(counts, dtype=torch.int32, device=DEV)
    assert st.caches[0].status() == st.caches[1].status() == 0


@pytest.mark.parametrize("kind", ["bf16", "paged_fp8", "int4"])
def test_prefill_rope_of_a_padded_batch_with_anything_in_its_padding(kind):
    st = Setup(kind, cap=800)
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    for C, counts in ((150, [150, 90, 0]), (70, [1, 70, 63])):
        n = torch.tensor(counts, dtype=torch.int32, device=DEV)
        clean = [t.contiguous() for t in _qkv(st, 0, C, (3, C))]
        want = st.caches[0].prefill_rope(0, st.rope, *clean, lens, st.d ** -0.5, n_new=n)
        bad = [t.clone() for t in clean]
        for t, x in zip(bad, (float("nan"), float("inf"), float("nan"))):
            for b, c in enumerate(counts):
                t[b, c:] = x
        bad[2][0, counts[0] + 3:] = 3e38
        got = st.caches[1].prefill_rope(0, st.rope, *bad, lens, st.d ** -0.5, n_new=n)
        for b, c in enumerate(counts):
            assert torch.isfinite(want[b, :, :c]).all() and torch.equal(want[b, :, :c], got[b, :, :c]), (C, b)
        assert torch.equal(st.caches[0].buf, st.caches[1].buf)
        lens = lens + n
    assert st.caches[0].status() == st.caches[1].status() == 0


def test_a_step_without_tokens():
    """A map of no entries, and a padded batch of none: nothing is written, and the rotated queries are empty."""
    from head_wise_kv_b200 import TokenMap
    st = Setup("bf16", caches=1)
    c = st.caches[0]
    before = c.buf.clone()
    zero = torch.zeros(3, dtype=torch.int32, device=DEV)
    q, k, v = _qkv(st, 0, 1)
    m = TokenMap(3, 0, DEV)
    c.reserve(zero, zero, m)
    assert m.cu.tolist() == [0] * 4
    for out in (None, torch.empty(0, st.hq, st.d, dtype=torch.bfloat16, device=DEV)):
        assert c.append_rope(0, st.rope, q, k, v, zero, m, out=out).shape == (0, st.hq, st.d)
    assert c.append_rope(0, st.rope, None, k, v, zero, m) is None
    q, k, v = _qkv(st, 0, 1, (3, 0))
    assert c.append_rope(0, st.rope, q, k, v, zero).shape == (3, 0, st.hq, st.d)
    assert c.append_rope(0, st.rope, q, k, v, zero, n_new=zero).shape == (3, 0, st.hq, st.d)
    assert torch.equal(c.buf, before) and c.status() == 0


def test_what_a_call_writes_counts_as_changed():
    """A backward pass that saved a tensor which a call has since written refuses, as after any in-place operation."""
    from head_wise_kv_b200 import Rope, TokenMap, window_attention
    st = Setup("bf16", B=2, caches=1)
    c, rope = st.caches[0], Rope(128)
    zero, one = torch.zeros(2, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    q, k, v = (t.contiguous() for t in _qkv(st, 2, 5))
    m = TokenMap(2, 2, DEV)

    def saved(t):
        w = torch.ones_like(t).requires_grad_()
        return w, (t * w).sum()
    x = torch.randn(2, 3, 4, 128, device=DEV).to(torch.bfloat16)
    out, lse, rot = torch.ones(2, 8, 128, device=DEV), torch.ones(2, 8, device=DEV), torch.ones_like(q)
    for written, call in (((x,), lambda: rope.apply(x, zero, out=x)), ((x,), lambda: rope.launch([(x, x, True)], zero)),
                          ((rot,), lambda: c.append_rope(0, st.rope, q[:, None], k[:, None], v[:, None], zero, out=rot[:, None])),
                          ((out, lse, rot), lambda: c.step_rope(0, st.rope, q, k, v, zero, one, 0.1, out=out, lse=lse, q_rot=rot))):
        graphs = [saved(t) for t in written]
        with torch.no_grad():
            call()
        for w, loss in graphs:
            with pytest.raises(RuntimeError, match="inplace"):
                loss.backward()
        w, loss = saved(written[0])     # and what is saved afterwards is good
        loss.backward()
        assert torch.equal(w.grad, written[0])
    # lengths and positions that a later step moves on
    x = [torch.randn(2, 2, 8, 128, device=DEV).to(torch.bfloat16).requires_grad_() for _ in range(3)]
    c.reserve(zero, None, m)
    att, y = window_attention(*x, lengths=m.len_after), rope.apply(x[0], m.len_after)
    c.reserve(m.len_after, None, m)
    for t in (att, y):
        with pytest.raises(RuntimeError, match="inplace"):
            t.sum().backward()
    with torch.inference_mode():        # no versions there
        t = torch.randn(2, 3, 4, 128, device=DEV).to(torch.bfloat16)
        rope.apply(t, zero, out=t)
    with pytest.raises(ValueError, match="recorded"):
        rope.apply(x[0].detach(), zero, out=x[0])


@pytest.mark.parametrize("kind,layout,rot", [("int4", "half", None), ("paged_int4", "interleaved", 64), ("paged_fp8", "half", 32)])
def test_step_rope_on_quantised_caches(kind, layout, rot):
    st = Setup(kind, B=4, window=8, layout=layout, rot=rot)
    lens = torch.tensor([0, 3, 700, 255], dtype=torch.int32, device=DEV)
    _, k0, v0 = _qkv(st, 0, 21, (4, 700))
    for c in st.caches:
        c.append_rope(0, st.rope, None, k0, v0, torch.zeros_like(lens), n_new=lens)
    for step in range(10):
        q, k, v = _qkv(st, 4, 30 + step)
        got, lse = st.caches[0].step_rope(0, st.rope, q, k, v, lens, lens + 1, 0.09, want_lse=True)
        qr = st.caches[1].append_rope(0, st.rope, q[:, None], k[:, None], v[:, None], lens)[:, 0].contiguous()
        ref, ref_lse = st.caches[1].decode(0, qr, lens + 1, 0.09, want_lse=True)
        assert torch.equal(got, ref) and torch.equal(lse, ref_lse) and torch.equal(st.caches[0].buf, st.caches[1].buf)
        lens = lens + 1
    assert st.caches[0].status() == st.caches[1].status() == 0


def test_a_map_with_a_negative_length_stays_within_the_ring():
    """Token 0 of a sequence whose len_after is not one: nothing before the sequence's slots is written."""
    from head_wise_kv_b200 import TokenMap
    st = Setup("bf16", caches=1)
    c = st.caches[0]
    c.buf[4096:].fill_(7)
    m = TokenMap(3, 2, DEV)
    m.seq[0], m.pos[0] = 0, 0
    m.len_after.copy_(torch.tensor([-30, 0, 0]))
    _, k, v = _qkv(st, 2, 5)
    keep = {n: t.clone() for n, t in c.layer_views(0).items() if torch.is_tensor(t)}
    c.append_rope(0, st.rope, None, k, v, torch.tensor([9, 9, 9], dtype=torch.int32, device=DEV), m)
    views = c.layer_views(0)
    SW = st.S + st.W
    assert torch.equal(views["positions"][1:], keep["positions"][1:])
    assert views["positions"][0].tolist() == [0] + [-1] * (SW - 1)
    for name, at in (("k_retrieval", (0, slice(None), 0)), ("v_retrieval", (0, slice(None), 0)), ("k_streaming", (0, slice(None), 0)),
                     ("v_streaming", (0, slice(None), 0))):
        mask = torch.ones(keep[name].shape[:3], dtype=torch.bool, device=DEV)
        mask[at] = False
        assert _same(views[name][mask], keep[name][mask]), name
