"""Rotary positions on the GPU (duo_rope_apply) against the fp64 oracle.

Bounds.  With y = m (x0 cos a - x1 sin a) in fp32: the angle, cosine and sine
carry at most 2^-22 each of the unit circle (a fixed-point fraction rounded
to fp32 within an eighth of a turn, a two-ulp sine, the product with m), each
product and the sum one rounding of 2^-24: together below
2^-20 m (|x0| + |x1|).  Storing rounds once more, by half a step of the type
(relative 2^-8 for bf16, 2^-11 for fp16, 2^-24 for fp32; fp16 has a smallest
step of 2^-24).
"""
import numpy as np
import pytest
import torch

from oracle import duo_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _positions(rng, B, n, per_token, far):
    shape = (B, n) if per_token else (B,)
    return rng.integers(-far // 2, far - n, shape).astype(np.int32)


def _spread(pos, n):
    return pos[:, None].astype(np.int64) + np.arange(n) if pos.ndim == 1 else pos.astype(np.int64)


def _check(got, x, pos, freq, mag, layout, transpose):
    """got, x: [B][H][n][d] tensors; pos [B][n] int64."""
    x64 = x.double().cpu().numpy()
    ref = O.rope_rotate(x64, pos[:, None], freq, mag, layout, transpose)
    pair = np.zeros_like(x64)
    rot = 2 * len(freq)
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    pair[..., a] = pair[..., b] = np.abs(x64[..., a]) + np.abs(x64[..., b])
    half = torch.finfo(x.dtype).eps / 2
    bound = np.abs(ref) * half * (1 + 2.0 ** -10) + mag * pair * 2.0 ** -20
    bound += 2.0 ** -25 if x.dtype == torch.float16 else 0
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= bound), f"off by {(err / np.maximum(bound, 1e-300)).max():.3g} bounds"


CASES = [   # dtype, d, rot, layout, scaling
    (torch.bfloat16, 128, 128, "half", dict()),
    (torch.bfloat16, 128, 64, "interleaved", dict(scaling="yarn", factor=8.0, original_len=4096)),
    (torch.bfloat16, 64, 16, "half", dict(scaling="linear", factor=4.0)),
    (torch.float16, 128, 96, "half", dict(scaling="bands", factor=8.0, original_len=8192, theta=500000.0)),
    (torch.float16, 64, 64, "interleaved", dict(scaling="ntk", factor=4.0)),
    (torch.float32, 128, 128, "interleaved", dict(theta=1000000.0)),
    (torch.float32, 64, 32, "half", dict(scaling="yarn", factor=32.0, original_len=2048)),
]


@pytest.mark.parametrize("dtype,d,rot,layout,scaling", CASES)
@pytest.mark.parametrize("B,H,n", [(1, 1, 1), (3, 5, 7), (2, 32, 130), (5, 3, 1021)])
@pytest.mark.parametrize("token_major,per_token,transpose,far", [
    (False, False, False, 4096), (True, True, False, 2 ** 31 - 1), (True, False, True, 1 << 20)])
def test_apply(dtype, d, rot, layout, scaling, B, H, n, token_major, per_token, transpose, far):
    from head_wise_kv_b200 import Rope
    rope = Rope(d, rot_dim=rot, layout=layout, **scaling)
    rng = np.random.default_rng(B * 1000 + n)
    g = torch.Generator().manual_seed(n)
    x = torch.randn(*((B, n, H, d) if token_major else (B, H, n, d)), generator=g).to(dtype).to(DEV)
    x = x.transpose(1, 2) if token_major else x
    pos = _positions(rng, B, n, per_token, far)
    before = x.clone()
    y = rope.apply(x, torch.from_numpy(pos).to(DEV), transpose=transpose)
    assert torch.equal(x, before)
    f, m = O.rope_frequencies(rot, **scaling)
    _check(y, x, _spread(pos, n), f, m, layout, transpose)
    assert torch.equal(y[..., rot:], x[..., rot:])


def test_in_place_counts_and_three_tensors():
    from head_wise_kv_b200 import Rope
    rope = Rope(128)
    f, m = O.rope_frequencies(128)
    g = torch.Generator().manual_seed(2)
    B, n = 3, 37
    pos = torch.tensor([0, 1000, 131000], dtype=torch.int32)
    x = torch.randn(B, 4, n, 128, generator=g).to(torch.bfloat16).to(DEV)
    y = x.clone()
    rope.apply(y, pos.to(DEV), out=y)
    _check(y, x, _spread(pos.numpy(), n), f, m, "half", False)
    # counts: rows behind them stay as they were; a count of zero and one beyond n
    keep = torch.full_like(x, 7.0)
    counts = torch.tensor([0, 5, 99], dtype=torch.int32, device=DEV)
    rope.apply(x, pos.to(DEV), n_new=counts, out=keep)
    assert (keep[0] == 7).all() and (keep[1, :, 5:] == 7).all()
    assert torch.equal(keep[1, :, :5], y[1, :, :5]) and torch.equal(keep[2], y[2])
    assert not rope.apply(x, pos.to(DEV), n_new=counts)[0].any()
    # q, k and v of one projection, token-major, laid out head-major in one launch
    qkv = torch.randn(B, n, 12, 128, generator=g).to(torch.bfloat16).to(DEV)
    src = [t.transpose(1, 2) for t in qkv.split([8, 2, 2], 2)]
    dst = [torch.empty(t.shape, dtype=t.dtype, device=DEV) for t in src]
    rope.launch([(src[0], dst[0], True), (src[1], dst[1], True), (src[2], dst[2], False)], pos.to(DEV))
    for i in (0, 1):
        _check(dst[i], src[i], _spread(pos.numpy(), n), f, m, "half", False)
    assert torch.equal(dst[2], src[2])


def test_broadcast_input_and_empty():
    from head_wise_kv_b200 import Rope
    rope = Rope(64, layout="interleaved")
    f, m = O.rope_frequencies(64)
    x = torch.randn(1, 1, 9, 64).to(torch.bfloat16).to(DEV).expand(2, 3, 9, 64)
    pos = torch.tensor([5, 70], dtype=torch.int32, device=DEV)
    _check(rope.apply(x, pos), x, _spread(pos.cpu().numpy(), 9), f, m, "interleaved", False)
    assert rope.apply(x[:, :, :0], pos).shape == (2, 3, 0, 64)
    assert rope.apply(x[:0], pos[:0]).shape == (0, 3, 9, 64)


def test_gradient_against_formula_and_differences():
    from head_wise_kv_b200 import Rope
    scaling = dict(scaling="yarn", factor=8.0, original_len=2048)
    rope = Rope(64, rot_dim=32, layout="interleaved", **scaling)
    f, m = O.rope_frequencies(32, **scaling)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(2, 3, 11, 64, generator=g).to(DEV).requires_grad_()
    pos = torch.tensor([3, 5000], dtype=torch.int32, device=DEV)
    w = torch.randn(2, 11, 3, 64, generator=g).to(DEV).transpose(1, 2)
    y = rope.apply(x, pos)
    grad, = torch.autograd.grad(y, x, w)
    _check(grad, w, _spread(pos.cpu().numpy(), 11), f, m, "interleaved", True)
    # the map is linear: a difference along any direction is the derivative
    v = torch.randn(x.shape, generator=g).to(DEV)
    with torch.no_grad():
        diff = ((rope.apply(x + v, pos) - rope.apply(x - v, pos)).double() * w.double()).sum() / 2
    slope = (grad.double() * v.double()).sum()
    # 2112 products of values below ~5, each rounded a few times at 2^-24 relative to terms below ~20
    assert abs(float(diff - slope)) <= 2112 * 20 * 4 * 2.0 ** -24
    # of a sum (a broadcast gradient), with counts: rows behind them get zero
    counts = torch.tensor([4, 0], dtype=torch.int32, device=DEV)
    rope.apply(x, pos, n_new=counts).sum().backward()
    assert not x.grad[1].any() and not x.grad[0, :, 4:].any() and x.grad[0, :, :4].any()
    with pytest.raises(ValueError):
        rope.apply(x, pos, out=torch.empty_like(x))


def test_other_stream_and_graph():
    from head_wise_kv_b200 import Rope
    rope = Rope(128)
    f, m = O.rope_frequencies(128)
    x = torch.randn(2, 4, 65, 128, device=DEV).to(torch.bfloat16)
    pos = torch.tensor([1, 400], dtype=torch.int32, device=DEV)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        rope.apply(x, pos, out=out)
    torch.cuda.current_stream().wait_stream(side)
    _check(out, x, _spread(pos.cpu().numpy(), 65), f, m, "half", False)
    with torch.cuda.graph(graph):
        rope.apply(x, pos, out=out)
        pos.add_(1)
    for _ in range(3):
        p = pos.clone()
        x.copy_(torch.randn_like(x, dtype=torch.float32))
        graph.replay()
        _check(out, x, _spread(p.cpu().numpy(), 65), f, m, "half", False)


def test_refusals():
    from head_wise_kv_b200 import DuoError, Rope
    rope = Rope(128)
    x = torch.zeros(2, 4, 6, 128, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    for bad in (lambda: rope.apply(x.cpu(), pos), lambda: rope.apply(x[..., :64], pos), lambda: rope.apply(x, pos.cpu()),
                lambda: rope.apply(x, pos[:1]), lambda: rope.apply(x, pos, out=x.float()),
                lambda: rope.apply(x, pos, n_new=pos.cpu()), lambda: rope.apply(x, pos, n_new=pos[:1]),
                lambda: rope.apply(x.transpose(2, 3).contiguous().transpose(2, 3), pos)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises((TypeError, ValueError)):
        rope.apply(x, pos.long())
    with pytest.raises(TypeError):
        rope.apply(x.double(), pos)
    with pytest.raises(DuoError) as e:
        rope.apply(torch.zeros(2, 4, 6, 132, dtype=torch.bfloat16, device=DEV)[..., 2:130], pos)
    assert e.value.code == -6
    rope.close()
    with pytest.raises(DuoError):
        rope.apply(x, pos)


def test_out_that_overlaps_is_refused():
    """out may be x or lie apart from it; a shifted or expanded one would be a race between rows."""
    from head_wise_kv_b200 import Rope
    r = Rope(64)
    flat = torch.arange(3 * 64 * 4, device=DEV, dtype=torch.float32)
    x, shifted = flat[:512].view(1, 2, 4, 64), flat[64:576].view(1, 2, 4, 64)
    pos = torch.zeros(1, dtype=torch.int32, device=DEV)
    keep = flat.clone()
    for out in (shifted, flat[:64].expand(1, 2, 4, 64), x.transpose(1, 2).reshape(1, 4, 2, 64)[:, :2, :1].expand(1, 2, 4, 64)):
        with pytest.raises(ValueError):
            r.apply(x, pos, out=out)
    assert torch.equal(flat, keep)
    want = r.apply(x, pos)
    assert r.apply(x, pos, out=x) is not None and torch.equal(x, want)


def test_out_within_the_storage_of_a_strided_input():
    """Parts of one projection: a shifted part races between rows, one that lies apart or the input itself does not."""
    from head_wise_kv_b200 import Rope
    r = Rope(128)
    pos = torch.tensor([3, 900], dtype=torch.int32, device=DEV)
    qkv = torch.randn(2, 70, 12, 128, device=DEV).to(torch.bfloat16)
    keep = qkv.clone()
    q, by_token = qkv.transpose(1, 2), qkv.transpose(1, 2)[:, :4]
    dense = qkv.view(-1)[:2 * 4 * 70 * 128].view(2, 4, 70, 128)
    for out in (q[:, 1:5], q.as_strided(by_token.shape, by_token.stride(), 64), dense):
        with pytest.raises(ValueError, match="apart"):
            r.apply(by_token, pos, out=out)
        with pytest.raises(ValueError, match="apart"):
            r.launch([(by_token, out, True)], pos)
    with pytest.raises(ValueError, match="itself"):
        r.apply(by_token, pos, out=torch.empty(2 * 200 * 128, device=DEV, dtype=torch.bfloat16).as_strided(
            (2, 4, 70, 128), (200 * 128, 64, 256, 1)))
    other = torch.empty_like(by_token)
    for tensors in ([(q[:, :4], q[:, 4:8], True), (q[:, 4:8], other, True)],         # one's result is another's input
                    [(q[:, :4], other, True), (q[:, 4:8], other, True)]):            # one result for two
        with pytest.raises(ValueError, match="apart"):
            r.launch(tensors, pos)
    assert torch.equal(qkv, keep)
    want = [r.apply(q[:, i:i + 4].contiguous(), pos) for i in (0, 4)]
    r.apply(q[:, :4], pos, out=q[:, 8:])
    assert torch.equal(q[:, 8:], want[0]) and torch.equal(q[:, :8], keep.transpose(1, 2)[:, :8])
    r.launch([(q[:, :4], q[:, :4], True), (q[:, 4:8], q[:, 4:8], True)], pos)        # in place
    assert torch.equal(q[:, :4], want[0]) and torch.equal(q[:, 4:8], want[1])


def test_launch_refusals():
    from head_wise_kv_b200 import Rope
    r = Rope(128)
    x = torch.zeros(2, 4, 6, 128, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)

    def new(t):
        return torch.empty_like(t)
    for tensors in ([], [(x, new(x), True)] * 4, [(x.cpu(), new(x), True)], [(x, new(x), True), (x[:, :, :3], new(x[:, :, :3]), True)],
                    [(x, new(x), True), (x.half(), new(x.half()), True)], [(x, new(x)[:, :3], True)],
                    [(x[..., :64], new(x[..., :64]), True)]):
        with pytest.raises(ValueError):
            r.launch(tensors, pos)
    with pytest.raises(TypeError):
        r.launch([(x.double(), new(x.double()), True)], pos)
    with pytest.raises(ValueError):
        r.launch([(x, new(x), True)], pos[:1])


def test_gradient_that_starts_askew():
    """A contiguous gradient whose storage no 16-byte load may start at: the part of a concatenation."""
    from head_wise_kv_b200 import Rope
    r = Rope(64)
    pos = torch.tensor([5, 8], dtype=torch.int32, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(2, 3, 4, 64, device=DEV).to(dtype).requires_grad_()
        w = torch.randn(1 + x.numel(), device=DEV).to(dtype)
        joined = torch.cat([torch.zeros(1, device=DEV, dtype=dtype), r.apply(x, pos).flatten()])
        grad, = torch.autograd.grad(joined, x, w)
        assert torch.equal(grad, r.apply(w[1:].clone().view(x.shape), pos, transpose=True))
