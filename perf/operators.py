"""Cases of the operators that surround the cache and its attention:

* ``rope``: rotary positions of queries and keys (``Rope.apply``);
* ``append``: rotary positions and the append of a ragged batch of new tokens
  in one call (``DuoKVCache.append_rope``);
* ``reserve``: block tables and slot maps built on the GPU from the requests'
  lengths (``DuoKVCache.reserve``);
* ``attn``: causal attention with a sliding window and sinks, forward and
  backward (``window_attention``): both branches of the gated forward that
  tells retrieval from streaming heads.

``own`` false: the operators in plain torch operations; true: the
framework's calls.  Sizes: the decode, prefill and tiny workloads of this
repository (32 query / 8 KV heads of 128, 4 of 8 KV heads retrieval, sinks and
windows of 64 / 256 and 16 / 64, 4096-token chunks, 65,536-token prompts,
contexts up to 131,072), and batches of a continuously batched server.
"""
import math
import random

import torch

own = False

PAGE = 256
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------- cases
def _rope_case(name, **kw):
    c = dict(op="rope", batch=1, heads=32, n=1, d=128, rot=128, layout="half", scaling="none", factor=1.0,
             original=8192, theta=10000.0, dtype="bf16", token_major=False, per_token=False, transpose=False, far=4096)
    c.update(kw)
    return dict(c, name=name) if name else c


def _append_case(name, **kw):
    c = dict(op="append", hq=32, n_kv=8, n_r=4, d=128, sink=64, window=256, rot=128, layout="half", scaling="none",
             factor=1.0, original=8192, theta=10000.0, kv="bf16", paged=False, decoding=8, prompts=0, chunk=1, pad=0,
             far=4096)
    c.update(kw)
    return dict(c, name=name) if name else c


def _reserve_case(name, **kw):
    c = dict(op="reserve", decoding=8, prompts=0, chunk=1, pad=0, far=131072, spare=64)
    c.update(kw)
    return dict(c, name=name) if name else c


def _attn_case(name, **kw):
    c = dict(op="attn", batch=1, hq=32, n_kv=8, d=128, tokens=4096, sink=64, window=256, token_major=True, ragged=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the queries of one decode step of 8 sequences deep in a 128K context: a latency
        _rope_case("rope decode q", batch=8, n=1, far=131071),
        # the gradient of a small model's packed training batch: fp32, pairs side by side, half of each head rotates
        _rope_case("rope gradient", batch=3, heads=8, n=1021, d=64, rot=32, layout="interleaved", scaling="bands",
                   factor=8.0, dtype="fp32", per_token=True, transpose=True, far=16384),
        # the queries of a 65,536-token prompt, read as the projection leaves them (token-major), written head-major
        _rope_case("rope prompt", n=65536, token_major=True, scaling="yarn", factor=8.0, far=0),
        # one decode step of 8 sequences, one token each
        _append_case("append decode step", decoding=8, far=8192),
        # the last layer of a server's step, where only each sequence's newest token is attended for: 61 sequences
        # decode while three prompts bring 2048-token chunks; FP8 pages
        _append_case("append mixed fp8 pages", kv="fp8", paged=True, decoding=61, prompts=3, chunk=2048, pad=64,
                     far=8192, scaling="bands", factor=8.0, theta=500000.0),
        # the same layer for eight prompts of 8192 tokens; also keys kept without positions that come back to the cache
        _append_case("append prompts", decoding=0, prompts=8, chunk=8192, far=4096),
        # block table and slots of one decode step of 8 long sequences: a latency
        _reserve_case("reserve decode step", decoding=8, far=131072),
        # a server's step: 248 sequences decode, 8 requests start in slots that others have left
        _reserve_case("reserve mixed", decoding=248, prompts=8, chunk=1024, pad=128, far=32768, spare=512),
        # half of 1024 sequences bring a prompt at once, and the pool runs out: the later ones are not served
        _reserve_case("reserve short pool", decoding=512, prompts=512, chunk=512, far=8192, spare=20),
        # a small model's batch of two sequences of odd lengths: a latency
        _attn_case("attn small", batch=2, hq=4, n_kv=4, tokens=257, sink=16, window=64, ragged=True),
        # the full branch of every head over one training sequence
        _attn_case("attn full branch", tokens=4096, sink=0, window=0),
        # the streaming branch over a long one
        _attn_case("attn streaming branch", hq=16, n_kv=4, tokens=8192, window=1024, token_major=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "reserve", "attn"])
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
    scaled = dict(scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                  original=rng.choice([2048, 4096, 8192]), theta=rng.choice([10000.0, 500000.0, 1000000.0]),
                  layout=rng.choice(["half", "interleaved"]))
    d = rng.choice([64, 128, 128])
    if op == "rope":
        heads = rng.choice([1, 4, 8, 32, 64])
        return _rope_case(None, batch=_log_int(rng, 1, 8), heads=heads, n=_log_int(rng, 1, 65536 // heads), d=d,
                          rot=rng.choice([d, d, d // 2, d // 4]), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                          token_major=rng.random() < 0.5, per_token=rng.random() < 0.3, transpose=rng.random() < 0.3,
                          far=_log_int(rng, 1, 1 << 20), **scaled)
    if op == "append":
        n_kv = rng.choice([1, 2, 4, 8])
        paged = d == 128 and rng.random() < 0.5
        return _append_case(None, hq=n_kv * rng.choice([1, 2, 4, 8]), n_kv=n_kv, n_r=rng.randint(0, n_kv), d=d,
                            sink=rng.choice([0, 4, 16, 64]), window=rng.choice([33, 64, 256, 1024]),
                            rot=rng.choice([d, d, d // 2]), kv="fp8" if d == 128 and rng.random() < 0.5 else "bf16",
                            paged=paged, decoding=rng.choice([0, 1, 7, 32]) if not paged else rng.choice([1, 8, 33]),
                            prompts=rng.randint(1, 4), chunk=_log_int(rng, 1, 4096), pad=rng.choice([0, 0, 5, 100]),
                            far=_log_int(rng, 256, 8192), **scaled)
    if op == "attn":
        n_kv, group, batch = rng.choice([1, 2, 4]), rng.choice([1, 2, 4, 8]), rng.randint(1, 3)
        most = int(math.sqrt(32 * 4096 ** 2 / (n_kv * group * batch)))
        return _attn_case(None, batch=batch, hq=n_kv * group, n_kv=n_kv, tokens=_log_int(rng, 20, min(most, 8192)),
                          sink=rng.choice([0, 4, 64, 200]), window=rng.choice([0, 33, 256, 1024]),
                          token_major=rng.random() < 0.5, ragged=rng.random() < 0.5)
    decoding, prompts = _log_int(rng, 1, 700), rng.choice([0, 1, 5, 40, 300])
    return _reserve_case(None, decoding=decoding, prompts=prompts, chunk=_log_int(rng, 1, 512),
                         pad=rng.choice([0, 1, 77]), far=_log_int(rng, 300, 16384),
                         spare=rng.choice([1, 30, 3000]))


# -------------------------------------------------------------- what a case says
def _counts(c):
    """New tokens of each sequence: one for those that decode, then the prompts' chunks, each a little shorter."""
    return [1] * c["decoding"] + [max(1, c["chunk"] - (13 * i) % (c["chunk"] // 2 + 1)) for i in range(c["prompts"])]


def _full_pages(c):
    """Whole pages that each sequence holds before the step: spread over the range; every other prompt is new."""
    top, k = max(1, c["far"] // PAGE), c["decoding"]
    held = [top * (2 * i + 1) // (2 * k) for i in range(k)]
    return held, [0 if i % 2 == 0 else min(top, 1 + i) for i in range(c["prompts"])]


def _row_cap(c):
    return -(-(c["far"] + c["chunk"] + 2 * PAGE) // PAGE) * PAGE


def _max_pages(c):
    return _row_cap(c) // PAGE


def _attn_lengths(c):
    return [c["tokens"] - (c["tokens"] * b // (2 * c["batch"]) if c["ragged"] else 0) for b in range(c["batch"])]


def work(c):
    if c["op"] == "attn":
        pairs, W = 0, c["window"] or c["tokens"]
        for n in _attn_lengths(c):
            whole = min(n, c["sink"] + W)                        # rows that see everything before them
            pairs += whole * (whole + 1) // 2 + (n - whole) * (c["sink"] + W)
        # forward: q, k, v in, out and a log-sum-exp out; backward: those and out's gradient in, three gradients out
        rows = sum(_attn_lengths(c))
        return {"bytes": rows * ((6 * c["hq"] + 6 * c["n_kv"]) * c["d"] * 2 + 8 * c["hq"]),
                "flops": 14 * c["d"] * pairs * c["hq"]}
    if c["op"] == "rope":
        n = c["batch"] * c["heads"] * c["n"] * c["d"]
        size = 4 if c["dtype"] == "fp32" else 2
        pos = c["batch"] * (c["n"] if c["per_token"] else 1) * 4
        return {"bytes": 2 * n * size + pos, "flops": 3 * n * c["rot"] // c["d"]}
    counts = _counts(c)
    T = sum(counts)
    if c["op"] == "append":
        n_s, code = c["n_kv"] - c["n_r"], 1 if c["kv"] == "fp8" else 2
        held = sum(min(n, c["window"]) for n in counts)          # rows that the rings keep
        rows = c["n_r"] * T + n_s * held                         # K rows, and as many V rows
        read = (T * c["hq"] + 2 * rows) * c["d"] * 2 + T * (16 if c["paged"] else 8)
        return {"bytes": read + (T * c["hq"] * 2 + 2 * rows * code) * c["d"],
                "flops": 3 * (T * c["hq"] + rows) * c["rot"]}
    B = len(counts)
    new = sum(-(-n // PAGE) for n in counts[c["decoding"]:])
    # lengths, counts and pages held in; lengths, offsets and pages held out; per token sequence, position and slot;
    # per new page its table entry and its count
    return {"bytes": 24 * B + 16 * (T + c["pad"]) + 8 * new}


# ------------------------------------------------------------------- rotary frequencies
def _inv_freq(c):
    """Angle per position of each pair (radians, 64 bits) and what cosine and sine are multiplied by."""
    rot, s, L = c["rot"], c["factor"], c["original"]
    theta = c["theta"] * (s ** (rot / (rot - 2.0)) if c["scaling"] == "ntk" else 1.0)
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = theta ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        f = f / s
    if c["scaling"] == "yarn":      # pairs that turn often keep their angle, slow ones are stretched, a ramp between
        def pair(turns):            # the pair that makes so many turns over the original length
            return rot * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / s * ramp
    if c["scaling"] == "bands":     # the same by wavelength: 1 and 4 turns over the original length
        ramp = ((L * f / (2 * math.pi) - 1.0) / 3.0).clamp(0, 1)
        f = f / s * (1 - ramp) + f * ramp
    return f, (0.1 * math.log(s) + 1.0 if c["scaling"] == "yarn" and s > 1 else 1.0)


def _own_rope(c):
    from head_wise_kv_b200 import Rope
    return Rope(c["d"], rot_dim=c["rot"], theta=c["theta"], layout=c["layout"], scaling=c["scaling"],
                factor=c["factor"], original_len=c["original"])


# ----------------------------------------------------------------------------- prepare
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _lengths(c, g):
    """(tokens held, tokens new, pages held): the decoding sequences in an order of the seed's."""
    dec, pro = _full_pages(c)
    order = torch.randperm(len(dec), generator=g, device=DEV)
    full = torch.cat([torch.tensor(dec, dtype=torch.int32, device=DEV)[order],
                      torch.tensor(pro, dtype=torch.int32, device=DEV)])
    part = _ints(g, 0, PAGE - 1, len(dec) + len(pro))
    new = torch.zeros_like(full)
    new[len(dec):] = (torch.tensor(pro, dtype=torch.int32, device=DEV) == 0).int()
    before = (full * PAGE + part) * (1 - new)                    # a request that starts holds nothing
    held = -(-before // PAGE) + new * (1 + torch.arange(full.numel(), device=DEV) % 5)   # pages of the one that left
    return before.int(), torch.tensor(_counts(c), dtype=torch.int32, device=DEV), held.int()


def _prepare_rope(c, g):
    dt = DTYPES[c["dtype"]]
    shape = (c["batch"], c["heads"], c["n"], c["d"])
    x = _normal(g, *((shape[0], shape[2], shape[1], shape[3]) if c["token_major"] else shape), dtype=dt)
    x = x.transpose(1, 2) if c["token_major"] else x
    start = _ints(g, 0, c["far"] + 1, c["batch"])
    pos = start
    if c["per_token"]:                                           # packed rows: positions start over inside a row
        pos = (start[:, None] + torch.arange(c["n"], device=DEV, dtype=torch.int32)) % (c["far"] // 2 + 1)
    s = {"case": c, "x": x, "positions": pos.int().contiguous()}
    if own:
        s["rope"] = _own_rope(c)
        s["out"] = torch.empty(shape, dtype=dt, device=DEV)
    else:
        s["freq"], s["magnitude"] = _inv_freq(c)
        s["freq"] = s["freq"].to(DEV)
    return s


def _prepare_append(c, g):
    before, count, _ = _lengths(c, g)
    B, T, d, SW = len(before), sum(_counts(c)) + c["pad"], c["d"], c["sink"] + c["window"]
    n_s = c["n_kv"] - c["n_r"]
    heads = torch.randperm(c["n_kv"], generator=torch.Generator().manual_seed(5)).tolist()
    retrieval = sorted(heads[:c["n_r"]])
    streaming = sorted(heads[c["n_r"]:])
    cap = _row_cap(c)
    qkv = _normal(g, T, c["hq"] + 2 * c["n_kv"], d)              # one projection's output, as the matrix product leaves it
    s = {"case": c, "before": before, "count": count, "after": before + count,
         "q": qkv[:, :c["hq"]], "k": qkv[:, c["hq"]:c["hq"] + c["n_kv"]], "v": qkv[:, c["hq"] + c["n_kv"]:],
         "q_out": torch.zeros(T, c["hq"], d, dtype=torch.bfloat16, device=DEV)}
    # the token map of the step: sequence, position and row of each token; -1 behind the last one
    cu = torch.cumsum(count, 0)
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(cu, t, right=True)
    at = seq.clamp(max=B - 1)
    pos = before[at] + (t - (cu - count)[at])
    seq = torch.where(t < cu[-1], seq, -1)
    s["seq"], s["pos"] = seq.int(), torch.where(seq >= 0, pos, -1).int()
    if c["paged"]:
        need = before.long() // PAGE + 1                         # pages of each sequence after the step, or one more
        need[c["decoding"]:] += -(-count[c["decoding"]:].long() // PAGE)
        total = int(need.sum())
        pages = torch.randperm(total, generator=g, device=DEV)   # in no order, as a running server has them
        j = torch.arange(cap // PAGE, device=DEV)[None]
        rank = (torch.cumsum(need, 0) - need)[:, None] + j
        table = torch.where(j < need[:, None], pages[rank.clamp(max=total - 1)], -1).int().contiguous()
        page = table[at, (pos // PAGE).clamp(max=cap // PAGE - 1)].long()
        s["slot"] = torch.where(seq >= 0, page * PAGE + pos % PAGE, -1)
        lead = (total, PAGE)
    else:
        s["slot"] = torch.where(seq >= 0, at * cap + pos, -1)
        lead = (B, cap)
    # what the caches hold before; FP8 codes with scale 1, so that a code is the value that it stands for
    dt = torch.float8_e4m3fn if c["kv"] == "fp8" else torch.bfloat16
    s["kr"], s["vr"] = (_normal(g, lead[0], c["n_r"], lead[1], d).to(dt) for _ in range(2))
    s["ks"], s["vs"] = (_normal(g, B, n_s, SW, d).to(dt) for _ in range(2))
    slot = torch.arange(SW, device=DEV)[None]
    last = before[:, None] - 1                                   # position held by each slot of the rings
    ring = last - (last - slot) % c["window"] if c["sink"] == 0 else \
        torch.where(slot < c["sink"], slot, last - (last - c["sink"] - (slot - c["sink"])) % c["window"])
    s["positions"] = torch.where((ring >= 0) & (ring <= last) & ((slot < c["sink"]) | (ring >= c["sink"])), ring,
                                 -1).int().contiguous()
    if own:
        from head_wise_kv_b200 import DuoKVCache, TokenMap
        mask = torch.zeros(1, c["n_kv"], dtype=torch.uint8)
        mask[0, retrieval] = 1
        paged = dict(page_tokens=PAGE, num_pages=lead[0]) if c["paged"] else {}
        cache = DuoKVCache(1, B, c["hq"], c["n_kv"], d, c["sink"], c["window"], cap, mask.numpy(), device=DEV,
                           kv_dtype=c["kv"], **paged)
        view = cache.layer_views(0)
        for name, key in (("kr", "k_retrieval"), ("vr", "v_retrieval"), ("ks", "k_streaming"), ("vs", "v_streaming")):
            view[key].view(dt).copy_(s[name])
            s[name] = view[key].view(dt)
        view["positions"].copy_(s["positions"])
        s["positions"] = view["positions"]
        tokens = TokenMap(B, T, cache.device)
        tokens.seq.copy_(s["seq"])
        tokens.pos.copy_(s["pos"])
        tokens.slot.copy_(s["slot"])
        tokens.len_after.copy_(s["after"])
        if c["paged"]:
            cache.set_page_table(table)
        s.update(cache=cache, tokens=tokens, rope=_own_rope(c))
    else:
        s["freq"], s["magnitude"] = _inv_freq(c)
        s.update(freq=s["freq"].to(DEV), retrieval=retrieval, streaming=streaming)
    return s


def _prepare_reserve(c, g):
    before, count, held = _lengths(c, g)
    B, T, width = len(before), sum(_counts(c)) + c["pad"], _max_pages(c)
    dec, pro = _full_pages(c)
    left = [1 + (len(dec) + i) % 5 for i in range(len(pro))]      # pages of the requests that have left
    pages = sum(p + 1 for p in dec) + sum(p + 1 if p else n for p, n in zip(pro, left)) + c["spare"]
    s = {"case": c, "before": before, "count": count, "T": T, "pages": pages}
    if own:
        from head_wise_kv_b200 import DuoKVCache, TokenMap
        cache = DuoKVCache(1, B, 1, 1, 128, 0, 1, _row_cap(c), [[1]], device=DEV, kv_dtype="int4", page_tokens=PAGE,
                           num_pages=pages)
        cache.manage_pages(width)
        # the server's earlier steps: every sequence has got its pages
        cache.reserve(torch.zeros_like(before), (held * PAGE).contiguous())
        s.update(cache=cache, tokens=TokenMap(B, T, cache.device), view=cache.page_state())
    else:
        first = (torch.cumsum(held, 0) - held)[:, None]
        j = torch.arange(width, device=DEV)[None]
        s["table"] = torch.where(j < held[:, None], first + j, -1).int()
        s["refs"] = (torch.arange(pages, device=DEV) < held.sum()).int()
        s["held"] = held
    return s


def _prepare_attn(c, g):
    s = {"case": c}
    for name, heads in (("q", c["hq"]), ("k", c["n_kv"]), ("v", c["n_kv"]), ("grad", c["hq"])):
        x = _normal(g, c["batch"], *((c["tokens"], heads) if c["token_major"] else (heads, c["tokens"])), c["d"])
        s[name] = x.transpose(1, 2) if c["token_major"] else x
    s["lengths"] = torch.tensor(_attn_lengths(c), dtype=torch.int32, device=DEV) if c["ragged"] else None
    if own:
        from head_wise_kv_b200 import window_attention
        s["attention"] = window_attention
        for name in ("q", "k", "v"):
            s[name].requires_grad_()
    return s


def prepare(case, seed):
    g = _gen(seed)
    return {"rope": _prepare_rope, "append": _prepare_append, "reserve": _prepare_reserve,
            "attn": _prepare_attn}[case["op"]](case, g)


# ------------------------------------------------------------------------- plain forms
def _cos_sin(s, positions):
    angle = positions.double()[..., None] * s["freq"]            # far positions: 64 bits
    return (torch.cos(angle) * s["magnitude"]).float(), (torch.sin(angle) * s["magnitude"]).float()


def _rotate(c, x, cos, sin):
    """x in 32 bits [..., d]; cos, sin broadcast against [..., rot / 2]."""
    rot = c["rot"]
    if c["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    y = x.clone()
    if c["layout"] == "half":
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    else:
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    return y


def _plain_rope(s):
    c, x = s["case"], s["x"]
    pos = s["positions"]
    if not c["per_token"]:
        pos = pos[:, None] + torch.arange(c["n"], device=DEV, dtype=torch.int32)
    cos, sin = _cos_sin(s, pos)
    if c["transpose"]:
        sin = -sin
    return _rotate(c, x.float(), cos[:, None], sin[:, None]).to(x.dtype)


def _as_cached(x, dtype):
    return x.clamp(-448, 448).to(dtype).view(torch.uint8) if dtype == torch.float8_e4m3fn else x.to(dtype)


def _plain_append(s):
    c = s["case"]
    dt = s["kr"].dtype
    store = (lambda t: t.view(torch.uint8)) if dt == torch.float8_e4m3fn else (lambda t: t)
    cos, sin = _cos_sin(s, s["pos"])
    cos, sin = cos[:, None], sin[:, None]
    here = (s["seq"] >= 0).nonzero()[:, 0]
    seq, pos, slot = s["seq"][here].long(), s["pos"][here].long(), s["slot"][here]
    q = _rotate(c, s["q"].float(), cos, sin).to(torch.bfloat16)
    q_out = torch.where((s["seq"] >= 0)[:, None, None], q, s["q_out"])
    k = _as_cached(_rotate(c, s["k"].float(), cos, sin), dt)[here]
    v = _as_cached(s["v"].float(), dt)[here]
    if c["n_r"] > 0:
        rows = PAGE if c["paged"] else s["kr"].shape[2]
        store(s["kr"])[slot // rows, :, slot % rows] = k[:, s["retrieval"]]
        store(s["vr"])[slot // rows, :, slot % rows] = v[:, s["retrieval"]]
    S, W = c["sink"], c["window"]
    kept = ((pos < S) | (pos >= s["after"][seq] - W)).nonzero()[:, 0]
    seq, pos = seq[kept], pos[kept]
    at = torch.where(pos < S, pos, S + (pos - S) % W)
    if c["n_r"] < c["n_kv"]:
        store(s["ks"])[seq, :, at] = k[kept][:, s["streaming"]]
        store(s["vs"])[seq, :, at] = v[kept][:, s["streaming"]]
    fresh = (s["before"] == 0)[:, None] & (torch.arange(S + W, device=DEV)[None] >= s["count"][:, None])
    s["positions"].masked_fill_(fresh, -1)
    s["positions"][seq, at] = pos.int()
    return q_out


def _plain_reserve(s):
    T, pages = s["T"], s["pages"]
    before, count, held, table = (s[k].long() for k in ("before", "count", "held", "table"))
    j = torch.arange(table.shape[1], device=DEV)[None]
    last = -(-before // PAGE)                                    # pages that hold tokens stay, the rest go back
    keep = torch.minimum(held, last)
    back = (j >= keep[:, None]) & (j < held[:, None])
    refs = s["refs"].long().index_add(0, table[back], torch.full_like(table[back], -1))
    table = torch.where(j < keep[:, None], table, -1)
    free = (refs == 0).nonzero()[:, 0]
    tail = table.gather(1, (keep - 1).clamp(min=0)[:, None])[:, 0]
    shared = (count > 0) & (before % PAGE != 0) & (keep == last) & (refs[tail.clamp(min=0)] > 1)
    total = -(-(before + count) // PAGE)
    valid = ~shared & (total <= table.shape[1])
    need = torch.where(valid, (total - keep).clamp(min=0), 0)
    tokens = torch.where(valid, count, 0)
    served = valid & ((need == 0) | (torch.cumsum(need, 0) <= free.numel())) & (torch.cumsum(tokens, 0) <= T)
    need, tokens = torch.where(served, need, 0), torch.where(served, tokens, 0)
    rank = (torch.cumsum(need, 0) - need - keep)[:, None] + j    # of a new page among the free ones, lowest first
    new = (j >= keep[:, None]) & (j < (keep + need)[:, None])
    table = torch.where(new, free[torch.where(new, rank, 0)], table)
    refs = refs.index_fill(0, free[:int(need.sum())], 1)
    after = torch.where(served, before + count, before)
    cu = torch.cat([count.new_zeros(1), torch.cumsum(tokens, 0)])
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(cu[1:], t, right=True)
    at = seq.clamp(max=len(before) - 1)
    pos = before[at] + t - cu[at]
    real = t < cu[-1]
    page = table[at, torch.where(real, pos // PAGE, 0)]
    return {"table": table.int(), "held": (keep + need).int(), "refs": refs.int(), "len_after": after.int(),
            "cu": cu.int(), "seq": torch.where(real, seq, -1).int(), "pos": torch.where(real, pos, -1).int(),
            "slot": torch.where(real, page * PAGE + pos % PAGE, -1)}


def _visible(c, lengths):
    """Which keys (last) each row (before it) sees: [1 or batch][1][tokens][tokens]."""
    i, j = torch.arange(c["tokens"], device=DEV)[:, None], torch.arange(c["tokens"], device=DEV)[None]
    sees = (j <= i)[None, None]
    if c["window"]:
        sees = sees & ((j < c["sink"]) | (j > i - c["window"]))
    return sees if lengths is None else sees & (i < lengths[:, None, None, None])


def _plain_attn(s):
    c = s["case"]
    group, scale = c["hq"] // c["n_kv"], c["d"] ** -0.5
    q, k, v, grad = (s[name].float() for name in ("q", "k", "v", "grad"))
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    sees = _visible(c, s["lengths"])
    score = torch.matmul(q, k.transpose(2, 3)).mul_(scale).masked_fill_(~sees, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score.sub_(torch.where(top == -math.inf, 0.0, top)))
    del score
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, 1.0, total))                  # a row that sees nothing is zero
    out = torch.matmul(p, v)
    dv = torch.matmul(p.transpose(2, 3), grad)
    dp = torch.matmul(grad, v.transpose(2, 3))
    ds = dp.sub_((grad * out).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    shape = (c["batch"], c["n_kv"], group, c["tokens"], c["d"])  # query heads that share a key head
    return [out.to(torch.bfloat16), dq.to(torch.bfloat16), dk.view(shape).sum(2).to(torch.bfloat16),
            dv.view(shape).sum(2).to(torch.bfloat16)]


# --------------------------------------------------------------------------------- run
def run(s):
    c = s["case"]
    if c["op"] == "rope":
        if own:
            return s["rope"].apply(s["x"], s["positions"], transpose=c["transpose"], out=s["out"])
        return _plain_rope(s)
    if c["op"] == "append":
        if own:
            q = s["cache"].append_rope(0, s["rope"], s["q"], s["k"], s["v"], s["before"], s["tokens"], out=s["q_out"])
        else:
            q = _plain_append(s)
        return [q, s["kr"], s["vr"], s["ks"], s["vs"], s["positions"]]
    if c["op"] == "attn":
        if own:
            x = (s["q"], s["k"], s["v"])
            out = s["attention"](*x, c["sink"], c["window"] or None, lengths=s["lengths"])
            return [out.detach(), *torch.autograd.grad(out, x, s["grad"])]
        return _plain_attn(s)
    if own:
        m = s["cache"].reserve(s["before"], s["count"], s["tokens"])
        return {"table": s["view"]["table"], "held": s["view"]["held"], "refs": s["view"]["refs"],
                "len_after": m.len_after, "cu": m.cu, "seq": m.seq, "pos": m.pos, "slot": m.slot}
    return _plain_reserve(s)


# ------------------------------------------------------------------------------- exact
def _exact_rotated(c, x, pos, back=False):
    """Each pair as a complex number times magnitude * e^(i angle), in 64 bits; x [..., d], pos broadcast against [...]."""
    f, m = _inv_freq(c)
    angle = pos.double()[..., None] * f.to(x.device)
    turn = torch.polar(torch.full_like(angle, m), -angle if back else angle)
    h = c["rot"] // 2
    pairs = x[..., :c["rot"]].double()
    pairs = pairs.unflatten(-1, (2, h)).movedim(-2, -1) if c["layout"] == "half" else pairs.unflatten(-1, (h, 2))
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = (y.movedim(-1, -2) if c["layout"] == "half" else y).flatten(-2)
    return torch.cat([y, x[..., c["rot"]:].double()], -1)


def _exact_attn(c, s):
    lens = _attn_lengths(c)
    got = [torch.zeros(c["batch"], h, c["tokens"], c["d"], dtype=torch.float64, device=DEV)
           for h in (c["hq"], c["hq"], c["n_kv"], c["n_kv"])]
    for b, n in enumerate(lens):
        at = torch.arange(n, device=DEV)
        hidden = (at[None] > at[:, None]) | ((at[None] <= at[:, None] - (c["window"] or n)) & (at[None] >= c["sink"]))
        for h in range(c["hq"]):
            g = h * c["n_kv"] // c["hq"]
            q, k, v, do = (s[x][b, i, :n].double() for x, i in (("q", h), ("k", g), ("v", g), ("grad", h)))
            w = torch.softmax((q @ k.T / math.sqrt(c["d"])).masked_fill(hidden, -math.inf), -1)
            o = w @ v
            got[0][b, h, :n] = o
            got[3][b, g, :n] += w.T @ do
            slope = w * (do @ v.T - (do * o).sum(-1, keepdim=True)) / math.sqrt(c["d"])
            got[1][b, h, :n] = slope @ k
            got[2][b, g, :n] += slope.T @ q
    return got


def exact(case, seed):
    if case["op"] == "reserve":
        return None                                              # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(case, s)
    if case["op"] == "rope":
        out = []
        for b in range(case["batch"]):
            at = s["positions"][b].long()
            at = at if case["per_token"] else at + torch.arange(case["n"], device=DEV)
            out.append(torch.stack([_exact_rotated(case, s["x"][b, h], at, case["transpose"])
                                    for h in range(case["heads"])]))
        return torch.stack(out)
    q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=DEV)
    kr, vr, ks, vs = (s[k].float().double() for k in ("kr", "vr", "ks", "vs"))
    S, W = case["sink"], case["window"]
    ret, stre = s["retrieval"], s["streaming"]
    first = 0
    for b, (n, at) in enumerate(zip(s["count"].tolist(), s["before"].tolist())):
        t = slice(first, first + n)
        pos = at + torch.arange(n, device=DEV)
        q[t] = _exact_rotated(case, s["q"][t], pos[:, None])
        k, v = _exact_rotated(case, s["k"][t], pos[:, None]), s["v"][t].double()
        slot = s["slot"][t]
        rows = kr.shape[2]
        for i, h in enumerate(ret):
            kr[slot // rows, i, slot % rows] = k[:, h]
            vr[slot // rows, i, slot % rows] = v[:, h]
        for p in [p for p in range(at, at + n) if p < S or p >= at + n - W]:
            place = p if p < S else S + (p - S) % W
            ks[b, :, place] = k[p - at, stre]
            vs[b, :, place] = v[p - at, stre]
        first += n
    return [q, kr, vr, ks, vs, None]
