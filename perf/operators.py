"""What is measured of the rotary, paged-cache and sink-window operators.

Each case is one call, or one training step, of an operator next to this
library's attention: rotary positions (forward and backward), appending keys
and values to a paged cache with the rotation on the way, attention over that
cache (8-bit with a scale for each page and head, or in the queries' type), and
packed attention with a sliding window and a few first tokens that stay
visible (forward and backward).  `run` computes them in their plain form from
elementary torch operations, or, with `own`, through this library's entry
points; `exact` gives the same results from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------

def _rotary(name, **over):
    c = {"name": name, "op": "rotary", "direction": "forward", "tokens": 64, "heads_q": 32, "heads_kv": 8,
         "head_dim": 128, "rotary_dim": 128, "interleaved": False, "scaling": "none", "factor": 1.0,
         "last_position": 8191, "dtype": "bf16"}
    return {**c, **over}


def _append(name, **over):
    c = {"name": name, "op": "append", "seqs": 64, "new_min": 1, "new_max": 1, "held_min": 0, "held_max": 2047,
         "heads_q": 32, "heads_kv": 8, "head_dim": 128, "rotary_dim": 128, "interleaved": False, "page": 64,
         "cache": "e4m3", "dtype": "bf16"}
    return {**c, **over}


def _paged(name, **over):
    c = {"name": name, "op": "paged", "seqs": 1, "q_len": 1, "kv_min": 1, "kv_max": 1000, "heads_q": 32,
         "heads_kv": 8, "head_dim": 128, "page": 64, "window": 0, "sinks": 0, "cache": "e4m3", "dtype": "bf16"}
    return {**c, **over}


def _window(name, **over):
    c = {"name": name, "op": "window", "direction": "forward", "seqs": 8, "len_min": 256, "len_max": 2048,
         "heads": 8, "head_dim": 128, "window": 512, "sinks": 4, "dtype": "bf16"}
    return {**c, **over}


def listed():
    return [
        # the queries and keys of one decoding step of 64 sequences: a few microseconds, latency counts
        _rotary("rotary_decode", last_position=131071),
        # a training batch of 16k packed tokens with positions scaled for a long context, both directions
        _rotary("rotary_train", direction="both", tokens=16384, scaling="yarn", factor=8.0, last_position=65535),
        # interleaved pairs in part of an odd-sized head, 32 bits, the gradients alone
        _rotary("rotary_partial", direction="backward", tokens=5003, heads_q=12, heads_kv=12, head_dim=96,
                rotary_dim=64, interleaved=True, scaling="linear", factor=4.0, dtype="f32"),
        # one new token of each of 64 sequences into an 8-bit cache
        _append("append_decode_8bit"),
        # the prompts of eight requests (256 to 2048 tokens) into an 8-bit cache
        _append("append_prompt_8bit", seqs=8, new_min=256, new_max=2048, held_max=0),
        # speculative tokens of 129 sequences, pairs interleaved, into a 16-bit cache of small pages
        _append("append_spec_16bit", seqs=129, new_min=1, new_max=7, heads_q=16, heads_kv=4, head_dim=64,
                rotary_dim=64, interleaved=True, page=16, cache="f16", dtype="f16", held_max=1023),
        # one user alone, a context of a thousand tokens: latency counts
        _paged("paged_single_8bit", kv_min=1000),
        # a full serving batch with contexts from 1k to 16k tokens, 8-bit cache
        _paged("paged_batch_8bit", seqs=64, kv_min=1024, kv_max=16384),
        # long streams of which a window and the first tokens stay visible
        _paged("paged_window_8bit", seqs=16, kv_min=32768, kv_max=65536, window=8192, sinks=4, page=128),
        # checking five speculative tokens of each of 16 sequences against a 16-bit cache of small pages
        _paged("paged_verify_16bit", seqs=16, q_len=5, kv_min=1, kv_max=4097, heads_q=16, heads_kv=4, head_dim=64,
               page=16, cache="bf16"),
        # the packed sequences of this library's own packed workload, window 512, four first tokens
        _window("window_prompt"),
        # a training step on long packed sequences
        _window("window_train", direction="both", seqs=3, len_min=777, len_max=8192, heads=8, head_dim=64,
                window=1024, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "paged", "window"])
    if op == "rotary":
        hk, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 256])
        c = _rotary("", direction=rng.choice(["forward", "backward", "both"]), heads_kv=hk,
                    heads_q=hk * rng.choice([1, 2, 4, 8]), head_dim=d, rotary_dim=rng.choice([d, d // 2, 32]),
                    interleaved=rng.random() < 0.5, last_position=_log(rng, 1000, 1 << 20),
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
        c["scaling"] = rng.choice(["none", "linear", "ntk", "yarn"])
        c["factor"] = 1.0 if c["scaling"] == "none" else rng.choice([2.0, 4.0, 8.0, 32.0])
        row = (c["heads_q"] + hk) * d * _BYTES[c["dtype"]]
        c["tokens"] = min(_log(rng, 1, 16384), (16384 * 40 * 128 * 2) // row)
    elif op == "append":
        hk, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 256])
        many = rng.random() < 0.4
        c = _append("", seqs=_log(rng, 1, 8 if many else 256), new_max=_log(rng, 16, 2048) if many else
                    rng.choice([1, 1, 1, 4, 7]), heads_kv=hk, heads_q=hk * rng.choice([1, 2, 4, 8]), head_dim=d,
                    rotary_dim=rng.choice([d, d // 2]), interleaved=rng.random() < 0.5,
                    page=rng.choice([16, 32, 64, 128]), held_max=_log(rng, 16, 1000),
                    dtype=rng.choice(["bf16", "bf16", "f16"]))
        c["new_min"] = max(1, c["new_max"] // rng.choice([1, 2, 8]))
        c["cache"] = rng.choice(["e4m3", "e4m3", c["dtype"]])
    elif op == "paged":
        hk, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 256])
        c = _paged("", seqs=_log(rng, 1, 128), q_len=rng.choice([1, 1, 1, 2, 5, 8]), heads_kv=hk,
                   heads_q=hk * rng.choice([1, 2, 4, 8]), head_dim=d, page=rng.choice([16, 32, 64, 128]),
                   dtype=rng.choice(["bf16", "bf16", "f16"]))
        c["cache"] = rng.choice(["e4m3", "e4m3", c["dtype"]])
        if rng.random() < 0.1:
            c["dtype"] = c["cache"] = "f32"
        most = (64 * 8700 * 8 * 128) // (c["seqs"] * hk * d * _BYTES[c["cache"]])
        c["kv_max"] = max(c["q_len"], min(_log(rng, 16, 65536), most))
        c["kv_min"] = max(1, c["kv_max"] // rng.choice([1, 4, 100]))
        if rng.random() < 0.4:
            c["window"], c["sinks"] = _log(rng, 16, 8192), rng.choice([0, 1, 4, 64])
    else:
        c = _window("", direction=rng.choice(["forward", "both"]), seqs=rng.choice([1, 2, 3, 8]),
                    len_max=_log(rng, 64, 6000), heads=rng.choice([1, 2, 4, 8]), head_dim=rng.choice([32, 64, 96, 128]),
                    window=_log(rng, 16, 2048), sinks=rng.choice([0, 1, 4, 64, 130]),
                    dtype=rng.choice(["bf16", "bf16", "f16"]))
        # no more products than the largest listed step has, dense and within the window
        while c["seqs"] * c["heads"] * c["head_dim"] * c["len_max"] * min(3000, c["len_max"]) > 8 * 64 * 13969 * 1500:
            c["len_max"] //= 2
        if rng.random() < 0.1:
            c["dtype"], c["len_max"] = "f32", min(c["len_max"], 1000)
        c["len_min"] = max(1, c["len_max"] // rng.choice([1, 2, 8]))
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, in an order of their own that the sizes alone fix."""
    v = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]
    np.random.RandomState(n).shuffle(v)
    v[0] = hi if n == 1 else v[0]
    return v


def _lengths(c):
    """(new tokens, held tokens after the call) of every sequence: plain lists that follow from the case."""
    if c["op"] == "append":
        new = _spread(c["new_min"], c["new_max"], c["seqs"])
        return new, [n + h for n, h in zip(new, reversed(_spread(c["held_min"], c["held_max"], c["seqs"])))]
    if c["op"] == "paged":
        held = [max(n, c["q_len"]) for n in _spread(c["kv_min"], c["kv_max"], c["seqs"])]
        return [c["q_len"]] * c["seqs"], held
    new = _spread(c["len_min"], c["len_max"], c["seqs"])
    return new, new


def _visible(c, position):
    """Keys that a token at `position` sees."""
    n = position + 1
    return n if not c["window"] or n <= c["window"] else c["window"] + min(c["sinks"], n - c["window"])


def work(case):
    c, e = case, _BYTES[case["dtype"]]
    if c["op"] == "rotary":
        n = c["tokens"] * (c["heads_q"] + c["heads_kv"])
        times = 2 if c["direction"] == "both" else 1
        return {"bytes": times * (2 * n * c["head_dim"] * e + 4 * c["tokens"]), "flops": times * 3 * n * c["rotary_dim"]}
    new, held = _lengths(c)
    if c["op"] == "append":
        t, pages = sum(new), sum((h - 1) // c["page"] - (h - n) // c["page"] + 1 for n, h in zip(new, held))
        scales = 2 * 2 * 4 * pages * c["heads_kv"] if c["cache"] == "e4m3" else 0
        return {"bytes": t * c["head_dim"] * (2 * c["heads_q"] * e + 2 * c["heads_kv"] * (e + _BYTES[c["cache"]])) + scales,
                "flops": 3 * t * (c["heads_q"] + c["heads_kv"]) * c["rotary_dim"]}
    if c["op"] == "paged":
        hq, d = c["heads_q"], c["head_dim"]
        pairs = sum(_visible(c, h - n + i) for n, h in zip(new, held) for i in range(n))
        keys = sum(min(h, _visible(c, h - 1) + (n - 1 if c["window"] else 0)) for n, h in zip(new, held))
        scales = 2 * 4 * (keys // c["page"]) * c["heads_kv"] if c["cache"] == "e4m3" else 0
        return {"bytes": 2 * keys * c["heads_kv"] * d * _BYTES[c["cache"]] + scales + sum(new) * hq * (2 * d * e + 4),
                "flops": 4 * pairs * hq * d}
    pairs = sum(sum(_visible(c, i) for i in range(n)) for n in new) * c["heads"]
    row = sum(new) * c["heads"] * c["head_dim"] * e
    if c["direction"] == "forward":
        return {"bytes": 4 * row + 4 * sum(new) * c["heads"], "flops": 4 * pairs * c["head_dim"]}
    return {"bytes": 12 * row + 8 * sum(new) * c["heads"], "flops": 14 * pairs * c["head_dim"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

_BASE, _ORIGINAL = 10000.0, 8192


def _frequencies(c):
    """Radians a position of each rotated pair, and the factor on cos and sin, in 64 bits."""
    dim, scaling, s = c["rotary_dim"], c.get("scaling", "none"), c.get("factor", 1.0)
    base = _BASE * s ** (dim / (dim - 2)) if scaling == "ntk" else _BASE
    f = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    if scaling == "linear":
        f = f / s
    if scaling == "yarn":  # by parts: pairs that turn over 32 times in the first context keep their speed
        keep = ((_ORIGINAL * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / s
    return f, 0.1 * math.log(s) + 1.0 if scaling == "yarn" and s > 1 else 1.0


def _plan(c, dev):
    import masked_attention_tri_gb300 as ta
    scaling = c.get("scaling", "none")
    return ta.Rotary(c["rotary_dim"], _BASE, interleaved=c["interleaved"], scaling=None if scaling == "none" else scaling,
                     factor=c.get("factor", 1.0), original_length=_ORIGINAL, device=dev)


def prepare(case, seed):
    c, dev = case, torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(int(seed))
    t = _TYPES[c["dtype"]]

    def randn(*shape, dtype=t, by=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16) * by).to(dtype)

    s = {"case": c}
    if c["op"] == "rotary":
        n, d = c["tokens"], c["head_dim"]
        s["positions"] = torch.randint(0, c["last_position"] + 1, (n,), generator=g, device=dev, dtype=torch.int32)
        if c["direction"] != "backward":
            s["q"], s["k"] = randn(n, c["heads_q"], d), randn(n, c["heads_kv"], d)
        if c["direction"] != "forward":
            s["gq"], s["gk"] = randn(n, c["heads_q"], d), randn(n, c["heads_kv"], d)
    elif c["op"] in ("append", "paged"):
        new, held = _lengths(c)
        total, S, hk, d, P = sum(new), len(new), c["heads_kv"], c["head_dim"], c["page"]
        s["q"] = randn(total, c["heads_q"], d, by=1.0 if c["op"] == "append" else 1.5)
        pages = [-(-h // P) for h in held]
        most = max(pages)
        order = torch.randperm(sum(pages), generator=g, device=dev).to(torch.int32)
        first = torch.tensor(np.cumsum([0] + pages[:-1]), device=dev)
        at = torch.arange(most, device=dev)
        s["table"] = order[(first[:, None] + at.clamp(max=most)).clamp(max=sum(pages) - 1)].contiguous()
        s["lengths"] = torch.tensor(held, dtype=torch.int32, device=dev)
        s["cu"] = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device=dev)
        s["max_new"] = max(new)
        shape = (sum(pages), hk, P, d)
        for x in ("k", "v"):
            if c["cache"] == "e4m3":
                codes = randn(*shape, dtype=torch.bfloat16, by=90.0).clamp_(-448, 448)
                s[x + "_cache"] = codes.to(torch.float8_e4m3fn)
                s[x + "_scale"] = torch.exp2(torch.randint(-7, -4, shape[:2], generator=g, device=dev).float())
            else:
                s[x + "_cache"], s[x + "_scale"] = randn(*shape), None
        if c["op"] == "append":
            # a few channels of the keys are far larger than the others, as in trained models
            s["k"] = (randn(total, hk, d) * (1 + 15 * (torch.arange(d, device=dev) % 61 == 7))).to(t)
            s["v"] = randn(total, hk, d)
    else:
        new, _ = _lengths(c)
        total, h, d = sum(new), c["heads"], c["head_dim"]
        for x in ("q", "k", "v") + (("g",) if c["direction"] == "both" else ()):
            s[x] = randn(total, h, d)
        s["cu"] = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device=dev)
        s["max_new"] = max(new)
    if c["op"] in ("rotary", "append"):
        f, s["mscale"] = _frequencies(c)
        s["frequencies"] = f.to(dev)
        if own:
            s["rotary"] = _plan(c, dev)
    if own and "k_cache" in s:  # the handle that a serving program keeps for the cache's memory
        import masked_attention_tri_gb300 as ta
        s["handle"] = ta.PagedKVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return s


# ---------------------------------------------------------------------------
# The plain forms, in 32 bits (W)
# ---------------------------------------------------------------------------

W = torch.float32


def _turn(x, positions, frequencies, mscale, interleaved, back):
    """x (tokens, heads, d) with the leading pairs turned by position * frequency; the angles in 64 bits."""
    half = frequencies.numel()
    angle = positions.double()[:, None] * frequencies
    cos, sin = (angle.cos() * mscale).to(W)[:, None], (angle.sin() * mscale).to(W)[:, None]
    if back:
        sin = -sin
    x = x.to(W)
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    u, w = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((r, rest), -1)


def _token_places(cu, total):
    """(sequence, place in it) of every packed token."""
    t = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu[1:].long().contiguous(), t, right=True)
    return seq, t - cu.long()[seq]


def _e4m3(x):
    return x.float().to(torch.float8_e4m3fn)


def _scale_for(most):
    """The smallest power of two that brings `most` to 448 or below, within 2**-56 and 2**56."""
    m, e = torch.frexp(most)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-56, 56)
    return torch.where(most > 0, torch.exp2(e.to(most.dtype)), torch.full_like(most, 2.0 ** -56))


def _append_plain(s, q, k, v, caches):
    """Rotates q and k and writes k and v into `caches` (in place): {"k": (codes or values, scale), "v": ...}."""
    c, P = s["case"], s["case"]["page"]
    seq, pos = _token_places(s["cu"], k.shape[0])
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    lengths, table = s["lengths"].long(), s["table"].long()
    start = lengths - new
    slot = start[seq] + pos
    turn = (slot, s["frequencies"], s["mscale"], c["interleaved"], False)
    rows = {"k": _turn(k, *turn), "v": v.to(W)}
    page, off = table[seq, slot // P], slot % P
    for x, (cache, scale) in caches.items():
        if scale is None:
            cache[page, :, off] = rows[x].to(cache.dtype)
            continue
        # the pages that each sequence touches (the last one again where it touches fewer)
        first, last = start // P, (lengths - 1) // P
        R = -(-c["new_max"] // P) + 1
        run = torch.minimum(first[:, None] + torch.arange(R, device=k.device), last[:, None])
        phys = table.gather(1, run)
        most = torch.zeros(len(new) * R, c["heads_kv"], dtype=W, device=k.device)
        at = (seq * R + slot // P - first[seq])[:, None].expand(-1, c["heads_kv"])
        most.scatter_reduce_(0, at, rows[x].abs().amax(-1), "amax")
        most = most.view(len(new), R, -1).gather(1, (run - first[:, None])[..., None].expand(-1, -1, c["heads_kv"]))
        kept = (start[:, None] - run * P).clamp(0, P)
        need = _scale_for(most).float()
        before = scale[phys]
        after = torch.where((kept > 0)[..., None], torch.maximum(before, need), need)
        codes = cache.view(torch.uint8)[phys].view(torch.float8_e4m3fn)
        again = _e4m3(codes.float() * (before / after)[..., None, None]).view(torch.uint8)
        held = (torch.arange(P, device=k.device) < kept[..., None])[:, :, None, :, None]
        cache.view(torch.uint8)[phys] = torch.where(held, again, codes.view(torch.uint8))
        scale[phys] = after
        fresh = rows[x] / after[seq, slot // P - first[seq]][..., None]
        cache.view(torch.uint8)[page, :, off] = _e4m3(fresh).view(torch.uint8)
    return _turn(q, *turn).to(q.dtype)


def _softmax(x):
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp_()
    l = p.sum(-1, keepdim=True)
    return p.div_(l), (m + l.log()).squeeze(-1)


def _kept(qpos, kpos, window, sinks):
    keep = kpos <= qpos
    return keep & ((qpos - kpos < window) | (kpos < sinks)) if window else keep


def _paged_plain(c, q, kc, vc, ks, vs, table, lengths):
    S, n, hk, d, P = table.shape[0], c["q_len"], c["heads_kv"], c["head_dim"], c["page"]
    grp, L = c["heads_q"] // hk, table.shape[1] * P

    def rows(cache, scale):
        x = (cache.view(torch.uint8)[table.long()].view(cache.dtype) if scale is not None else cache[table.long()]).to(W)
        x = x if scale is None else x * scale[table.long()][..., None, None].to(W)
        return x.transpose(1, 2).reshape(S, hk, L, d)

    x = q.to(W).view(S, n, hk, grp, d).permute(0, 2, 1, 3, 4).reshape(S, hk, n * grp, d)
    x = torch.matmul(x, rows(kc, ks).transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(S, hk, n, grp, L)
    qpos = (lengths.long() - n)[:, None, None] + torch.arange(n, device=q.device)[:, None]
    keep = _kept(qpos, torch.arange(L, device=q.device), c["window"], c["sinks"])
    p, lse = _softmax(x.masked_fill_(~keep[:, None, :, None], -math.inf))
    o = torch.matmul(p.view(S, hk, n * grp, L), rows(vc, vs)).view(S, hk, n, grp, d)
    return o.permute(0, 2, 1, 3, 4).reshape(S * n, hk * grp, d), lse.permute(1, 3, 0, 2).reshape(hk * grp, S * n)


def _window_plain(c, q, k, v, cu, most, g):
    d, total = c["head_dim"], q.shape[0]
    lens = (cu[1:] - cu[:-1]).long()
    at = torch.arange(most, device=q.device)
    rows = (cu[:-1].long()[:, None] + at).clamp(max=total - 1)
    inside = at < lens[:, None]
    seq, pos = _token_places(cu, total)

    def padded(x):
        return (x[rows].to(W) * inside[..., None, None]).transpose(1, 2)

    def packed(x, dtype):
        return x[seq, :, pos].to(dtype)

    Q, K, V = padded(q), padded(k), padded(v)
    x = torch.matmul(Q, K.transpose(-1, -2)).mul_(1 / math.sqrt(d))
    keep = _kept(at[:, None], at, c["window"], c["sinks"])
    p, lse = _softmax(x.masked_fill_(~keep, -math.inf))
    o = torch.matmul(p, V)
    out = {"out": packed(o, q.dtype), "lse": packed(lse, W).t().contiguous()}
    if g is None:
        return out
    G = padded(g)
    out["dv"] = packed(torch.matmul(p.transpose(-1, -2), G), q.dtype)
    dx = torch.matmul(G, V.transpose(-1, -2)).sub_((G * o).sum(-1, keepdim=True)).mul_(p).mul_(1 / math.sqrt(d))
    out["dq"] = packed(torch.matmul(dx, K), q.dtype)
    out["dk"] = packed(torch.matmul(dx.transpose(-1, -2), Q), q.dtype)
    return out


def run(state):
    s = state
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "rotary":
        turn = lambda x, back: _turn(x, s["positions"], s["frequencies"], s["mscale"], c["interleaved"], back).to(x.dtype)  # noqa: E731
        out = {}
        if c["direction"] != "backward":
            out["q"], out["k"] = turn(s["q"], False), turn(s["k"], False)
        if c["direction"] != "forward":
            out["dq"], out["dk"] = turn(s["gq"], True), turn(s["gk"], True)
        return out
    if c["op"] == "append":
        caches = {x: (s[x + "_cache"], s[x + "_scale"]) for x in ("k", "v")}
        return _append_out(s, _append_plain(s, s["q"], s["k"], s["v"], caches))
    if c["op"] == "paged":
        o, lse = _paged_plain(c, s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lengths"])
        return {"out": o.to(s["q"].dtype), "lse": lse}
    return _window_plain(c, s["q"], s["k"], s["v"], s["cu"], s["max_new"], s.get("g"))


def _append_out(s, q):
    return {"q": q, **{x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale") if s[x] is not None}}


def _run_own(s):
    import masked_attention_tri_gb300 as ta
    c = s["case"]
    if c["op"] == "rotary":
        out = {}
        if c["direction"] != "backward":
            out["q"], out["k"] = ta.rotary_embedding(s["q"], s["k"], s["positions"], s["rotary"])
        if c["direction"] != "forward":
            out["dq"], out["dk"] = ta.rotary_embedding_backward(s["gq"], s["gk"], s["positions"], s["rotary"])
        return out
    if c["op"] == "append":
        q = ta.kv_cache_append(s["handle"], s["k"], s["v"], s["table"], s["lengths"], s["cu"], s["max_new"],
                               rotary=s["rotary"], q=s["q"])
        return _append_out(s, q)
    if c["op"] == "paged":
        o, lse = ta.paged_attention(s["q"], s["handle"], s["table"], s["lengths"],
                                    s["cu"] if c["q_len"] > 1 else None, s["max_new"], window=c["window"] or None,
                                    sinks=c["sinks"], return_aux=True)
        return {"out": o, "lse": lse}
    mask = {"mask_mod": "sink_window", "window": c["window"], "sinks": c["sinks"]}
    cu, n = s["cu"], s["max_new"]
    o, lse, _ = ta.varlen_attention(s["q"], s["k"], s["v"], cu, cu, n, n, return_aux=True, **mask)
    out = {"out": o, "lse": lse}
    if c["direction"] == "both":
        out["dq"], out["dk"], out["dv"], _ = ta.varlen_attention_backward(s["q"], s["k"], s["v"], cu, cu, n, n, o, lse,
                                                                          s["g"], **mask)
    return out


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_turn(x, positions, c):
    """Each pair as a complex number, times mscale * exp(i * position * frequency)."""
    f, mscale = _frequencies(c)
    angle = positions.double()[:, None, None] * f.to(x.device)
    w = torch.polar(torch.full_like(angle, mscale), angle)
    x, half = x.double().clone(), f.numel()
    first = slice(0, 2 * half, 2) if c["interleaved"] else slice(0, half)
    second = slice(1, 2 * half, 2) if c["interleaved"] else slice(half, 2 * half)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * w
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_append(c, s):
    """Token by token of a sequence, page by page, from the definition of the 8-bit cache."""
    new, held = _lengths(c)
    P, W = c["page"], torch.float64
    out = {"k_cache": s["k_cache"].to(W), "v_cache": s["v_cache"].to(W)}
    eight = c["cache"] == "e4m3"
    if eight:
        out["k_scale"], out["v_scale"] = s["k_scale"].to(W), s["v_scale"].to(W)
    slots = torch.cat([torch.arange(h - n, h) for n, h in zip(new, held)]).to(s["q"].device)
    rows = {"k": _exact_turn(s["k"], slots, c), "v": s["v"].to(W)}
    out["q"] = _exact_turn(s["q"], slots, c)
    table, t = s["table"].tolist(), 0
    for i, (n, h) in enumerate(zip(new, held)):
        a = h - n
        while a < h:
            b = min(h, (a // P + 1) * P)
            page, off = table[i][a // P], a % P
            for x in ("k", "v"):
                fresh = rows[x][t:t + b - a].transpose(0, 1)
                cache = out[x + "_cache"][page]
                if eight:
                    scale = out[x + "_scale"]
                    most = fresh.abs().amax((-1, -2)).clamp(min=2.0 ** -80)
                    need = torch.exp2(torch.ceil(torch.log2(most / 448)).clamp(-56, 56))
                    if off:
                        need = torch.maximum(need, scale[page])
                        cache[:, :off] = _nearest_code(cache[:, :off] * (scale[page] / need)[:, None, None])
                    scale[page] = need
                    fresh = _nearest_code(fresh / need[:, None, None])
                cache[:, off:off + b - a] = fresh
            t += b - a
            a = b
    return out


_codes = None


def _nearest_code(x):
    """The nearest of the 253 finite values that e4m3 holds (ties to the even code), found in their list."""
    global _codes
    if _codes is None or _codes.device != x.device:
        _codes = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    y = x.abs().clamp(max=448.0).contiguous()
    i = torch.searchsorted(_codes, y).clamp(1, 126)
    lo, hi = _codes[i - 1], _codes[i]
    up = (y - lo > hi - y) | ((y - lo == hi - y) & (i % 2 == 0))
    return torch.where(up, hi, lo) * x.sign()


def _exact_paged(c, s):
    W, grp, P = torch.float64, c["heads_q"] // c["heads_kv"], c["page"]
    new, held = _lengths(c)
    outs, lses, t = [], [], 0
    for i, (n, h) in enumerate(zip(new, held)):
        pages = s["table"][i, :-(-h // P)].long()

        def rows(x):
            y = s[x + "_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).to(W) if c["cache"] == "e4m3" else s[x + "_cache"][pages].to(W)
            y = y * s[x + "_scale"][pages].to(W)[..., None, None] if c["cache"] == "e4m3" else y
            return y.transpose(0, 1).flatten(1, 2)[:, :h].repeat_interleave(grp, 0)

        x = torch.einsum("nhd,hld->hnl", s["q"][t:t + n].to(W), rows("k")) / math.sqrt(c["head_dim"])
        j, p = torch.arange(h, device=x.device), torch.arange(h - n, h, device=x.device)[:, None]
        hide = j > p
        if c["window"]:
            hide = hide | ((j <= p - c["window"]) & (j >= c["sinks"]))
        x[:, hide] = -math.inf
        lses.append(torch.logsumexp(x, -1))
        outs.append(torch.einsum("hnl,hld->nhd", (x - lses[-1][..., None]).exp(), rows("v")))
        t += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses, 1)}


def _exact_window(c, s):
    W, both = torch.float64, c["direction"] == "both"
    new, _ = _lengths(c)
    scale, out = 1 / math.sqrt(c["head_dim"]), {}
    for x in ("out", "dq", "dk", "dv") if both else ("out",):
        out[x] = torch.empty(s["q"].shape, dtype=W, device=s["q"].device)
    out["lse"] = torch.empty(c["heads"], sum(new), dtype=W, device=s["q"].device)
    t = 0
    for n in new:
        j = torch.arange(n, device=s["q"].device)
        hide = (j > j[:, None]) | ((j <= j[:, None] - c["window"]) & (j >= c["sinks"]))
        for h in range(c["heads"]):
            q, k, v = (s[x][t:t + n, h].to(W) for x in ("q", "k", "v"))
            x = (q @ k.t()) * scale
            x[hide] = -math.inf
            lse = torch.logsumexp(x, -1)
            p = (x - lse[:, None]).exp()
            out["lse"][h, t:t + n], out["out"][t:t + n, h] = lse, p @ v
            if both:
                g = s["g"][t:t + n, h].to(W)
                dp = g @ v.t()
                dx = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
                out["dq"][t:t + n, h], out["dk"][t:t + n, h], out["dv"][t:t + n, h] = dx @ k, dx.t() @ q, p.t() @ g
        t += n
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rotary":
        out = {}
        if c["direction"] != "backward":
            out["q"], out["k"] = _exact_turn(s["q"], s["positions"], c), _exact_turn(s["k"], s["positions"], c)
        if c["direction"] != "forward":  # the transposed turn: by the opposite angle
            out["dq"], out["dk"] = _exact_turn(s["gq"], -s["positions"], c), _exact_turn(s["gk"], -s["positions"], c)
        return out
    return {"append": _exact_append, "paged": _exact_paged, "window": _exact_window}[c["op"]](c, s)
