"""What is measured of prompts, the 4-bit cache and positions with several axes.

Each case is one call, or one training step, of an operator next to this
library's packed and paged attention: rotary positions with several axes (forward
and backward), rows written into a paged cache of 4-bit codes and read back from it,
attention over that cache, and the attention of whole prompts or chunks of them with
grouped heads (forward and backward).  `run` computes them in their plain form from
elementary torch operations, or, with `own`, through this library's entry points;
`exact` gives the same results from the definitions in 64 bits.

The 4-bit cache: 16 neighbouring elements of a row share a scale.  Element x of head h is
n * s * f_h with a whole number n from -7 to 7 (held as n + 8, two a byte, the even element
in the low half), s an e4m3 number for the 16, f_h a power of two for the head:
s = e4m3(max |x| / (7 f_h)), from 2^-9 to 448, and n = x / (f_h s) rounded to the nearest.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_GROUP = 16


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------

def _rotary(name, **over):
    c = {"name": name, "op": "rotary", "direction": "forward", "tokens": 64, "heads_q": 32, "heads_kv": 8,
         "head_dim": 128, "rotary_dim": 128, "axes": 3, "layout": "blocks", "frequencies": "shared",
         "interleaved": False, "last_position": 4095, "dtype": "bf16"}
    return {**c, **over}


def _append(name, **over):
    c = {"name": name, "op": "append", "seqs": 64, "new_min": 1, "new_max": 1, "held_min": 0, "held_max": 2047,
         "heads_kv": 8, "head_dim": 128, "page": 64, "dtype": "bf16"}
    return {**c, **over}


def _read(name, **over):
    c = {"name": name, "op": "read", "seqs": 1, "new_min": 1000, "new_max": 1000, "held_min": 0, "held_max": 0,
         "heads_kv": 8, "head_dim": 128, "page": 64, "dtype": "bf16"}
    return {**c, **over}


def _paged(name, **over):
    c = {"name": name, "op": "paged", "seqs": 1, "q_len": 1, "kv_min": 1, "kv_max": 1000, "heads_q": 32,
         "heads_kv": 8, "head_dim": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"}
    return {**c, **over}


def _prompt(name, **over):
    c = {"name": name, "op": "prompt", "direction": "forward", "seqs": 8, "len_min": 256, "len_max": 2048,
         "before_min": 0, "before_max": 0, "heads_q": 32, "heads_kv": 8, "head_dim": 128, "dtype": "bf16"}
    return {**c, **over}


def listed():
    return [
        # one decoding step of 64 sequences that hold images: three positions a token, latency counts
        _rotary("rotary_axes_decode"),
        # a training batch of 16k packed tokens of text, images and video, both directions
        _rotary("rotary_axes_train", direction="both", tokens=16384, layout="interleaved"),
        # one new token of each of 64 sequences
        _append("append_decode_4bit"),
        # the prompts of eight requests (256 to 2048 tokens)
        _append("append_prompt_4bit", seqs=8, new_min=256, new_max=2048, held_max=0),
        # one short context that a chunk of its prompt attends to
        _read("read_chunk_4bit"),
        # the contexts of 16 requests (2k to 16k tokens) before their prompts' next chunks
        _read("read_context_4bit", seqs=16, new_min=2048, new_max=16384),
        # one user alone, a context of a thousand tokens: latency counts
        _paged("paged_single_4bit", kv_min=1000),
        # a full serving batch with contexts from 1k to 16k tokens
        _paged("paged_batch_4bit", seqs=64, kv_min=1024, kv_max=16384),
        # a few short questions of odd lengths: latency counts
        _prompt("prompt_short", seqs=4, len_min=17, len_max=300),
        # a batch of whole prompts
        _prompt("prompt_batch", seqs=8, len_min=512, len_max=4096),
        # the next 2048 tokens of two long prompts, of which 8k and 30k tokens were processed before
        _prompt("prompt_chunk", seqs=2, len_min=2048, len_max=2048, before_min=8192, before_max=30000),
        # a training step on packed sequences, forward and backward
        _prompt("prompt_train", direction="both", seqs=3, len_min=777, len_max=8192, heads_q=16, heads_kv=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "read", "paged", "prompt", "prompt"])
    hk, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 256])
    t = rng.choice(["bf16", "bf16", "f16"])
    if op == "rotary":
        t = rng.choice([t, t, "f32"])
        c = _rotary("", direction=rng.choice(["forward", "backward", "both"]), heads_kv=hk,
                    heads_q=hk * rng.choice([1, 2, 4, 8]), head_dim=d, rotary_dim=rng.choice([d, d // 2, 32]),
                    axes=rng.choice([2, 3, 3, 4]), layout=rng.choice(["blocks", "interleaved"]),
                    frequencies=rng.choice(["shared", "own"]), interleaved=rng.random() < 0.5,
                    last_position=_log(rng, 100, 1 << 20), dtype=t)
        row = (c["heads_q"] + hk) * d * _BYTES[t]
        c["tokens"] = min(_log(rng, 1, 16384), (16384 * 40 * 128 * 2) // row)
    elif op in ("append", "read"):
        make = _append if op == "append" else _read
        many = op == "read" or rng.random() < 0.5
        c = make("", seqs=_log(rng, 1, 16 if many else 256), new_max=_log(rng, 16, 8192) if many else
                 rng.choice([1, 1, 1, 4, 7]), heads_kv=hk, head_dim=d, page=rng.choice([16, 32, 64, 128]),
                 held_max=_log(rng, 16, 1000), dtype=rng.choice([t, t, "f32"]))
        c["new_max"] = max(1, min(c["new_max"], (16 * 9000 * 8 * 128) // (c["seqs"] * hk * d)))
        c["new_min"] = max(1, c["new_max"] // rng.choice([1, 2, 8]))
    elif op == "paged":
        c = _paged("", seqs=_log(rng, 1, 128), q_len=rng.choice([1, 1, 1, 2, 5, 8]), heads_kv=hk,
                   heads_q=hk * rng.choice([1, 2, 4, 8]), head_dim=d, page=rng.choice([16, 32, 64, 128]), dtype=t)
        most = (64 * 8700 * 8 * 128) // (c["seqs"] * hk * d)
        if rng.random() < 0.1:
            c["dtype"], most = "f32", most // 8
        c["kv_max"] = max(c["q_len"], min(_log(rng, 16, 65536), most))
        c["kv_min"] = max(1, c["kv_max"] // rng.choice([1, 4, 100]))
        if rng.random() < 0.3:
            c["window"], c["sinks"] = _log(rng, 16, 8192), rng.choice([0, 1, 4, 64])
    else:
        c = _prompt("", direction=rng.choice(["forward", "both"]), seqs=rng.choice([1, 2, 3, 8, 20]),
                    len_max=_log(rng, 16, 8192), heads_kv=hk, heads_q=hk * rng.choice([1, 2, 3, 4, 8]),
                    head_dim=rng.choice([64, 96, 128, 128]), dtype=t)
        if c["direction"] == "forward" and rng.random() < 0.4:
            c["before_max"] = _log(rng, 16, 16384)
            c["before_min"] = c["before_max"] // rng.choice([1, 2, 100])
        # no more products than the largest listed step has, of padded sequences
        both = 2 if c["direction"] == "both" else 1
        while both * c["seqs"] * c["heads_q"] * c["len_max"] * (c["len_max"] + c["before_max"]) > 3e9:
            c["len_max"] = -(-c["len_max"] // 2)
            c["before_max"], c["before_min"] = c["before_max"] // 2, c["before_min"] // 2
        if rng.random() < 0.1:
            c["dtype"], c["len_max"], c["before_max"] = "f32", min(c["len_max"], 1000), min(c["before_max"], 1000)
            c["before_min"] = min(c["before_min"], c["before_max"])
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
    """(rows of the call, slots or keys held after it) of every sequence: plain lists that follow from the case."""
    if c["op"] in ("append", "read"):
        new = _spread(c["new_min"], c["new_max"], c["seqs"])
        return new, [n + h for n, h in zip(new, reversed(_spread(c["held_min"], c["held_max"], c["seqs"])))]
    if c["op"] == "paged":
        held = [max(n, c["q_len"]) for n in _spread(c["kv_min"], c["kv_max"], c["seqs"])]
        return [c["q_len"]] * c["seqs"], held
    new = _spread(c["len_min"], c["len_max"], c["seqs"])
    return new, [n + b for n, b in zip(new, _spread(c["before_min"], c["before_max"], c["seqs"]))]


def _visible(c, position):
    """Slots that a token at `position` sees."""
    n = position + 1
    return n if not c["window"] or n <= c["window"] else c["window"] + min(c["sinks"], n - c["window"])


def work(case):
    c, e = case, _BYTES[case["dtype"]]
    if c["op"] == "rotary":
        n = c["tokens"] * (c["heads_q"] + c["heads_kv"])
        times = 2 if c["direction"] == "both" else 1
        return {"bytes": times * (2 * n * c["head_dim"] * e + 4 * c["axes"] * c["tokens"]),
                "flops": times * 3 * n * c["rotary_dim"]}
    new, held = _lengths(c)
    if c["op"] in ("append", "read"):
        values = 2 * sum(new) * c["heads_kv"] * c["head_dim"]
        return {"bytes": values * e + values // 2 + values // _GROUP, "flops": 3 * values if c["op"] == "append" else values}
    if c["op"] == "paged":
        hq, d = c["heads_q"], c["head_dim"]
        pairs = sum(_visible(c, h - n + i) for n, h in zip(new, held) for i in range(n))
        keys = sum(min(h, _visible(c, h - 1) + (n - 1 if c["window"] else 0)) for n, h in zip(new, held))
        values = 2 * keys * c["heads_kv"] * d
        return {"bytes": values // 2 + values // _GROUP + sum(new) * hq * (2 * d * e + 4), "flops": 4 * pairs * hq * d}
    pairs = sum(n * (h - n) + n * (n + 1) // 2 for n, h in zip(new, held)) * c["heads_q"]
    q_row, k_row = sum(new) * c["heads_q"] * c["head_dim"] * e, sum(held) * c["heads_kv"] * c["head_dim"] * e
    lse = 4 * sum(new) * c["heads_q"]
    if c["direction"] == "forward":
        return {"bytes": 2 * q_row + 2 * k_row + lse, "flops": 4 * pairs * c["head_dim"]}
    return {"bytes": 6 * q_row + 6 * k_row + 2 * lse, "flops": 14 * pairs * c["head_dim"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

_BASE = 10000.0


def _sections(c):
    """Pairs of each axis: the first axis (time) has what is left, as the others have equal parts."""
    pairs, a = c["rotary_dim"] // 2, c["axes"]
    rest = pairs // (a + 1) + (1 if pairs % (a + 1) > 1 else 0)
    return [pairs - rest * (a - 1)] + [rest] * (a - 1)


def _pair_axes(c):
    """The axis of each pair: blocks one after the other, or dealt in turn to the axes that still want some."""
    want, out = _sections(c), []
    if c["layout"] == "blocks":
        return [a for a, n in enumerate(want) for _ in range(n)]
    while len(out) < c["rotary_dim"] // 2:
        for a in range(c["axes"]):
            if want[a] > 0:
                want[a] -= 1
                out.append(a)
    return out


def _frequencies(c):
    """Radians a position of each pair in 64 bits: over all pairs, or for each axis over its own."""
    axes, want, seen, f = _pair_axes(c), _sections(c), [0] * c["axes"], []
    for i, a in enumerate(axes):
        x = seen[a] / want[a] if c["frequencies"] == "own" else 2 * i / c["rotary_dim"]
        seen[a] += 1
        f.append(_BASE ** -x)
    return torch.tensor(f, dtype=torch.float64)


def _plan(c, dev):
    import masked_attention_tri_gb300 as ta
    return ta.Rotary(c["rotary_dim"], _BASE, interleaved=c["interleaved"], sections=_sections(c),
                     section_layout=c["layout"], section_frequencies=c["frequencies"], device=dev)


def prepare(case, seed):
    c, dev = case, torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(int(seed))
    t = _TYPES[c["dtype"]]

    def randn(*shape, by=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32 if t == torch.float32 else torch.bfloat16) * by).to(t)

    s = {"case": c}
    if c["op"] == "rotary":
        n, d = c["tokens"], c["head_dim"]
        s["positions"] = torch.randint(0, c["last_position"] + 1, (c["axes"], n), generator=g, device=dev, dtype=torch.int32)
        for x in (("q", "k") if c["direction"] != "backward" else ()) + (("gq", "gk") if c["direction"] != "forward" else ()):
            s[x] = randn(n, c["heads_q"] if x[-1] == "q" else c["heads_kv"], d)
        s["frequencies"] = _frequencies(c).to(dev)
        s["axis"] = torch.tensor(_pair_axes(c), device=dev)
        if own:
            s["rotary"] = _plan(c, dev)
        return s
    new, held = _lengths(c)
    total, S, hk, d = sum(new), len(new), c["heads_kv"], c["head_dim"]
    s["cu"] = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device=dev)
    s["max_new"], s["total"] = max(new), total
    if c["op"] == "prompt":
        s["cu_k"] = s["cu"] if held == new else torch.tensor(np.cumsum([0] + held), dtype=torch.int32, device=dev)
        s["max_held"] = max(held)
        s["q"] = randn(total, c["heads_q"], d, by=1.5)
        s["k"], s["v"] = randn(sum(held), hk, d), randn(sum(held), hk, d)
        if c["direction"] == "both":
            s["g"] = randn(total, c["heads_q"], d)
        return s
    P = c["page"]
    pages = [-(-h // P) for h in held]
    most = max(pages)
    order = torch.randperm(sum(pages), generator=g, device=dev).to(torch.int32)
    first = torch.tensor(np.cumsum([0] + pages[:-1]), device=dev)
    s["table"] = order[(first[:, None] + torch.arange(most, device=dev)).clamp(max=sum(pages) - 1)].contiguous()
    s["lengths"] = torch.tensor(held, dtype=torch.int32, device=dev)
    shape = (sum(pages), hk, P)
    for x in ("k", "v"):
        # codes from -7 to 7 of values with a bell's shape, scales from 1/16 to 1
        codes = [(torch.randn(*shape, d // 2, generator=g, device=dev, dtype=torch.bfloat16) * 3).round_().clamp_(-7, 7).add_(8).to(torch.uint8) for _ in range(2)]
        s[x + "_codes"] = codes[0] | (codes[1] << 4)
        s[x + "_scale"] = torch.exp2(torch.rand(*shape, d // _GROUP, generator=g, device=dev) * -4).to(torch.float8_e4m3fn)
        s[x + "_factor"] = torch.exp2(torch.randint(-2, 3, (hk,), generator=g, device=dev).float())
    if c["op"] == "append":
        # a few channels of the keys are far larger than the others, as in trained models
        s["k"] = (randn(total, hk, d) * (1 + 15 * (torch.arange(d, device=dev) % 61 == 7))).to(t)
        s["v"] = randn(total, hk, d)
    if c["op"] == "paged":
        s["q"] = randn(total, c["heads_q"], d)
    if own:  # the handle that a serving program keeps for the cache's memory
        import masked_attention_tri_gb300 as ta
        s["handle"] = ta.PagedKVCache4(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["k_factor"], s["v_factor"])
    return s


# ---------------------------------------------------------------------------
# The plain forms, in 32 bits (W)
# ---------------------------------------------------------------------------

W = torch.float32


def _turn(x, positions, s, interleaved, back):
    """x (tokens, heads, d) with the leading pairs turned by their axes' positions; the angles in 64 bits."""
    half = s["frequencies"].numel()
    angle = positions.double()[s["axis"]].t() * s["frequencies"]
    cos, sin = angle.cos().to(W)[:, None], angle.sin().to(W)[:, None]
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


def _slots(s):
    """(page, slot in the page) of every row of the call: the last slots that its sequence holds."""
    seq, pos = _token_places(s["cu"], s["total"])
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    slot = (s["lengths"].long() - new)[seq] + pos
    return s["table"].long()[seq, slot // s["case"]["page"]], slot % s["case"]["page"]


def _codes_of(x, factor):
    """(bytes, scales) of rows x (total, heads, d)."""
    y = (x.to(W) / factor[:, None]).unflatten(-1, (-1, _GROUP))
    # (by a tensor: a division by a number may be done as a product, which leaves the border between two scales)
    scale = (y.abs().amax(-1) / torch.full((1,), 7.0, device=x.device)).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    n = (torch.round(y / scale.to(W)[..., None]).clamp_(-7, 7) + 8).to(torch.uint8).flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), scale


def _values_of(codes, scale, factor):
    """The values that bytes (..., heads, d / 2) with scales (..., heads, d / 16) stand for."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(W) - 8
    return (n.unflatten(-1, (-1, _GROUP)) * scale.to(W)[..., None]).flatten(-2) * factor[:, None]


def _softmax(x):
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp_()
    l = p.sum(-1, keepdim=True)
    return p.div_(l), (m + l.log()).squeeze(-1)


def _paged_plain(s):
    c, table, lengths = s["case"], s["table"].long(), s["lengths"].long()
    S, n, hk, d, P = table.shape[0], c["q_len"], c["heads_kv"], c["head_dim"], c["page"]
    grp, L = c["heads_q"] // hk, table.shape[1] * P

    def rows(x):  # (S, pages, heads, page, d) -> (S, heads, L, d)
        y = _values_of(s[x + "_codes"][table].transpose(2, 3), s[x + "_scale"].view(torch.uint8)[table].view(torch.float8_e4m3fn).transpose(2, 3), s[x + "_factor"])
        return y.permute(0, 3, 1, 2, 4).reshape(S, hk, L, d)

    x = s["q"].to(W).view(S, n, hk, grp, d).permute(0, 2, 1, 3, 4).reshape(S, hk, n * grp, d)
    x = torch.matmul(x, rows("k").transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(S, hk, n, grp, L)
    qpos, kpos = (lengths - n)[:, None, None] + torch.arange(n, device=x.device)[:, None], torch.arange(L, device=x.device)
    keep = kpos <= qpos
    if c["window"]:
        keep = keep & ((qpos - kpos < c["window"]) | (kpos < c["sinks"]))
    p, lse = _softmax(x.masked_fill_(~keep[:, None, :, None], -math.inf))
    o = torch.matmul(p.view(S, hk, n * grp, L), rows("v")).view(S, hk, n, grp, d)
    o = o.permute(0, 2, 1, 3, 4).reshape(S * n, hk * grp, d)
    return {"out": o.to(s["q"].dtype), "lse": lse.permute(1, 3, 0, 2).reshape(hk * grp, S * n)}


def _prompt_plain(s):
    c, t, W_ = s["case"], s["q"].dtype, W
    hk, grp, d, S = c["heads_kv"], c["heads_q"] // c["heads_kv"], c["head_dim"], c["seqs"]
    n, m = s["max_new"], s["max_held"]
    lq, lk = (s["cu"][1:] - s["cu"][:-1]).long(), (s["cu_k"][1:] - s["cu_k"][:-1]).long()

    def padded(x, cu, length, most):  # (S, heads, most, d), zeros past the end
        at = torch.arange(most, device=x.device)
        rows = (cu[:-1].long()[:, None] + at).clamp(max=x.shape[0] - 1)
        return (x[rows].to(W_) * (at < length[:, None])[..., None, None]).transpose(1, 2)

    def queries(x):  # (S, hk, grp * n, d): the grouped heads share the keys of one product
        return padded(x, s["cu"], lq, n).reshape(S, hk, grp * n, d)

    def packed(x, cu, total, heads, most):
        seq, pos = _token_places(cu, total)
        return x.reshape(S, heads, most, -1)[seq, :, pos].to(t)

    Q, K, V = queries(s["q"]), padded(s["k"], s["cu_k"], lk, m), padded(s["v"], s["cu_k"], lk, m)
    x = torch.matmul(Q, K.transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(S, hk, grp, n, m)
    # the last token sees every key, the one before it one less
    late = (lk - lq)[:, None, None] + torch.arange(n, device=x.device)[:, None]
    hide = torch.arange(m, device=x.device) > late
    p, lse = _softmax(x.masked_fill_(hide[:, None, None], -math.inf))
    p = p.view(S, hk, grp * n, m)
    o = torch.matmul(p, V)
    seq, pos = _token_places(s["cu"], s["total"])
    out = {"out": packed(o, s["cu"], s["total"], c["heads_q"], n),
           "lse": lse.reshape(S, c["heads_q"], n)[seq, :, pos].t().contiguous()}
    if c["direction"] == "forward":
        return out
    G = queries(s["g"])
    out["dv"] = packed(torch.matmul(p.transpose(-1, -2), G), s["cu_k"], s["k"].shape[0], hk, m)
    dx = torch.matmul(G, V.transpose(-1, -2)).sub_((G * o).sum(-1, keepdim=True)).mul_(p).mul_(1 / math.sqrt(d))
    out["dq"] = packed(torch.matmul(dx, K), s["cu"], s["total"], c["heads_q"], n)
    out["dk"] = packed(torch.matmul(dx.transpose(-1, -2), Q), s["cu_k"], s["k"].shape[0], hk, m)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "rotary":
        turn = lambda x, back: _turn(s[x], s["positions"], s, c["interleaved"], back).to(s[x].dtype)  # noqa: E731
        out = {}
        if c["direction"] != "backward":
            out["q"], out["k"] = turn("q", False), turn("k", False)
        if c["direction"] != "forward":
            out["dq"], out["dk"] = turn("gq", True), turn("gk", True)
        return out
    if c["op"] == "append":
        page, off = _slots(s)
        for x in ("k", "v"):
            codes, scale = _codes_of(s[x], s[x + "_factor"])
            s[x + "_codes"][page, :, off] = codes
            s[x + "_scale"].view(torch.uint8)[page, :, off] = scale.view(torch.uint8)
        return _cache_out(s)
    if c["op"] == "read":
        page, off = _slots(s)
        return {x: _values_of(s[x + "_codes"][page, :, off], s[x + "_scale"].view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn),
                              s[x + "_factor"]).to(_TYPES[c["dtype"]]) for x in ("k", "v")}
    return _paged_plain(s) if c["op"] == "paged" else _prompt_plain(s)


def _cache_out(s):
    """The cache's own memory: bytes of two codes, equal or not, and the scales as the numbers that they are."""
    return {x: s[x] for x in ("k_codes", "v_codes", "k_scale", "v_scale")}


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
        ta.kv_cache_append(s["handle"], s["k"], s["v"], s["table"], s["lengths"], s["cu"], s["max_new"])
        return _cache_out(s)
    if c["op"] == "read":
        k, v = ta.kv_cache_read(s["handle"], s["table"], s["lengths"], s["cu"], s["max_new"], s["total"], dtype=_TYPES[c["dtype"]])
        return {"k": k, "v": v}
    if c["op"] == "paged":
        o, lse = ta.paged_attention(s["q"], s["handle"], s["table"], s["lengths"],
                                    s["cu"] if c["q_len"] > 1 else None, s["max_new"], window=c["window"] or None,
                                    sinks=c["sinks"], return_aux=True)
        return {"out": o, "lse": lse}
    args = s["q"], s["k"], s["v"], s["cu"], s["cu_k"], s["max_new"], s["max_held"]
    o, lse = ta.prompt_attention(*args, return_aux=True)
    out = {"out": o, "lse": lse}
    if c["direction"] == "both":
        out["dq"], out["dk"], out["dv"] = ta.prompt_attention_backward(*args, o, lse, s["g"])
    return out


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_turn(x, positions, c):
    """Each pair as a complex number, times exp(i * position * frequency) of its own axis."""
    f, axis, half = _frequencies(c).tolist(), _pair_axes(c), c["rotary_dim"] // 2
    x = x.double().clone()
    for i in range(half):
        angle = positions[axis[i]].double()[:, None] * f[i]
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        z = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * torch.polar(torch.ones_like(angle), angle)
        x[..., a], x[..., b] = z.real, z.imag
    return x


def _exact_rows(s, x, pages, length):
    """(heads, length, d) values of one sequence's pages in 64 bits."""
    codes, scale = s[x + "_codes"][pages].long(), s[x + "_scale"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
    v = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    v[..., 0::2], v[..., 1::2] = codes % 16 - 8, codes // 16 - 8
    v = v * scale.repeat_interleave(_GROUP, -1) * s[x + "_factor"].double()[:, None, None]
    return v.transpose(0, 1).flatten(1, 2)[:, :length]


def _exact_append(c, s):
    """The scales after the call: the nearest of the e4m3 numbers, found in their list (the codes are whole numbers)."""
    new, held = _lengths(c)
    numbers = torch.arange(1, 127, dtype=torch.uint8, device=s["k"].device).view(torch.float8_e4m3fn).double()
    out, table, t = {"k_codes": None, "v_codes": None}, s["table"].tolist(), 0
    want = {}
    for x in ("k", "v"):
        out[x + "_scale"] = s[x + "_scale"].double()
        a = s[x].double().unflatten(-1, (-1, _GROUP)).abs().amax(-1) / (7 * s[x + "_factor"].double()[:, None])
        a = a.clamp(2.0 ** -9, 448.0).contiguous()
        i = torch.searchsorted(numbers, a).clamp(1, 125)
        lo, hi = numbers[i - 1], numbers[i]
        up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 1))
        want[x] = torch.where(up, hi, lo)
    for i, (n, h) in enumerate(zip(new, held)):
        a = h - n
        while a < h:
            b = min(h, (a // c["page"] + 1) * c["page"])
            for x in ("k", "v"):
                out[x + "_scale"][table[i][a // c["page"]], :, a % c["page"]:a % c["page"] + b - a] = want[x][t:t + b - a].transpose(0, 1)
            t, a = t + b - a, b
    return out


def _exact_read(c, s):
    new, held = _lengths(c)
    out = {"k": [], "v": []}
    for i, (n, h) in enumerate(zip(new, held)):
        for x in out:
            out[x].append(_exact_rows(s, x, s["table"][i, :-(-h // c["page"])].long(), h)[:, h - n:].transpose(0, 1))
    return {x: torch.cat(y) for x, y in out.items()}


def _exact_paged(c, s):
    grp = c["heads_q"] // c["heads_kv"]
    new, held = _lengths(c)
    outs, lses, t = [], [], 0
    for i, (n, h) in enumerate(zip(new, held)):
        pages = s["table"][i, :-(-h // c["page"])].long()
        K, V = (_exact_rows(s, x, pages, h).repeat_interleave(grp, 0) for x in ("k", "v"))
        x = torch.einsum("nhd,hld->hnl", s["q"][t:t + n].double(), K) / math.sqrt(c["head_dim"])
        j, p = torch.arange(h, device=x.device), torch.arange(h - n, h, device=x.device)[:, None]
        hide = j > p
        if c["window"]:
            hide = hide | ((j <= p - c["window"]) & (j >= c["sinks"]))
        x[:, hide] = -math.inf
        lses.append(torch.logsumexp(x, -1))
        outs.append(torch.einsum("hnl,hld->nhd", (x - lses[-1][..., None]).exp(), V))
        t += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses, 1)}


def _exact_prompt(c, s):
    D, both = torch.float64, c["direction"] == "both"
    new, held = _lengths(c)
    scale, grp, dev, out = 1 / math.sqrt(c["head_dim"]), c["heads_q"] // c["heads_kv"], s["q"].device, {}
    out["out"] = torch.empty(s["q"].shape, dtype=D, device=dev)
    out["lse"] = torch.empty(c["heads_q"], sum(new), dtype=D, device=dev)
    if both:
        out["dq"] = torch.empty(s["q"].shape, dtype=D, device=dev)
        out["dk"], out["dv"] = (torch.zeros(s["k"].shape, dtype=D, device=dev) for _ in range(2))
    t = u = 0
    for n, h in zip(new, held):
        hide = torch.arange(h, device=dev) > torch.arange(h - n, h, device=dev)[:, None]
        for a in range(c["heads_q"]):
            b = a // grp
            q, k, v = s["q"][t:t + n, a].to(D), s["k"][u:u + h, b].to(D), s["v"][u:u + h, b].to(D)
            x = (q @ k.t()) * scale
            x[hide] = -math.inf
            lse = torch.logsumexp(x, -1)
            p = (x - lse[:, None]).exp()
            out["lse"][a, t:t + n], out["out"][t:t + n, a] = lse, p @ v
            if both:
                g = s["g"][t:t + n, a].to(D)
                dp = g @ v.t()
                dx = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
                out["dq"][t:t + n, a] = dx @ k
                out["dk"][u:u + h, b] += dx.t() @ q
                out["dv"][u:u + h, b] += p.t() @ g
        t, u = t + n, u + h
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
    return {"append": _exact_append, "read": _exact_read, "paged": _exact_paged, "prompt": _exact_prompt}[c["op"]](c, s)
