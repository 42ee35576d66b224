"""The serving step's operators around the paged KV cache: their cases, plain forms and calls.

Four operators, in the order in which a step uses them:

* ``plan``     block table, slot map and row offsets of a step from the requests' lengths;
* ``rope``     rotary positions (one or several axes) on q and k, k and v written to the cache;
* ``prefill``  attention of a chunk of new tokens over the paged cache (causal, windowed, sinks);
* ``sinks``    single-token decode with a sliding window and first tokens that stay visible.

``run`` computes the plain form (elementary torch operations in 32 bits, angles in 64) where
``own`` is false, and calls the library's operators where it is true.
"""
import math
import random

import torch

own = False

D = 128  # head dimension
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # A decode step of 64 sequences: one new token each (the latency of the step's first call).
        {"name": "plan_decode_b64", "op": "plan", "batch": 64, "block": 16, "max_blocks": 512, "chunk": 1, "mix": False, "shape": 1},
        # A large mixed step: single tokens, prompt chunks, trimmed drafts, ended and idle requests.
        {"name": "plan_mixed_b1024", "op": "plan", "batch": 1024, "block": 16, "max_blocks": 512, "chunk": 512, "mix": True, "shape": 2},
        # The same decode step's rotation and cache write in one layer.
        {"name": "rope_decode_t64", "op": "rope", "tokens": 64, "h_q": 64, "h_kv": 8, "dtype": "bf16", "axes": 1, "rot": 128, "pairs": "half", "block": 16, "fp8": False, "pad": 0, "shape": 3},
        # A chunk of 8192 prompt tokens with time, height and width positions (images and video).
        {"name": "rope_video_t8192", "op": "rope", "tokens": 8192, "h_q": 64, "h_kv": 8, "dtype": "bf16", "axes": 3, "rot": 128, "pairs": "half", "block": 16, "fp8": False, "pad": 0, "shape": 4},
        # An odd chunk into an 8-bit cache, half of each head rotated, neighbouring pairs, padded rows.
        {"name": "rope_fp8_t1111", "op": "rope", "tokens": 1111, "h_q": 32, "h_kv": 8, "dtype": "fp16", "axes": 1, "rot": 64, "pairs": "next", "block": 64, "fp8": True, "pad": 17, "shape": 5},
        # A few drafted tokens per sequence checked over long caches.
        {"name": "prefill_verify_b32", "op": "prefill", "batch": 32, "q_lo": 1, "q_hi": 8, "ctx_lo": 4096, "ctx_hi": 8184, "h_q": 64, "h_kv": 8, "dtype": "bf16", "block": 16, "window": 0, "sinks": 0, "fp8": False, "shape": 6},
        # One whole prompt of 8192 tokens.
        {"name": "prefill_prompt_8192", "op": "prefill", "batch": 1, "q_lo": 8192, "q_hi": 8192, "ctx_lo": 0, "ctx_hi": 0, "h_q": 64, "h_kv": 8, "dtype": "bf16", "block": 64, "window": 0, "sinks": 0, "fp8": False, "shape": 7},
        # Ragged prompt chunks, some with a long cached prefix.
        {"name": "prefill_chunks_b8", "op": "prefill", "batch": 8, "q_lo": 33, "q_hi": 1024, "ctx_lo": 0, "ctx_hi": 7000, "h_q": 32, "h_kv": 8, "dtype": "fp16", "block": 16, "window": 0, "sinks": 0, "fp8": False, "shape": 8},
        # Chunks of a windowed model with one KV head per query head and four kept first tokens.
        {"name": "prefill_window_mha_b4", "op": "prefill", "batch": 4, "q_lo": 1500, "q_hi": 2048, "ctx_lo": 0, "ctx_hi": 4096, "h_q": 32, "h_kv": 32, "dtype": "bf16", "block": 16, "window": 1024, "sinks": 4, "fp8": False, "shape": 9},
        # Chunks over an 8-bit cache.
        {"name": "prefill_fp8_b4", "op": "prefill", "batch": 4, "q_lo": 512, "q_hi": 1024, "ctx_lo": 1000, "ctx_hi": 7000, "h_q": 64, "h_kv": 8, "dtype": "bf16", "block": 32, "window": 0, "sinks": 0, "fp8": True, "shape": 10},
        # A decode step of a windowed model at full batch.
        {"name": "sinks_decode_b64", "op": "sinks", "batch": 64, "ctx_lo": 4200, "ctx_hi": 8192, "h_q": 64, "h_kv": 8, "dtype": "bf16", "block": 16, "window": 4096, "sinks": 4, "fp8": False, "shape": 11},
        # A small step far into long sequences over an 8-bit cache (latency and splitting).
        {"name": "sinks_fp8_b8", "op": "sinks", "batch": 8, "ctx_lo": 1, "ctx_hi": 32768, "h_q": 32, "h_kv": 8, "dtype": "fp16", "block": 64, "window": 2048, "sinks": 64, "fp8": True, "shape": 12},
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "prefill", "prefill", "sinks"])
    shape = rng.randrange(1 << 20)
    if op == "plan":
        return {"op": op, "batch": _spread(rng, 1, 1024), "block": rng.choice([8, 16, 32, 64, 128, 256]), "max_blocks": rng.randint(65, 512), "chunk": _spread(rng, 1, 512),
                "mix": rng.random() < 0.7, "shape": shape}
    h_q, h_kv = rng.choice([(64, 8), (32, 8), (32, 32), (32, 1), (28, 4), (12, 4), (8, 8), (64, 1), (5, 1)])
    dtype = rng.choice(["bf16", "fp16"])
    block = rng.choice([8, 16, 32, 64, 128, 256])
    fp8 = rng.random() < 0.35
    if op == "rope":
        return {"op": op, "tokens": _spread(rng, 1, 8192), "h_q": h_q, "h_kv": h_kv, "dtype": dtype, "axes": rng.choice([1, 1, 2, 3]), "rot": rng.choice([128, 128, 64, 96, 32]),
                "pairs": rng.choice(["half", "next"]), "block": block, "fp8": fp8, "pad": rng.choice([0, 0, rng.randint(1, 40)]), "shape": shape}
    if op == "sinks":
        batch = _spread(rng, 1, 64)
        hi = _spread(rng, 64, 32768)
        window = _spread(rng, 1, 8192)
        while batch * min(hi, window) * h_kv > 64 * 4096 * 8:
            batch = (batch + 1) // 2
            window = max(1, window * 3 // 4)
        return {"op": op, "batch": batch, "ctx_lo": rng.randint(1, hi), "ctx_hi": hi, "h_q": h_q, "h_kv": h_kv, "dtype": dtype, "block": block, "window": window,
                "sinks": rng.choice([1, 4, 4, rng.randint(2, 200)]), "fp8": fp8, "shape": shape}
    batch, q_hi, ctx = _spread(rng, 1, 32), _spread(rng, 1, 4096), _spread(rng, 1, 16384)
    while batch * q_hi * (q_hi + ctx) * h_q > 8192 * 4096 * 64 or batch * (q_hi + ctx) * h_kv > 16 * 8192 * 8:
        batch, q_hi, ctx = (batch + 1) // 2, max(1, q_hi * 3 // 4), max(1, ctx * 3 // 4)
    window = rng.choice([0, 0, _spread(rng, 1, 4096)])
    return {"op": op, "batch": batch, "q_lo": rng.randint(1, q_hi), "q_hi": q_hi, "ctx_lo": rng.randint(0, ctx), "ctx_hi": ctx, "h_q": h_q, "h_kv": h_kv, "dtype": dtype, "block": block,
            "window": window, "sinks": rng.choice([0, 4, rng.randint(1, 300)]) if window else 0, "fp8": fp8, "shape": shape}


def _lens(case):
    """The lengths of a case: they belong to its shape, so that its work is known."""
    r = random.Random(case["shape"])
    if case["op"] == "plan":
        most = case["max_blocks"] * case["block"]
        cached, new = [], []
        for _ in range(case["batch"]):
            n = case["chunk"]
            kind = r.random() if case["mix"] else 1.0
            c = r.randint(0, max(0, min(most, 8192) - n))
            if kind < 0.25:
                n = r.randint(1, n)      # a prompt's chunk
            elif kind < 0.35:
                n = -min(c, r.randint(1, 64))  # drafted tokens taken back
            elif kind < 0.40:
                n = -c                   # an ended request
            elif kind < 0.45:
                n = 0
            elif case["mix"]:
                n = 1
            cached.append(c)
            new.append(n)
        return cached, new
    if case["op"] == "sinks":
        return [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])], None
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    return [n + r.randint(case["ctx_lo"], case["ctx_hi"]) for n in q], q


def _blocks(n, block):
    return -(-n // block)


# ------------------------------------------------------------------ work


def work(case):
    op = case["op"]
    if op == "plan":
        cached, new = _lens(case)
        grown = sum(max(0, n) for n in new)
        moved = sum(abs(_blocks(c + n, case["block"]) - _blocks(c, case["block"])) for c, n in zip(cached, new))
        # lengths in, lengths and row offsets out; each moved block id read and written; slot and position of each token
        return {"bytes": 16 * case["batch"] + 8 * moved + 8 * grown, "flops": 0}
    h_q, h_kv = case["h_q"], case["h_kv"]
    size = 1 if case["fp8"] else 2
    if op == "rope":
        t = case["tokens"]
        return {"bytes": t * D * (2 * (h_q + 2 * h_kv) + 2 * h_q + 2 * h_kv * size) + 4 * t * (case["axes"] + 1), "flops": 3 * t * (h_q + h_kv) * case["rot"]}
    lens, q = _lens(case)
    pairs = rows = tokens = 0
    for n, m in zip(lens, q or [1] * len(lens)):
        if not case["window"]:
            pairs += m * (n - m) + m * (m + 1) // 2
            rows += n
        else:
            w, s = case["window"], case["sinks"]
            for p in range(n - m, n):
                first = max(0, p + 1 - w)
                pairs += p + 1 - first + min(s, first)
            first = max(0, n - m + 1 - w)
            rows += n - first + min(s, first)
        tokens += m
    return {"bytes": 2 * 2 * tokens * h_q * D + 2 * rows * h_kv * D * size, "flops": 4 * D * h_q * pairs}


# ------------------------------------------------------------------ inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cache(g, blocks, case):
    """K and V caches and, over 8 bits, the scales of the KV heads."""
    shape = (blocks, case["block"], case["h_kv"], D)
    if not case["fp8"]:
        return [torch.randn(shape, generator=g, device="cuda").to(TYPES[case["dtype"]]) for _ in range(2)], None
    codes = [(torch.randn(shape, generator=g, device="cuda") * 112).clamp_(-448, 448).to(torch.float8_e4m3fn) for _ in range(2)]
    return codes, [(torch.rand(case["h_kv"], generator=g, device="cuda") + 0.5) / 112 for _ in range(2)]


def _table(g, lens, block):
    """A permuted block table of these lengths (-1 past a sequence's last block) and the number of blocks."""
    need = torch.tensor([_blocks(n, block) for n in lens], device="cuda")
    total, most = sum(_blocks(n, block) for n in lens), max(1, max(_blocks(n, block) for n in lens))
    ids = torch.randperm(total + 3, generator=g, device="cuda").int()
    at = (need.cumsum(0) - need)[:, None] + torch.arange(most, device="cuda")
    used = torch.arange(most, device="cuda") < need[:, None]
    return torch.where(used, ids[at.clamp(max=total + 2)], -1).contiguous(), total + 3


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case}
    if op == "plan":
        cached, new = _lens(case)
        block, batch, most = case["block"], case["batch"], case["max_blocks"]
        held = [_blocks(c, block) for c in cached]
        need = sum(max(0, _blocks(c + n, block) - h) for c, n, h in zip(cached, new, held))
        total = sum(held) + need + 64
        ids = torch.randperm(total, generator=g, device="cuda").int()
        h = torch.tensor(held, device="cuda")
        at = (h.cumsum(0) - h)[:, None] + torch.arange(most, device="cuda")
        s["table"] = torch.where(torch.arange(most, device="cuda") < h[:, None], ids[at.clamp(max=total - 1)], -1).contiguous()
        s["free"] = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        s["free"][: total - sum(held)] = ids[sum(held):]
        s["free_count"] = torch.tensor([total - sum(held)], dtype=torch.int32, device="cuda")
        s["cached"] = torch.tensor(cached, dtype=torch.int32, device="cuda")
        s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        s["tokens"] = sum(max(0, n) for n in new) + 5  # a step's list has a few rows to spare
        return s
    dtype = TYPES[case["dtype"]]
    h_q, h_kv = case["h_q"], case["h_kv"]
    if op == "rope":
        t, rot, axes = case["tokens"], case["rot"], case["axes"]
        qkv = torch.randn((t, (h_q + 2 * h_kv) * D), generator=g, device="cuda").to(dtype)  # one projection's output
        s["q"] = qkv[:, : h_q * D].view(t, h_q, D)
        s["k"] = qkv[:, h_q * D: (h_q + h_kv) * D].view(t, h_kv, D)
        s["v"] = qkv[:, (h_q + h_kv) * D:].view(t, h_kv, D)
        s["positions"] = torch.randint(0, 120000, (axes, t), generator=g, device="cuda", dtype=torch.int32)
        blocks = _blocks(t, case["block"]) + 2
        s["caches"], s["scales"] = _cache(g, blocks, case)
        s["slots"] = torch.randperm(blocks * case["block"], generator=g, device="cuda")[:t].int()
        if case["pad"]:
            s["slots"][-min(t - 1, case["pad"]) or t:] = -1  # rows behind the last sequence
        pairs = rot // 2
        s["inv_freq"] = [1e6 ** (-i / pairs) for i in range(pairs)]
        cut = [pairs - (pairs // axes) * (axes - 1)] + [pairs // axes] * (axes - 1)
        s["sections"] = cut
        s["axis"] = torch.tensor([a for a, n in enumerate(cut) for _ in range(n)], device="cuda")
        s["inv"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda")
        if own:
            import gqa_mqa_mla_gb300 as da
            s["rope"] = da.rope_table(s["inv_freq"], sections=cut, interleaved=case["pairs"] == "next", device="cuda")
        return s
    lens, q = _lens(case)
    s["table"], blocks = _table(g, lens, case["block"])
    s["caches"], s["scales"] = _cache(g, blocks, case)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["max_len"] = max(lens)
    if op == "prefill":
        s["max_q"] = max(q)
        s["start"] = torch.tensor([sum(q[:i]) for i in range(len(q) + 1)], dtype=torch.int32, device="cuda")
    s["q"] = torch.randn((sum(q) if q else len(lens), h_q, D), generator=g, device="cuda").to(dtype)
    return s


# ------------------------------------------------------------------ plain forms


def _plain_plan(s):
    block, tokens = s["case"]["block"], s["tokens"]
    cached, new, table, free = s["cached"].long(), s["new"].long(), s["table"].clone(), s["free"].clone()
    held, now = -(-cached // block), -(-(cached + new) // block)
    lost, need, grown = (held - now).clamp(min=0), (now - held).clamp(min=0), new.clamp(min=0)
    count = s["free_count"].long()
    col = torch.arange(table.shape[1], device=table.device)
    gone = (col >= now[:, None]) & (col < held[:, None])
    rank = (lost.cumsum(0) - lost)[:, None] + col - now[:, None]
    free[(count + rank)[gone]] = table[gone]
    top = count + lost.sum()
    fresh = (col >= held[:, None]) & (col < now[:, None])
    rank = (need.cumsum(0) - need)[:, None] + col - held[:, None]
    table[fresh] = free[(top - 1 - rank)[fresh]]
    start = torch.cat([grown.new_zeros(1), grown.cumsum(0)])
    i = torch.arange(tokens, device=table.device)
    b = torch.searchsorted(start[1:], i, right=True).clamp(max=len(cached) - 1)
    live = i < start[-1]
    pos = torch.where(live, cached[b] + i - start[b], 0)
    slot = table[b, pos // block].long() * block + pos % block
    return {"table": table, "free": free, "free_count": (top - need.sum()).int(), "lens": (cached + new).int(), "start": start.int(),
            "slots": torch.where(live, slot, -1).int(), "positions": torch.where(live, pos, -1).int()}


def _plain_rope(s):
    case = s["case"]
    angle = s["positions"].double()[s["axis"]].T * s["inv"]  # [tokens, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    n = case["rot"] // 2

    def turn(x):
        x = x.float()
        a, b = (x[..., :n], x[..., n:2 * n]) if case["pairs"] == "half" else (x[..., 0:2 * n:2], x[..., 1:2 * n:2])
        u, w = a * cos - b * sin, a * sin + b * cos
        r = torch.cat([u, w], -1) if case["pairs"] == "half" else torch.stack([u, w], -1).flatten(-2)
        return torch.cat([r, x[..., 2 * n:]], -1)

    live = s["slots"] >= 0
    at = s["slots"][live].long()
    rows = [turn(s["k"])[live], s["v"].float()[live]]
    if case["fp8"]:
        rows = [(r / c[:, None]).clamp(-448, 448) for r, c in zip(rows, s["scales"])]
    for c, r in zip(s["caches"], rows):
        if case["fp8"]:
            c.view(torch.uint8).view(-1, *r.shape[1:])[at] = r.to(c.dtype).view(torch.uint8)
        else:
            c.view(-1, *r.shape[1:])[at] = r.to(c.dtype)
    return {"q": turn(s["q"]).to(s["q"].dtype), "k": s["caches"][0], "v": s["caches"][1]}


def _rows(s, k, at):
    """The cache's rows of logical positions `at` [batch, n], in 32 bits: [batch, heads, n, D]."""
    case = s["case"]
    block = s["table"].gather(1, at // case["block"]).clamp(min=0).long()
    c = s["caches"][k]
    c = (c.view(torch.uint8) if case["fp8"] else c).view(-1, *c.shape[2:])[block * case["block"] + at % case["block"]]
    c = c.view(torch.float8_e4m3fn).float() * s["scales"][k][:, None] if case["fp8"] else c.float()
    return c.transpose(1, 2)


def _attend(q, k, v, seen):
    """Softmax attention in 32 bits: q [b, h, g, n, D], k and v [b, h, m, D], seen [b, n, m]."""
    b, h, g, n, _ = q.shape
    x = (q.reshape(b, h, g * n, D) @ k.transpose(-1, -2)).view(b, h, g, n, -1)
    x.mul_(D ** -0.5).masked_fill_(~seen[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    return (x.view(b, h, g * n, -1) @ v).view(b, h, g, n, D) / total.clamp(min=1e-30)


def _plain_prefill(s):
    case = s["case"]
    dev, h_kv = s["q"].device, case["h_kv"]
    g, n, m = case["h_q"] // h_kv, s["max_q"], s["max_len"]
    start, lens = s["start"].long(), s["lens"].long()
    count = start[1:] - start[:-1]
    i = torch.arange(n, device=dev)
    q = s["q"][(start[:-1, None] + i).clamp(max=len(s["q"]) - 1)].float().view(-1, n, h_kv, g, D).permute(0, 2, 3, 1, 4)
    t = torch.arange(m, device=dev)
    at = torch.minimum(t, (lens - 1)[:, None])
    pos = ((lens - count)[:, None] + i)[:, :, None]
    seen = t <= pos
    if case["window"]:
        seen &= (t > pos - case["window"]) | (t < case["sinks"])
    seen &= t < lens[:, None, None]
    o = _attend(q, _rows(s, 0, at), _rows(s, 1, at), seen).permute(0, 3, 1, 2, 4).reshape(-1, n, case["h_q"], D)
    r = torch.arange(len(s["q"]), device=dev)
    b = torch.searchsorted(start[1:], r, right=True)
    return o[b, r - start[b]].to(s["q"].dtype)


def _plain_sinks(s):
    case = s["case"]
    dev, h_kv = s["q"].device, case["h_kv"]
    lens = s["lens"].long()[:, None]
    first = (lens - case["window"]).clamp(min=0)
    t = torch.arange(case["sinks"] + min(case["window"], s["max_len"]), device=dev)
    sink = t < case["sinks"]
    at = torch.where(sink, t, first + t - case["sinks"])
    seen = torch.where(sink, t < first, at < lens)
    at = torch.minimum(at, lens - 1)
    q = s["q"].float().view(len(lens), h_kv, -1, 1, D)
    return _attend(q, _rows(s, 0, at), _rows(s, 1, at), seen[:, None]).reshape(s["q"].shape).to(s["q"].dtype)


# ------------------------------------------------------------------ one pass


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"plan": _plain_plan, "rope": _plain_rope, "prefill": _plain_prefill, "sinks": _plain_sinks}[op](state)
    import gqa_mqa_mla_gb300 as da
    s = state
    if op == "plan":
        p = da.paged_plan(s["cached"], s["new"], s["table"], s["free"], s["free_count"], block_size=case["block"], max_tokens=s["tokens"])
        return {"table": s["table"], "free": s["free"], "free_count": p.free_count, "lens": p.seq_lens, "start": p.q_start, "slots": p.slots, "positions": p.positions}
    if op == "rope":
        if case["fp8"]:
            q = da.gqa_rope_append_fp8kv(s["q"], s["k"], s["v"], *s["scales"], s["positions"], s["rope"], s["slots"], *s["caches"])
        else:
            q = da.gqa_rope_append(s["q"], s["k"], s["v"], s["positions"], s["rope"], s["slots"], *s["caches"])
        return {"q": q, "k": s["caches"][0], "v": s["caches"][1]}
    if op == "prefill":
        more = {"scale": D ** -0.5, "max_q_len": s["max_q"], "max_seq_len": s["max_len"], "window": case["window"] or None, "sinks": case["sinks"]}
        if case["fp8"]:
            return da.gqa_prefill_fp8kv(s["q"], *s["caches"], *s["scales"], s["table"], s["start"], s["lens"], **more)
        return da.gqa_prefill(s["q"], *s["caches"], s["table"], s["start"], s["lens"], **more)
    more = {"scale": D ** -0.5, "max_seq_len": s["max_len"], "window": case["window"], "sinks": case["sinks"]}
    if case["fp8"]:
        return da.gqa_decode_fp8kv_sinks(s["q"], *s["caches"], *s["scales"], s["table"], s["lens"], **more)
    return da.gqa_decode_sinks(s["q"], *s["caches"], s["table"], s["lens"], **more)


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "plan":
        return None  # whole numbers: nothing to round
    if op == "rope":
        turns = (s["positions"].double().index_select(0, s["axis"]).T * s["inv"]).unsqueeze(1)
        z = torch.polar(torch.ones_like(turns), turns)
        n = case["rot"] // 2
        out = []
        for x in (s["q"].double(), s["k"].double()):
            head, rest = x[..., : 2 * n], x[..., 2 * n:]
            c = torch.view_as_complex((head.unflatten(-1, (2, n)).transpose(-1, -2) if case["pairs"] == "half" else head.unflatten(-1, (n, 2))).contiguous())
            y = torch.view_as_real(c * z)
            y = (y.transpose(-1, -2) if case["pairs"] == "half" else y).flatten(-2)
            out.append(torch.cat([y, rest], -1))
        out.append(s["v"].double())
        live = s["slots"] >= 0
        kept = s["slots"][live].long()
        for j in (0, 1):
            c = s["caches"][j].double()
            new = out[1 + j][live]
            if case["fp8"]:  # the value that a code stands in for, before its rounding
                new = (new / s["scales"][j].double()[None, :, None]).clamp(-448, 448)
            c.view(-1, case["h_kv"], D).index_copy_(0, kept, new)
            out[1 + j] = c
        return {"q": out[0], "k": out[1], "v": out[2]}
    lens, count = _lens(case)
    count = count or [1] * len(lens)
    g = case["h_q"] // case["h_kv"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, m) in enumerate(zip(lens, count)):
        blocks = s["table"][b, : _blocks(n, case["block"])].long()
        kv = []
        for j in (0, 1):
            c = s["caches"][j]
            x = (c.view(torch.uint8)[blocks].view(torch.float8_e4m3fn) if case["fp8"] else c[blocks]).double().flatten(0, 1)[:n]
            kv.append(x * s["scales"][j].double()[:, None] if case["fp8"] else x)
        t = torch.arange(n, device="cuda")
        p = torch.arange(n - m, n, device="cuda")[:, None]
        hidden = t > p
        if case["window"]:
            hidden |= (p - t >= case["window"]) & (t >= case["sinks"])
        for h in range(case["h_q"]):
            x = s["q"][row: row + m, h].double() @ kv[0][:, h // g].T / math.sqrt(D)
            o[row: row + m, h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ kv[1][:, h // g]
        row += m
    return o
