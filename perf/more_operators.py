"""Long caches: reading less of them and keeping less of them. Cases, plain forms and calls.

Five operators over the paged KV cache, in the order in which a serving step uses them:

* ``bounds``   per-block smallest and largest key of each dimension, kept up as tokens arrive;
* ``select``   the blocks whose keys can score highest for a query, per sequence and KV head;
* ``blocks``   single-token decode attention over the selected blocks only;
* ``weights``  single-token decode attention that adds up each cached token's attention weight;
* ``evict``    the heaviest and the latest tokens stay, the cache is closed up behind them.

``run`` computes the plain form (elementary torch operations in 32 bits, block scores in 64)
where ``own`` is false, and calls the library's operators where it is true.
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
        # After a decode step of 64 sequences: the block that got the new token (latency).
        {"name": "bounds_decode_b64", "op": "bounds", "batch": 64, "ctx_lo": 4096, "ctx_hi": 8192, "new": 1, "h_q": 64, "h_kv": 8, "dtype": "bf16", "block": 16, "fp8": False, "shape": 1},
        # After whole prompts of four ragged documents.
        {"name": "bounds_prompt_b4", "op": "bounds", "batch": 4, "ctx_lo": 20000, "ctx_hi": 65536, "new": 0, "h_q": 64, "h_kv": 8, "dtype": "bf16", "block": 64, "fp8": False, "shape": 2},
        # One very long sequence: 8192 blocks to choose from (latency and splitting).
        {"name": "select_b1_131072", "op": "select", "batch": 1, "ctx_lo": 131001, "ctx_hi": 131072, "h_q": 64, "h_kv": 8, "dtype": "bf16", "block": 16, "count": 128, "first": 1, "last": 2, "fp8": False, "shape": 3},
        # A full decode step over long caches.
        {"name": "select_b32", "op": "select", "batch": 32, "ctx_lo": 16384, "ctx_hi": 32768, "h_q": 64, "h_kv": 8, "dtype": "bf16", "block": 16, "count": 128, "first": 1, "last": 2, "fp8": False, "shape": 4},
        # The same step's attention: 128 of up to 2048 blocks.
        {"name": "blocks_b32", "op": "blocks", "batch": 32, "ctx_lo": 16384, "ctx_hi": 32768, "h_q": 64, "h_kv": 8, "dtype": "bf16", "block": 16, "count": 128, "fp8": False, "shape": 5},
        # A small step of a model with one KV head over an 8-bit cache, odd counts (latency).
        {"name": "blocks_mqa_fp8_b5", "op": "blocks", "batch": 5, "ctx_lo": 1, "ctx_hi": 32768, "h_q": 32, "h_kv": 1, "dtype": "bf16", "block": 64, "count": 33, "fp8": True, "shape": 6},
        # A full decode step that keeps account of each token's weight.
        {"name": "weights_b64", "op": "weights", "batch": 64, "ctx_lo": 4096, "ctx_hi": 8192, "h_q": 64, "h_kv": 8, "dtype": "bf16", "block": 16, "fp8": False, "shape": 7},
        # A ragged one over an 8-bit cache, one KV head per query head.
        {"name": "weights_mha_fp8_b7", "op": "weights", "batch": 7, "ctx_lo": 1, "ctx_hi": 5000, "h_q": 32, "h_kv": 32, "dtype": "fp16", "block": 32, "fp8": True, "shape": 8},
        # One long sequence with a single KV head.
        {"name": "weights_mqa_b1", "op": "weights", "batch": 1, "ctx_lo": 32768, "ctx_hi": 32768, "h_q": 32, "h_kv": 1, "dtype": "bf16", "block": 16, "fp8": False, "shape": 9},
        # Sequences that have grown past 5120 tokens go back to 4096.
        {"name": "evict_b64", "op": "evict", "batch": 64, "ctx_lo": 2000, "ctx_hi": 6000, "h_q": 64, "h_kv": 8, "dtype": "bf16", "block": 16, "keep": 4096, "recent": 1024, "limit": 5120, "fp8": False, "shape": 10},
        # A long prompt over an 8-bit cache cut to an odd length right after it was read.
        {"name": "evict_prompt_fp8_b2", "op": "evict", "batch": 2, "ctx_lo": 30000, "ctx_hi": 32768, "h_q": 32, "h_kv": 8, "dtype": "bf16", "block": 64, "keep": 2111, "recent": 64, "limit": 2111, "fp8": True, "shape": 11},
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["bounds", "select", "select", "blocks", "blocks", "weights", "weights", "evict"])
    h_q, h_kv = rng.choice([(64, 8), (32, 8), (32, 32), (32, 1), (28, 4), (12, 4), (8, 8), (64, 1), (5, 1)])
    case = {"op": op, "batch": _spread(rng, 1, 64), "h_q": h_q, "h_kv": h_kv, "dtype": rng.choice(["bf16", "fp16"]), "block": rng.choice([8, 16, 32, 64, 128, 256]),
            "fp8": rng.random() < 0.35, "shape": rng.randrange(1 << 20)}
    hi = _spread(rng, 64 * case["block"] if op == "select" else 1, 131072 if op in ("select", "bounds") else 32768)
    most = {"bounds": 200000, "select": 700000, "blocks": 300000, "weights": 350000, "evict": 200000}[op] * 8
    while case["batch"] * hi * h_kv > most:
        case["batch"], hi = (case["batch"] + 1) // 2, max(1, hi * 3 // 4)
    case["ctx_lo"], case["ctx_hi"] = rng.randint(1, hi), hi
    if op == "bounds":
        case["new"] = rng.choice([0, 1, 1, _spread(rng, 1, 512)])
    elif op in ("select", "blocks"):
        case["count"] = _spread(rng, 3, 4096 // case["block"])
        if op == "select":
            # some sequence has a choice to make
            case["ctx_lo"] = rng.randint(1 if case["batch"] >= 8 else hi // 2, hi)
            case["count"] = max(5, min(case["count"], max(_lens(case)) // case["block"] // 2))
            case["first"] = rng.choice([0, 1, 1])
            case["last"] = rng.choice([0, 1, 1, 2])
    elif op == "evict":
        case["keep"] = _spread(rng, 1, min(hi, 6000))
        case["recent"] = rng.randint(0, case["keep"])
        case["limit"] = case["keep"] + rng.choice([0, 0, rng.randint(1, 1000)])
    return case


def _lens(case):
    """The lengths of a case: they belong to its shape, so that its work is known."""
    r = random.Random(case["shape"])
    return [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]


def _first(case, lens):
    """Tokens that each sequence had when its bounds were last brought up to date."""
    return [max(0, n - case["new"]) if case["new"] else 0 for n in lens]


def _blocks(n, block):
    return -(-n // block)


# ------------------------------------------------------------------ work


def work(case):
    op, block, h_q, h_kv = case["op"], case["block"], case["h_q"], case["h_kv"]
    size = 1 if case["fp8"] else 2
    lens = _lens(case)
    if op == "bounds":
        rows = blocks = 0
        for n, f in zip(lens, _first(case, lens)):
            at = min(f, n - 1) // block
            rows += n - at * block
            blocks += _blocks(n, block) - at
        return {"bytes": (rows + 2 * blocks) * h_kv * D * size, "flops": 2 * rows * h_kv * D}
    if op == "select":
        # sequences with no more blocks than are taken need no scores
        scored = sum(_blocks(n, block) - case["first"] - case["last"] for n in lens if _blocks(n, block) > case["count"])
        return {"bytes": scored * h_kv * 2 * D * size + case["batch"] * (2 * h_q * D + 4 * h_kv * case["count"]), "flops": 2 * scored * h_q * D}
    if op == "blocks":
        rows = entries = 0
        for n in lens:
            k = min(case["count"], _blocks(n, block))
            entries += k
            rows += k * block - (_blocks(n, block) * block - n)
        return {"bytes": rows * h_kv * 2 * D * size + 4 * entries * h_kv + case["batch"] * 4 * h_q * D, "flops": 4 * rows * h_q * D}
    if op == "weights":
        rows = sum(lens)
        return {"bytes": rows * h_kv * (2 * D * size + 8) + case["batch"] * 4 * h_q * D, "flops": 4 * rows * h_q * D}
    cut = [n for n in lens if n > case["limit"]]
    return {"bytes": h_kv * (4 * sum(cut) + len(cut) * case["keep"] * (4 * D * size + 4)) + case["batch"] * (4 * h_kv * case["keep"] + 8), "flops": 0}


# ------------------------------------------------------------------ inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cache(g, blocks, case, both=True):
    """K (and V) caches and, over 8 bits, the scales of the KV heads.

    Keys have an offset of their own in each dimension, as models' keys do."""
    shape = (blocks, case["block"], case["h_kv"], D)
    made = []
    for k in range(2 if both else 1):
        x = torch.randn(shape, generator=g, device="cuda")
        if k == 0:
            x += 0.7 * torch.randn(shape[2:], generator=g, device="cuda")
        made.append((x * 100).clamp_(-448, 448).to(torch.float8_e4m3fn) if case["fp8"] else x.to(TYPES[case["dtype"]]))
        del x
    scales = [(torch.rand(case["h_kv"], generator=g, device="cuda") + 0.5) / 100 for _ in made] if case["fp8"] else None
    return made, scales


def _table(g, lens, block):
    """A permuted block table of these lengths (-1 past a sequence's last block) and the number of blocks."""
    need = torch.tensor([_blocks(n, block) for n in lens], device="cuda")
    total, most = sum(_blocks(n, block) for n in lens), max(1, max(_blocks(n, block) for n in lens))
    ids = torch.randperm(total + 3, generator=g, device="cuda").int()
    at = (need.cumsum(0) - need)[:, None] + torch.arange(most, device="cuda")
    used = torch.arange(most, device="cuda") < need[:, None]
    return torch.where(used, ids[at.clamp(max=total + 2)], -1).contiguous(), total + 3


def _some_blocks(g, lens, case):
    """For each sequence and KV head: the first block, the last and random others, ascending, -1 behind them."""
    have = torch.tensor([_blocks(n, case["block"]) for n in lens], device="cuda")[:, None, None]
    most = max(case["count"], int(have.max()))
    t = torch.arange(most, device="cuda")
    x = torch.rand((len(lens), case["h_kv"], most), generator=g, device="cuda")
    x = torch.where((t == 0) | (t == have - 1), 2.0, x).masked_fill(t >= have, -1.0)
    best = x.topk(case["count"])
    ids = torch.where(best.values >= 0, best.indices, most).sort(-1).values
    return torch.where(ids < most, ids, -1).int()


def prepare(case, seed):
    g = _generator(seed)
    op, h_q, h_kv, block = case["op"], case["h_q"], case["h_kv"], case["block"]
    lens = _lens(case)
    s = {"case": case, "max_len": max(lens), "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    s["table"], blocks = _table(g, lens, block)
    if op in ("select", "blocks", "weights"):
        s["q"] = torch.randn((len(lens), h_q, D), generator=g, device="cuda").to(TYPES[case["dtype"]])
    if op == "bounds":
        (s["k"],), _ = _cache(g, blocks, case, both=False)
        s["first"] = torch.tensor(_first(case, lens), dtype=torch.int32, device="cuda")
        s["bounds"] = torch.zeros((blocks, 2, h_kv, D), device="cuda").to(s["k"].dtype)
        return s
    if op == "select":
        # the spread of a block's keys about the dimension's own offset and the block's
        mid = 0.7 * torch.randn((h_kv, D), generator=g, device="cuda") + 0.5 * torch.randn((blocks, h_kv, D), generator=g, device="cuda")
        half = 0.8 + torch.rand((blocks, 2, h_kv, D), generator=g, device="cuda")
        x = torch.stack([mid - half[:, 0], mid + half[:, 1]], 1)
        s["bounds"] = (x * 100).clamp_(-448, 448).to(torch.float8_e4m3fn) if case["fp8"] else x.to(TYPES[case["dtype"]])
        return s
    s["caches"], s["scales"] = _cache(g, blocks, case)
    if op == "blocks":
        s["selected"] = _some_blocks(g, lens, case)
    else:
        # accumulated weights are heavy-tailed: few tokens hold most of them
        s["weights"] = torch.randn((blocks, h_kv, block), generator=g, device="cuda").mul_(2).exp_().mul_(h_q / h_kv / 50)
    return s


# ------------------------------------------------------------------ plain forms


def _bytes(c):
    return c.view(torch.uint8) if c.dtype == torch.float8_e4m3fn else c


def _plain_bounds(s):
    block, lens, first = s["case"]["block"], s["lens"].long(), s["first"].long()
    t = torch.arange(s["table"].shape[1], device=lens.device)
    touched = (t >= (torch.minimum(first, lens - 1) // block)[:, None]) & (t < -(-lens // block)[:, None])
    seq, at = touched.nonzero(as_tuple=True)
    ids = s["table"][seq, at].long()
    k = _bytes(s["k"])[ids].view(s["k"].dtype).float()
    gone = (at[:, None] * block + torch.arange(block, device=lens.device) >= lens[seq, None])[:, :, None, None]
    low, high = k.masked_fill(gone, math.inf).amin(1), k.masked_fill_(gone, -math.inf).amax(1)
    _bytes(s["bounds"])[ids] = _bytes(torch.stack([low, high], 1).to(s["k"].dtype))
    return s["bounds"]


def _plain_select(s):
    case = s["case"]
    have = -(-s["lens"].long() // case["block"])[:, None]
    b = s["bounds"]
    x = _bytes(b)[s["table"].clamp(min=0).long()].view(b.dtype).double()  # [B, blocks, 2, h_kv, D]
    low, high = x[:, :, 0].permute(0, 2, 3, 1), x[:, :, 1].permute(0, 2, 3, 1)
    q = s["q"].double().view(len(have), case["h_kv"], -1, D)
    score = (q.clamp(min=0) @ high + q.clamp(max=0) @ low).amax(2)  # 64 bits: the order of close scores counts
    score = torch.where(score.isnan(), math.inf, score)
    t = torch.arange(score.shape[-1], device=score.device)
    rank = torch.where((t < case["first"]) | (t >= have - case["last"]), 2, 1).masked_fill(t >= have, 0)[:, None].expand(score.shape)
    order = score.sort(dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, rank.gather(-1, order).sort(dim=-1, descending=True, stable=True).indices)[..., : case["count"]]
    some = torch.where(order < have[..., None], order, len(t)).sort(-1).values
    some = torch.where(some < have[..., None], some, -1)
    return torch.nn.functional.pad(some, (0, case["count"] - some.shape[-1]), value=-1).int()


def _rows(s, k, at):
    """The cache's rows of logical positions `at` [batch, heads, n], in 32 bits: [batch, heads, n, D]."""
    case = s["case"]
    c = s["caches"][k]
    block = s["table"].gather(1, (at // case["block"]).flatten(1)).view(at.shape).clamp(min=0).long()
    x = _bytes(c)[block, at % case["block"], torch.arange(case["h_kv"], device=at.device)[:, None]]
    return x.view(c.dtype).float() * s["scales"][k][:, None, None] if case["fp8"] else x.float()


def _attend(s, at, seen):
    """Softmax attention in 32 bits of each sequence's query over rows `at` where `seen`, and the weights."""
    case = s["case"]
    q = s["q"].float().view(len(s["q"]), case["h_kv"], -1, D)
    x = (q @ _rows(s, 0, at).transpose(-1, -2)) * D ** -0.5
    x = x.masked_fill(~seen[:, :, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp()
    x = x / x.sum(-1, keepdim=True)
    return (x @ _rows(s, 1, at)).reshape(s["q"].shape).to(s["q"].dtype), x


def _plain_blocks(s):
    block = s["case"]["block"]
    some = s["selected"].long()
    at = (some.clamp(min=0)[..., None] * block + torch.arange(block, device=some.device)).flatten(2)
    seen = (some >= 0).repeat_interleave(block, -1) & (at < s["lens"][:, None, None])
    return _attend(s, at.minimum(s["lens"].long()[:, None, None] - 1), seen)[0]


def _plain_weights(s):
    case, w = s["case"], s["weights"]
    lens = s["lens"].long()[:, None, None]
    t = torch.arange(s["max_len"], device=w.device).expand(len(lens), case["h_kv"], -1)
    out, p = _attend(s, t.minimum(lens - 1), t < lens)
    seq, head, pos = (t < lens).nonzero(as_tuple=True)
    at = s["table"][seq, pos // case["block"]].long(), head, pos % case["block"]
    w[at] = torch.where(pos < lens[seq, 0, 0] - 1, w[at], 0) + p.sum(2)[seq, head, pos]
    return {"out": out, "weights": w}


def _plain_evict(s):
    case, w = s["case"], s["weights"]
    block, keep, h_kv = case["block"], case["keep"], case["h_kv"]
    lens = s["lens"].long()
    kept = torch.full((len(lens), h_kv, keep), -1, device=lens.device)
    moved = torch.where(lens > case["limit"], keep - lens, 0)
    cut = (lens > case["limit"]).nonzero()[:, 0]
    if len(cut):
        n, table = lens[cut, None, None], s["table"][cut].long()
        head = torch.arange(h_kv, device=lens.device)[:, None]
        t = torch.arange(s["max_len"], device=lens.device)
        at = t.minimum(n - 1).expand(-1, h_kv, -1)
        x = w[table.gather(1, (at // block).flatten(1)).view(at.shape), head, at % block]
        x = x.masked_fill(t >= n - case["recent"], math.inf).masked_fill(t >= n, -math.inf)
        some = x.sort(dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values
        place = torch.arange(keep, device=lens.device).expand(some.shape)
        source, target = (table.gather(1, (x // block).flatten(1)).view(x.shape) for x in (some, place))
        for c in map(_bytes, s["caches"]):
            c[target, place % block, head] = c[source, some % block, head]
        w[target, head, place % block] = w[source, head, some % block]
        kept[cut] = some
    return {"k": s["caches"][0], "v": s["caches"][1], "weights": w, "moved": moved.int(), "kept": kept.int()}


# ------------------------------------------------------------------ one pass


def run(state):
    s = state
    case = s["case"]
    op = case["op"]
    if not own:
        return {"bounds": _plain_bounds, "select": _plain_select, "blocks": _plain_blocks, "weights": _plain_weights, "evict": _plain_evict}[op](s)
    import gqa_mqa_mla_gb300 as da
    most = s["max_len"]
    if op == "bounds":
        return da.gqa_block_bounds(s["k"], s["table"], s["lens"], s["bounds"], first_lens=s["first"] if case["new"] else None, max_seq_len=most)
    if op == "select":
        return da.gqa_select_blocks(s["q"], s["bounds"], s["table"], s["lens"], block_size=case["block"], max_seq_len=most, count=case["count"], first=case["first"], last=case["last"])
    if op == "blocks":
        if case["fp8"]:
            return da.gqa_decode_fp8kv_blocks(s["q"], *s["caches"], *s["scales"], s["table"], s["lens"], s["selected"], scale=D ** -0.5, max_seq_len=most)
        return da.gqa_decode_blocks(s["q"], *s["caches"], s["table"], s["lens"], s["selected"], scale=D ** -0.5, max_seq_len=most)
    if op == "weights":
        if case["fp8"]:
            out = da.gqa_decode_fp8kv_weights(s["q"], *s["caches"], *s["scales"], s["weights"], s["table"], s["lens"], scale=D ** -0.5, max_seq_len=most)
        else:
            out = da.gqa_decode_weights(s["q"], *s["caches"], s["weights"], s["table"], s["lens"], scale=D ** -0.5, max_seq_len=most)
        return {"out": out, "weights": s["weights"]}
    e = da.gqa_kv_evict(*s["caches"], s["weights"], s["table"], s["lens"], max_seq_len=most, keep=case["keep"], recent=case["recent"], limit=case["limit"])
    return {"k": s["caches"][0], "v": s["caches"][1], "weights": s["weights"], "moved": e.new_lens, "kept": e.kept}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    op, block, h_kv = case["op"], case["block"], case["h_kv"]
    if op == "select":
        return None  # whole numbers
    s = prepare(case, seed)
    lens = _lens(case)
    if op == "evict":
        o = [x.double() for x in (*s["caches"], s["weights"])]
        old = case["keep"] - case["recent"]
        for b, n in enumerate(lens):
            if n <= case["limit"]:
                continue
            ids = s["table"][b, : _blocks(n, block)].long()
            for h in range(h_kv):
                w = s["weights"][ids, h].flatten()[: n - case["recent"]]
                heavy = torch.argsort(-w, stable=True)[:old].sort().values
                at = torch.cat([heavy, torch.arange(n - case["recent"], n, device="cuda")])
                to = torch.arange(case["keep"], device="cuda")
                for x in o[:2]:
                    x[ids[to // block], to % block, h] = x[ids[at // block], at % block, h]
                o[2][ids[to // block], h, to % block] = o[2][ids[at // block], h, at % block]
        return {"k": o[0], "v": o[1], "weights": o[2], "moved": None, "kept": None}
    if op == "bounds":
        o, table = s["bounds"].double(), s["table"].tolist()
        for b, (n, f) in enumerate(zip(lens, _first(case, lens))):
            for t in range(min(f, n - 1) // block, _blocks(n, block)):
                i = table[b][t]
                x = s["k"][i, : n - t * block].double()
                o[i, 0], o[i, 1] = x.min(0).values, x.max(0).values
        return o
    g = case["h_q"] // h_kv
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    w = s["weights"].double() if op == "weights" else None
    for b, n in enumerate(lens):
        blocks = s["table"][b, : _blocks(n, block)].long()
        kv = []
        for j in (0, 1):
            c = s["caches"][j]
            x = _bytes(c)[blocks].view(c.dtype).double().flatten(0, 1)[:n]
            kv.append(x * s["scales"][j].double()[:, None] if case["fp8"] else x)
        for h in range(h_kv):
            k, v = kv[0][:, h], kv[1][:, h]
            if op == "blocks":
                some = s["selected"][b, h]
                some = some[some >= 0].long()
                at = (some[:, None] * block + torch.arange(block, device="cuda")).flatten()
                at = at[at < n]
                k, v = k[at], v[at]
            p = torch.softmax(s["q"][b, h * g: (h + 1) * g].double() @ k.T / math.sqrt(D), -1)
            o[b, h * g: (h + 1) * g] = p @ v
            if op == "weights":
                row = torch.zeros(len(blocks) * block, dtype=torch.float64, device="cuda")
                row[: n - 1] = w[blocks, h].flatten()[: n - 1]
                row[:n] += p.sum(0)
                past = w[blocks, h].flatten()[n:]
                row[n:] = past
                w[blocks, h] = row.view(-1, block)
    return {"out": o, "weights": w} if op == "weights" else o
