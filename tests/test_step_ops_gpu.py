"""The serving step's operators on the GPU against their plain forms in 64
bits (oracle/step.py): the paged plan, the rotary cache write, attention of a
chunk of new tokens, windowed decode with kept first tokens, and a run of them
together.

Tolerances of the attention outputs, per element, from the arithmetic (u = half
a step of the 16-bit type, relative): the output's own rounding u |out|; the
probabilities' rounding u sum p |v| / sum p =: u A; a score error of D = 130
2^-24 |scale| sum |q| |k| (fp32 sums of 128 products, two more roundings)
changes p and the sum by D each, 2 D A; 2^-19 A for exp2, the sums and the
division in fp32; and, for fp16 probabilities, what falls below half of their
smallest step, 2^-25 sum |v| / sum e^(s - max)."""
import numpy as np
import pytest
import torch

import gqa_mqa_mla_gb300 as da
import oracle
from gqa_mqa_mla_gb300 import synth
from oracle import step

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"bf16": 2.0**-8, "fp16": 2.0**-11}


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _close(got, ref, dtype, what=""):
    out, spread, tiny, reach = ref
    u = HALF[dtype]
    tol = u * np.abs(out) + (u + 2.0**-19 + 2 * 130 * 2.0**-24 * reach[..., None]) * spread
    if dtype == "fp16":
        tol = tol + 2.0**-25 * tiny
    got = got.double().cpu().numpy()
    live = ~np.isnan(out)
    assert np.isfinite(got[live]).all(), what
    err = np.abs(got - out)[live]
    worst = (err / (tol[live] + 1e-30)).max() if err.size else 0.0
    assert (err <= tol[live]).all(), (what, float(err.max()), float(worst))


# ------------------------------------------------------------------ paged plan


def _plan_case(rng, B, bs, M, lo, hi, spare):
    cached = rng.integers(0, M * bs + 1, B)
    new = np.clip(rng.integers(lo, hi + 1, B), -cached, M * bs - cached)
    held = -(-cached // bs)
    nb = max(1, int(held.sum()) + spare)
    ids = rng.permutation(nb)
    table = np.full((B, M), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(nb, -1)
    free[:nb - at] = ids[at:]
    return cached, new, table, free, nb - at


def _run_plan(cached, new, table, free, count, bs, tokens, **kw):
    t, f, c = _i32(table), _i32(free), _i32([count])
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = da.paged_plan(_i32(cached), _i32(new), t, f, c, block_size=bs, max_tokens=tokens,
                      err_flag=flag, **kw)
    torch.cuda.synchronize()
    return dict(table=t, free=f, count=p.free_count, seq_lens=p.seq_lens, q_start=p.q_start,
                slots=p.slots, positions=p.positions, flag=flag)


def _same_plan(got, want):
    for k, v in want.items():
        g = got[k].cpu().numpy()
        assert np.array_equal(g.reshape(np.shape(v)), v), (k, g, v)


@pytest.mark.parametrize("B,bs,M,lo,hi,spare,tokens", [
    (1, 16, 8, 1, 1, 5, 1), (1, 8, 4, -40, 40, 9, 64), (7, 16, 9, -30, 60, 100, 500),
    (64, 16, 32, 1, 1, 70, 64), (300, 64, 5, -100, 200, 900, 40000),
    (1025, 8, 6, -20, 48, 6000, 30000), (3000, 256, 3, -300, 3, 10, 9001),
])
def test_plan_matches_the_plain_form(B, bs, M, lo, hi, spare, tokens):
    rng = np.random.default_rng(B + bs)
    for _ in range(3):
        case = _plan_case(rng, B, bs, M, lo, hi, spare)
        want = step.paged_plan(*case, block_size=bs, max_tokens=tokens)
        _same_plan(_run_plan(*case, bs, tokens), want)


@pytest.mark.parametrize("B,tokens", [(5, 30), (5, 4000), (600, 4000)])
def test_plan_without_room_trims_and_grows_nothing(B, tokens):
    rng = np.random.default_rng(7)
    cached, new, table, free, count = _plan_case(rng, B, 16, 10, 30, 150, 6 * B)
    new[0] = -min(cached[0], 16)  # one request gives a block back
    # too few blocks, then too few rows
    for n_free, rows in ((min(2, count), tokens * 50), (count, 3)):
        want = step.paged_plan(cached, new, table, free, n_free, block_size=16, max_tokens=rows)
        assert want["flag"] == step.NO_ROOM and want["q_start"][-1] == 0
        _same_plan(_run_plan(cached, new, table, free, n_free, 16, rows), want)


def test_plan_bad_lengths_bad_pool_and_bad_ids():
    table, free = np.arange(12).reshape(3, 4), np.arange(12, 20)
    free = np.concatenate([free, np.full(12, -1)])
    cases = [([-5, 20, 30], [1, 1, 1], 8), ([20, 65, 30], [1, 1, -30], 8), ([20, 10, 30], [1, -11, 60], 8),
             ([20, 10, 30], [13, 1, -30], -1), ([20, 10, 30], [13, 1, -30], 21),
             ([20, 10, 30], [-20, 1, -30], 18)]
    for cached, new, count in cases:
        want = step.paged_plan(cached, new, table, free, count, block_size=16, max_tokens=40)
        assert want["flag"] in (step.BAD_SEQ_LEN, step.BAD_BLOCK)
        _same_plan(_run_plan(cached, new, table, free, count, 16, 40), want)
    bad = free.copy()
    bad[7], bad[5] = 99, -3
    t2 = table.copy()
    t2[1, 0] = 20  # the block that request 1 fills further
    want = step.paged_plan([16, 10, 30], [20, 2, 30], t2, bad, 8, block_size=16, max_tokens=80)
    assert want["flag"] == step.BAD_BLOCK and (want["slots"][:52] == -1).sum() > 10
    _same_plan(_run_plan([16, 10, 30], [20, 2, 30], t2, bad, 8, 16, 80), want)


def test_plan_in_place_over_many_steps_and_in_a_graph():
    """Lengths and free count updated in place, step after step, equal the plain
    form's; a captured call replays on the state it finds."""
    rng = np.random.default_rng(11)
    B, bs, M, T = 40, 16, 20, 2100
    cached, _, table, free, count = _plan_case(rng, B, bs, M, 0, 0, 400)
    lens, t, f, c = _i32(cached), _i32(table), _i32(free), _i32([count])
    new = _i32(np.zeros(B))
    bufs = dict(q_start=_i32(np.zeros(B + 1)), slots=_i32(np.zeros(T)), positions=_i32(np.zeros(T)))
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        da.paged_plan(lens, new, t, f, c, block_size=bs, max_tokens=T, seq_lens=lens,
                      free_count_out=c, **bufs)
    for _ in range(12):
        n = np.clip(rng.integers(-60, 60, B), -cached, M * bs - cached)
        new.copy_(_i32(n))
        graph.replay()
        torch.cuda.synchronize()
        want = step.paged_plan(cached, n, table, free, count, block_size=bs, max_tokens=T)
        _same_plan(dict(table=t, free=f, count=c, seq_lens=lens, **bufs),
                   {k: want[k] for k in want if k != "flag"})
        cached, table, free, count = want["seq_lens"], want["table"], want["free"], want["count"]


# ------------------------------------------------------------------ rotary cache write


def _rope_case(T, h_q, h_kv, dtype, bs, fp8, seed, fused=True):
    g = _gen(seed)
    qkv = torch.randn((T, (h_q + 2 * h_kv) * 128), generator=g, device=DEV).to(TYPES[dtype])
    parts = [p.view(T, -1, 128) for p in qkv.split([h_q * 128, h_kv * 128, h_kv * 128], 1)]
    if not fused:
        parts = [p.contiguous() for p in parts]
    nb = -(-T // bs) + 2
    caches = [torch.randn((nb, bs, h_kv, 128), generator=g, device=DEV).to(TYPES[dtype])
              for _ in range(2)]
    scales = None
    if fp8:
        caches = [c.float().to(torch.float8_e4m3fn).view(torch.uint8) for c in caches]
        scales = [(torch.rand(h_kv, generator=g, device=DEV) + 0.5) / 112 for _ in range(2)]
    slots = torch.randperm(nb * bs, generator=g, device=DEV)[:T].int()
    return parts, caches, scales, slots


@pytest.mark.parametrize("T,h_q,h_kv,dtype,bs,fp8,axes,rot,inter,fused", [
    (1, 8, 2, "bf16", 16, False, 1, 128, False, True),
    (5, 5, 1, "fp16", 8, False, 3, 128, True, True),
    (33, 64, 8, "bf16", 64, False, 3, 128, False, False),
    (130, 32, 32, "fp16", 256, False, 2, 64, False, True),
    (17, 28, 4, "bf16", 16, False, 1, 96, True, False),
    (1, 8, 8, "fp16", 16, True, 1, 128, False, True),
    (70, 12, 4, "bf16", 32, True, 3, 32, True, True),
    (41, 64, 8, "fp16", 16, True, 2, 112, False, False),
    (9, 40, 40, "bf16", 128, True, 1, 16, False, True),
])
def test_rope_append_matches_the_plain_form(T, h_q, h_kv, dtype, bs, fp8, axes, rot, inter, fused):
    (q, k, v), caches, scales, slots = _rope_case(T, h_q, h_kv, dtype, bs, fp8, T + rot, fused)
    pairs = rot // 2
    freq = [1e4 ** (-i / pairs) for i in range(pairs)]
    cut = [pairs - (axes - 1) * (pairs // axes)] + [pairs // axes] * (axes - 1)
    axis = [a for a, n in enumerate(cut) for _ in range(n)]
    pos = torch.randint(-1000, 2**31 - 1, (axes, T), generator=_gen(9), device=DEV, dtype=torch.int32)
    pos[:, : T // 2] %= 5000
    if T > 4:
        slots[T // 3] = -1
    before = [c.clone() for c in caches]
    rope = da.rope_table(freq, sections=cut, interleaved=inter)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    if fp8:
        got = da.gqa_rope_append_fp8kv(q, k, v, *scales, pos, rope, slots, *caches, err_flag=flag)
    else:
        got = da.gqa_rope_append(q, k, v, pos, rope, slots, *caches, err_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == 0
    host = [x.double().cpu().numpy() for x in (q, k, v)]
    p = pos.cpu().numpy()
    # Angles: the phase is exact to 2^-32 + 2^-25 of a turn (its float), and the
    # plain form's own product rounds by 2^-53 |angle|; sine and cosine 2^-22.
    slack = 2 * np.pi * 2.0**-24 + 2.0**-21
    want = step.rope(host[0], p, freq, axis, inter)
    size = np.sqrt((host[0] ** 2).max())
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= HALF[dtype] * np.abs(want) + 2 * slack * size).all(), err.max()
    sl, live = slots.cpu().numpy(), (slots >= 0).cpu().numpy()
    for c, c0, x, j in zip(caches, before, (step.rope(host[1], p, freq, axis, inter), host[2]), (0, 1)):
        flat, flat0 = c.view(-1, h_kv, 128), c0.view(-1, h_kv, 128)
        rows = slots[slots >= 0].long()
        keep = torch.ones(len(flat), dtype=torch.bool, device=DEV)
        keep[rows] = False
        assert torch.equal(flat[keep], flat0[keep])
        x = x[live]
        if not fp8:
            w = flat[rows].double().cpu().numpy()
            near = 2 * slack * size if j == 0 else 0.0
            assert (np.abs(w - x) <= HALF[dtype] * np.abs(x) + near).all()
            continue
        # The stored value: within half an e4m3 step (2^-4 relative, 2^-10 below
        # the smallest normal) of x / scale, up to the angle's error and the two
        # fp32 roundings; 448 beyond it.
        code = oracle.e4m3_to_double(flat[rows].cpu().numpy())
        y = np.clip(x / scales[j].double().cpu().numpy()[None, :, None], -448, 448)
        off = 2 * slack * size * 300 if j == 0 else 0.0
        assert (np.abs(code - y) <= 2.0**-4 * np.abs(y) + 2.0**-10 + off + 2.0**-22 * np.abs(y)).all()


def test_rope_append_in_place_past_the_cache_and_single_axis_vector():
    (q, k, v), caches, _, slots = _rope_case(6, 8, 2, "bf16", 16, False, 1, fused=False)
    rope = da.rope_table([0.5 ** i for i in range(64)])
    pos = torch.arange(6, dtype=torch.int32, device=DEV)
    other = [c.clone() for c in caches]
    want = da.gqa_rope_append(q, k, v, pos, rope, slots, *other)
    slots2 = slots.clone()
    slots2[2] = caches[0].shape[0] * 16  # one past the last slot
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    ret = da.gqa_rope_append(q, k, v, pos, rope, slots2, *caches, q_out=q, err_flag=flag)
    torch.cuda.synchronize()
    assert ret.data_ptr() == q.data_ptr() and torch.equal(q, want)
    assert int(flag) == da.FLAG_BAD_BLOCK
    for c, o in zip(caches, other):
        a, b = c.view(-1, 2, 128), o.view(-1, 2, 128)
        keep = torch.ones(len(a), dtype=torch.bool, device=DEV)
        keep[slots[2].long()] = False
        assert torch.equal(a[keep], b[keep])


def test_rope_append_of_position_zero_moves_bytes():
    """No rotation: q comes back bit for bit and the cache rows are k and v."""
    (q, k, v), caches, _, slots = _rope_case(50, 4, 4, "fp16", 8, False, 2)
    rope = da.rope_table([0.3] * 64, interleaved=True)
    out = da.gqa_rope_append(q, k, v, torch.zeros(50, dtype=torch.int32, device=DEV), rope, slots, *caches)
    assert torch.equal(out, q)
    for c, x in zip(caches, (k, v)):
        assert torch.equal(c.view(-1, 4, 128)[slots.long()], x)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rope_append_quantises_as_the_single_token_write(dtype):
    """Without a turn the e4m3 codes are gqa_kv_append_fp8kv's bit for bit: every
    16-bit pattern (ties, signed zeros, subnormals, infinities, NaN) under scales
    that make ties, odd ones, tiny, huge, negative, zero and infinite ones."""
    h_kv, T = 16, 512
    scale = [1.0, 0.5, 1 / 448, 0.0123, 3.0, 7.7e-3, -0.3, 1e-19, 1e19, 2.0**-70, 2.0**70,
             1.9999999, 0.33333334, 1e-40, 0.0, float("inf")]
    scales = [torch.tensor(scale, device=DEV), torch.tensor(scale[::-1], device=DEV)]
    bits = torch.arange(2**16, device=DEV, dtype=torch.int32).to(torch.int16)
    rows = bits.view(TYPES[dtype]).view(T, 1, 128).repeat(1, h_kv, 1).contiguous()
    back = rows.flip(0).contiguous()
    nb = T // 16
    got = [torch.zeros((nb, 16, h_kv, 128), dtype=torch.uint8, device=DEV) for _ in range(2)]
    want = [torch.zeros_like(c) for c in got]
    rope = da.rope_table([0.0] * 64)
    slots = torch.arange(T, device=DEV, dtype=torch.int32)
    # (v is never turned; k only by zero angles: x * 1 - y * 0 is x where y is finite.)
    da.gqa_rope_append_fp8kv(rows, back, rows, *scales, _i32(np.zeros((1, T))), rope, slots, *got)
    table = torch.arange(nb, device=DEV, dtype=torch.int32)
    da.gqa_kv_append_fp8kv(back, rows, *scales, slots % 16, (table[slots.long() // 16])[:, None],
                           *want)
    torch.cuda.synchronize()
    assert torch.equal(got[1], want[1])
    flat = lambda c: c.view(T, h_kv, 128)  # noqa: E731
    x = back.float()
    partner = torch.cat([x[..., 64:], x[..., :64]], -1)
    plain = torch.isfinite(partner) & (x != 0)  # (a zero may gain the other sign: -0 + 0)
    assert bool(plain.any()) and torch.equal(flat(got[0])[plain], flat(want[0])[plain])


# ------------------------------------------------------------------ chunk attention


def _attn_case(q_lens, lens, h_q, h_kv, dtype, bs, seed, fp8=False, pad=0, tail="nan"):
    g = _gen(seed)
    table, nb = synth.make_block_table(torch.tensor(lens), bs, "permuted", seed, spare_blocks=2)
    shape = (nb, bs, h_kv, 128)
    if fp8:
        caches = [(torch.randn(shape, generator=g, device=DEV) * 112).clamp_(-448, 448)
                  .to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
        scales = [(torch.rand(h_kv, generator=g, device=DEV) + 0.5) / 112 for _ in range(2)]
    else:
        caches = [torch.randn(shape, generator=g, device=DEV).to(TYPES[dtype]) for _ in range(2)]
        scales = None
    # Everything that no sequence holds is NaN.
    used = torch.zeros(nb * bs, dtype=torch.bool)
    for b, n in enumerate(lens):
        t = torch.arange(n)
        used[table[b][t // bs].long() * bs + t % bs] = True
    if tail == "nan":
        for c in caches:
            c.view(nb * bs, h_kv, 128)[~used.to(DEV)] = 0x7F if fp8 else float("nan")
    start = np.concatenate([[0], np.cumsum(q_lens)])
    q = torch.randn((int(start[-1]) + pad, h_q, 128), generator=g, device=DEV).to(TYPES[dtype])
    return dict(q=q, caches=caches, scales=scales, table=table.to(DEV), start=_i32(start),
                lens=_i32(lens), max_q=max(1, max(q_lens)), max_len=max(lens), dtype=dtype)


def _plain_cache(x):
    r = []
    for j, c in enumerate(x["caches"]):
        if x["scales"] is None:
            d = c.double()
        else:
            d = c.view(torch.float8_e4m3fn).double() * x["scales"][j].double()[:, None]
        r.append(np.nan_to_num(d.cpu().numpy()))
    return r


def _run_prefill(x, scale=128 ** -0.5, **kw):
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    fn = da.gqa_prefill if x["scales"] is None else da.gqa_prefill_fp8kv
    out = fn(x["q"], *x["caches"], *(x["scales"] or []), x["table"], x["start"], x["lens"],
             scale=scale, max_q_len=x["max_q"], max_seq_len=x["max_len"], err_flag=flag, **kw)
    torch.cuda.synchronize()
    return out, int(flag)


def _plain_prefill(x, scale=128 ** -0.5, window=0, sinks=0):
    return step.attend(x["q"].double().cpu().numpy(), *_plain_cache(x), x["table"].cpu().numpy(),
                       x["start"].cpu().numpy(), x["lens"].cpu().numpy(), scale=scale,
                       window=window, sinks=sinks)


CHUNKS = [
    # q_lens, lens, h_q, h_kv, dtype, block, window, sinks
    ([1], [1], 8, 1, "bf16", 16, 0, 0),
    ([5], [5], 8, 8, "fp16", 16, 0, 0),
    ([1, 1, 1], [1, 128, 300], 16, 2, "bf16", 16, 0, 0),
    ([3, 0, 7, 2], [130, 77, 7, 500], 8, 2, "bf16", 8, 0, 0),
    ([129], [129], 2, 2, "bf16", 64, 0, 0),
    ([257, 5], [257, 640], 2, 1, "fp16", 128, 0, 0),
    ([40, 33], [700, 33], 28, 4, "bf16", 256, 0, 0),
    ([20], [150], 5, 1, "fp16", 32, 0, 0),
    ([9, 64], [200, 64], 64, 1, "bf16", 16, 0, 0),
    ([10], [90], 33, 1, "bf16", 16, 0, 0),
    ([300], [1000], 4, 4, "bf16", 16, 0, 0),
    ([2, 2], [0, 1], 8, 2, "fp16", 16, 0, 0),          # rows before position 0 see nothing
    ([300], [290], 2, 2, "bf16", 16, 0, 0),
    ([50, 1, 200], [400, 900, 200], 8, 2, "bf16", 16, 1, 0),
    ([50, 1, 200], [400, 900, 200], 8, 2, "fp16", 16, 60, 0),
    ([50, 3, 200], [400, 900, 333], 8, 2, "bf16", 16, 60, 4),
    ([50, 3, 200], [400, 900, 333], 4, 4, "fp16", 256, 129, 130),
    ([80], [500], 16, 2, "bf16", 8, 100, 250),
    ([80], [500], 16, 2, "bf16", 64, 100, 1000),
    ([10, 260], [700, 760], 1, 1, "bf16", 32, 300, 17),
    ([17], [600], 8, 1, "fp16", 16, 5, 1),
]


@pytest.mark.parametrize("splits", [1, 0, 3])
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_prefill_matches_the_plain_form(case, splits):
    q_lens, lens, h_q, h_kv, dtype, bs, window, sinks = CHUNKS[case]
    x = _attn_case(q_lens, lens, h_q, h_kv, dtype, bs, case)
    out, flag = _run_prefill(x, window=window or None, sinks=sinks, num_splits=splits)
    assert flag == 0
    _close(out, _plain_prefill(x, window=window, sinks=sinks), dtype)


def _fp16_probs(ref, dtype):
    """An 8-bit cache's probabilities are fp16 for either output type: fewer
    bits are lost than bf16's bound allows, but their lost small values count."""
    return ref if dtype == "fp16" else (ref[0], ref[1] + 2.0**-25 * ref[2] / HALF[dtype], *ref[2:])


@pytest.mark.parametrize("splits", [1, 0, 3])
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_prefill_over_an_8_bit_cache(case, splits):
    q_lens, lens, h_q, h_kv, dtype, bs, window, sinks = CHUNKS[case]
    for kind in ("bf16", "fp16") if splits == 1 else (dtype,):
        x = _attn_case(q_lens, lens, h_q, h_kv, kind, bs, 200 + case, fp8=True)
        out, flag = _run_prefill(x, window=window or None, sinks=sinks, num_splits=splits)
        assert flag == 0
        _close(out, _fp16_probs(_plain_prefill(x, window=window, sinks=sinks), kind), kind)


def test_prefill_over_an_8_bit_cache_with_odd_scales():
    """Negative and zero head scales, a negative scale, bad blocks."""
    x = _attn_case([30, 140], [200, 140], 6, 3, "bf16", 16, 250, fp8=True)
    x["scales"][0].mul_(torch.tensor([-1.0, 0.0, 1.0], device=DEV))
    x["scales"][1].mul_(torch.tensor([1.0, -1.0, 0.0], device=DEV))
    for scale in (0.09, -0.09):
        for splits in (1, 2):
            out, flag = _run_prefill(x, scale=scale, num_splits=splits)
            assert flag == 0
            _close(out, _fp16_probs(_plain_prefill(x, scale=scale), "bf16"), "bf16")
    ref = _plain_prefill(x)
    x["table"][0, 5] = -1
    out, flag = _run_prefill(x)
    assert flag == da.FLAG_BAD_BLOCK and bool((out[:30] == 0).all())
    for a in ref:
        a[:30] = np.nan
    _close(out, _fp16_probs(ref, "bf16"), "bf16")


def test_prefill_more_pieces_than_sms():
    """CTAs take over waiting pieces: a ragged batch of many pieces, twice, bit
    for bit the same (a piece's result does not depend on who computes it)."""
    rng = np.random.default_rng(9)
    q_lens = rng.integers(0, 70, 60).tolist()
    lens = [n + int(rng.integers(0, 200)) for n in q_lens]
    for fp8 in (False, True):
        x = _attn_case(q_lens, lens, 16, 4, "fp16", 16, 300, fp8=fp8)
        a, flag = _run_prefill(x, num_splits=1)
        b, _ = _run_prefill(x, num_splits=1)
        assert flag == 0 and torch.equal(a, b)
        rows = np.sort(rng.choice(int(sum(q_lens)), 40, replace=False))
        start = np.concatenate([[0], np.cumsum(q_lens)])
        for i in rows:  # each sampled row on its own, as a chunk of one token
            s = int(np.searchsorted(start, i, side="right") - 1)
            n = lens[s] - q_lens[s] + int(i - start[s]) + 1
            y = dict(x, q=x["q"][i: i + 1], table=x["table"][s: s + 1], start=_i32([0, 1]),
                     lens=_i32([n]))
            ref = _plain_prefill(y)
            _close(a[i: i + 1], ref, "fp16")


@pytest.mark.parametrize("scale", [-0.07, 0.0, 1.5])
def test_prefill_scales(scale):
    """A negative scale, equal weights, and a sharp softmax (rescaling)."""
    x = _attn_case([30, 140], [200, 140], 4, 2, "bf16", 16, 50)
    for splits in (1, 2):
        out, flag = _run_prefill(x, scale=scale, num_splits=splits)
        assert flag == 0
        _close(out, _plain_prefill(x, scale=scale), "bf16", scale)


@pytest.mark.parametrize("growth", [1, -1])
def test_prefill_running_maximum(growth):
    """Scores that grow (or shrink) along the cache move the running maximum in
    every tile (or in the first only)."""
    x = _attn_case([70], [900], 8, 2, "fp16", 16, 51)
    t = torch.arange(900, device=DEV)
    rows = x["table"][0][t // 16].long() * 16 + t % 16
    ramp = (t if growth > 0 else 900 - t).float()[:, None, None] / 900
    k = x["caches"][0].view(-1, 2, 128)
    k[rows] = (k[rows].float() * 0.1 + 3 * ramp).half()
    x["q"] = (x["q"].float() * 0.1 + 1).half()
    for splits in (1, 4):
        out, _ = _run_prefill(x, num_splits=splits)
        _close(out, _plain_prefill(x), "fp16")


def test_prefill_leaves_rows_behind_the_last_sequence():
    x = _attn_case([30, 0, 11], [30, 50, 300], 8, 2, "bf16", 16, 52, pad=9)
    for splits in (1, 3):
        out = torch.full_like(x["q"], 7.0)
        got, flag = _run_prefill(x, out=out, num_splits=splits)
        assert got is out and flag == 0 and bool((out[-9:] == 7).all())
        _close(out, _plain_prefill(x), "bf16")
    # rows before the first sequence too
    x["start"] = x["start"] + 4
    out = torch.full_like(x["q"], 7.0)
    _run_prefill(x, out=out)
    assert bool((out[:4] == 7).all()) and bool((out[-5:] == 7).all())
    _close(out, _plain_prefill(x), "bf16")


def test_prefill_bad_lengths_blocks_and_offsets():
    x = _attn_case([30, 20, 11], [30, 150, 300], 8, 2, "bf16", 16, 53)
    ref = _plain_prefill(x)
    for splits in (1, 3):
        for what, flag in (("len", da.FLAG_BAD_SEQ_LEN), ("neg", da.FLAG_BAD_SEQ_LEN),
                           ("block", da.FLAG_BAD_BLOCK)):
            y = dict(x, lens=x["lens"].clone(), table=x["table"].clone())
            if what == "block":
                y["table"][1, 3] = 10**6
            else:
                y["lens"][1] = 301 if what == "len" else -2
            out, got = _run_prefill(y, num_splits=splits)
            assert got == flag and bool((out[30:50] == 0).all()), what
            r = [a.copy() for a in ref]
            for a in r:
                a[30:50] = np.nan
            _close(out, r, "bf16", what)
        for start in ([0, 30, 20, 61], [0, -5, 50, 61], [0, 30, 50, 62], [0, 30, 50, 50 + 2**30]):
            out, got = _run_prefill(dict(x, start=_i32(start)), num_splits=splits)
            assert got & da.FLAG_BAD_SEQ_LEN
        out, got = _run_prefill(dict(x, max_q=29), num_splits=splits)
        assert got == da.FLAG_BAD_SEQ_LEN
        r = [a.copy() for a in ref]
        for a in r:
            a[:30] = np.nan
        _close(out, r, "bf16")


def test_prefill_reads_no_block_outside_the_window_and_the_sinks():
    x = _attn_case([20], [1000], 8, 2, "bf16", 16, 54)
    first = 980 + 1 - 100  # the first row's window start
    y = dict(x, table=x["table"].clone())
    y["table"][0, 1: first // 16] = -1
    for splits in (1, 2):
        out, flag = _run_prefill(y, window=100, sinks=9, num_splits=splits)
        assert flag == 0
        _close(out, _plain_prefill(x, window=100, sinks=9), "bf16")


def test_prefill_on_many_sequences_and_another_stream():
    rng = np.random.default_rng(5)
    q_lens = rng.integers(0, 4, 500).tolist()
    lens = [n + int(rng.integers(0, 60)) for n in q_lens]
    x = _attn_case(q_lens, lens, 4, 2, "fp16", 8, 55)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, flag = _run_prefill(x)
    assert flag == 0
    _close(out, _plain_prefill(x), "fp16")
    again, _ = _run_prefill(x, stream=s)
    assert torch.equal(again, out)


def test_prefill_of_one_token_is_decode():
    x = _attn_case([1] * 6, [1, 64, 65, 300, 511, 130], 16, 2, "bf16", 16, 56)
    ref = da.gqa_decode(x["q"], *x["caches"], x["table"], x["lens"], scale=0.09,
                        max_seq_len=x["max_len"])
    out, _ = _run_prefill(x, scale=0.09)
    plain = _plain_prefill(x, scale=0.09)
    _close(out, plain, "bf16")
    _close(ref, plain, "bf16")


def test_prefill_in_a_graph_with_a_shared_workspace():
    """Two captured calls share one workspace; replays on new data in the same
    buffers give what eager calls give."""
    x = _attn_case([4, 2], [700, 300], 8, 2, "bf16", 16, 57)
    y = _attn_case([3, 3], [650, 200], 8, 2, "bf16", 16, 58)
    ws = torch.empty(da.gqa_prefill_workspace_size(6, 8, 4), dtype=torch.uint8, device=DEV)
    outs = [torch.zeros_like(z["q"]) for z in (x, y)]
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        for z, o in zip((x, y), outs):
            da.gqa_prefill(z["q"], *z["caches"], z["table"], z["start"], z["lens"], scale=0.1,
                           max_q_len=z["max_q"], max_seq_len=z["max_len"], num_splits=4,
                           workspace=ws, out=o)
    for seed in (1, 2):
        for z in (x, y):
            z["q"].copy_(torch.randn(z["q"].shape, generator=_gen(seed), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        for z, o in zip((x, y), outs):
            _close(o, _plain_prefill(z, scale=0.1), "bf16")


# ------------------------------------------------------------------ decode with sinks


SINKS = [
    # lens, h_q, h_kv, dtype, block, window, sinks
    ([1, 5, 64, 65, 0], 8, 8, "bf16", 16, 3, 1),
    ([300, 64, 500, 129], 16, 2, "bf16", 16, 60, 4),
    ([300, 64, 500, 129], 8, 8, "fp16", 8, 100, 64),
    ([300, 700, 500, 129], 32, 1, "bf16", 64, 70, 66),
    ([1000, 900], 64, 1, "fp16", 256, 200, 130),
    ([1000, 450], 9, 1, "bf16", 32, 300, 500),
    ([1000, 450, 77], 28, 4, "fp16", 128, 129, 7),
    ([2000], 16, 4, "bf16", 16, 1, 1999),
    ([2000], 16, 4, "bf16", 16, 1000, 1000),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("splits", [1, 0, 4])
@pytest.mark.parametrize("case", range(len(SINKS)))
def test_sinks_decode_matches_the_plain_form(case, splits, fp8):
    lens, h_q, h_kv, dtype, bs, window, sinks = SINKS[case]
    x = _attn_case([1] * len(lens), lens, h_q, h_kv, dtype, bs, 70 + case, fp8=fp8)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    # Blocks between the sinks and the window may have been given away.
    table = x["table"].clone()
    for b, n in enumerate(lens):
        first = max(0, n - window)
        if sinks < first:
            table[b, -(-sinks // bs): first // bs] = -1
    fn = da.gqa_decode_fp8kv_sinks if fp8 else da.gqa_decode_sinks
    out = fn(x["q"], *x["caches"], *(x["scales"] or []), table, x["lens"], scale=0.09,
             max_seq_len=x["max_len"], window=window, sinks=sinks, num_splits=splits,
             err_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == 0
    # (A row of an empty sequence has position -1: it sees nothing.)  An 8-bit
    # cache's probabilities, and up to 16 query heads per KV head its queries,
    # are fp16: less rounding than bf16's bound allows, but their lost small
    # values count for either type.
    ref = _plain_prefill(x, scale=0.09, window=window, sinks=sinks)
    if fp8:
        ref = (ref[0], ref[1] + 2.0**-25 * ref[2] / HALF[dtype], ref[2], ref[3])
    _close(out, ref, dtype)


def test_sinks_decode_flags_and_no_sinks():
    x = _attn_case([1, 1], [300, 400], 16, 2, "bf16", 16, 90)
    args = (x["q"], *x["caches"])
    kw = dict(scale=0.09, max_seq_len=400, window=64)
    a = da.gqa_decode_sinks(*args, x["table"], x["lens"], sinks=0, **kw)
    b = da.gqa_decode_window(*args, x["table"], x["lens"], **kw)
    assert torch.equal(a, b)
    for blk in (0, 24):  # in the sinks, in the window
        bad = x["table"].clone()
        bad[1, blk] = -7
        for splits in (1, 2):
            flag = torch.zeros(1, dtype=torch.int32, device=DEV)
            out = da.gqa_decode_sinks(*args, bad, x["lens"], sinks=4, err_flag=flag,
                                      num_splits=splits, **kw)
            torch.cuda.synchronize()
            assert int(flag) == da.FLAG_BAD_BLOCK and bool((out[1] == 0).all())
            assert bool(torch.isfinite(out[0]).all()) and bool((out[0] != 0).any())


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_a_run_of_steps(fp8, window, sinks):
    """Prompts in chunks, drafted tokens taken back, single tokens, a request
    that ends and another in its blocks: plan, rotate and write, attend; every
    step's rows equal attention over the tokens that each request holds, built
    without a cache.  The caches start as NaN."""
    h_q, h_kv, bs, M, B = 8, 2, 16, 24, 4
    nb, T, dtype = 60, 160, "bf16"
    g = _gen(100)
    freq = [1e4 ** (-i / 64) for i in range(64)]
    rope = da.rope_table(freq)
    shape = (nb, bs, h_kv, 128)
    if fp8:
        caches = [torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.tensor([1 / 64, 1 / 32], device=DEV) for _ in range(2)]
    else:
        caches = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        scales = []
    lens, table = _i32([0] * B), _i32(np.full((B, M), -1))
    free, count = _i32(np.random.default_rng(1).permutation(nb)), _i32([nb])
    held = [[np.zeros((0, h_kv, 128)) for _ in range(B)] for _ in range(2)]
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    steps = [[70, 33, 0, 5], [50, 1, 90, 1], [4, 1, 4, 1], [-3, 1, 0, 1], [1, -35, 1, 1],
             [1, 100, -2, 1], [1, 1, 1, 1]]
    cached = [0] * B
    for new in steps:
        p = da.paged_plan(lens, _i32(new), table, free, count, block_size=bs, max_tokens=T,
                          seq_lens=lens, free_count_out=count, err_flag=flag)
        qkv = torch.randn((T, (h_q + 2 * h_kv) * 128), generator=g, device=DEV).bfloat16()
        q, k, v = (x.view(T, -1, 128) for x in qkv.split([h_q * 128, h_kv * 128, h_kv * 128], 1))
        if fp8:
            qr = da.gqa_rope_append_fp8kv(q, k, v, *scales, p.positions, rope, p.slots, *caches,
                                          err_flag=flag)
        else:
            qr = da.gqa_rope_append(q, k, v, p.positions, rope, p.slots, *caches, err_flag=flag)
        single = max(new) <= 1 and min(new) == 1
        out = torch.zeros_like(qr)
        fn = da.gqa_prefill_fp8kv if fp8 else da.gqa_prefill
        fn(qr, *caches, *scales, table, p.q_start, lens, scale=0.09, max_q_len=T,
           max_seq_len=M * bs, window=window or None, sinks=sinks, out=out, err_flag=flag)
        if single and window:
            fn = da.gqa_decode_fp8kv_sinks if fp8 else da.gqa_decode_sinks
            dec = fn(qr[:B].contiguous(), *caches, *scales, table, lens, scale=0.09,
                     max_seq_len=M * bs, window=window, sinks=sinks, err_flag=flag)
        torch.cuda.synchronize()
        assert int(flag) == 0
        start = p.q_start.cpu().numpy()
        pos = p.positions.cpu().numpy()
        kv = [step.rope(k.double().cpu().numpy(), pos[None], freq, [0] * 64, False),
              v.double().cpu().numpy()]
        # What the cache holds of this step's rows (near the plain rotation; its
        # own test is stricter), kept per request without any paging.
        stored = []
        for j in (0, 1):
            rows = caches[j].view(-1, h_kv, 128)[p.slots[: start[-1]].long()]
            if fp8:
                rows = rows.view(torch.float8_e4m3fn).double() * scales[j].double()[:, None]
            stored.append(rows.double().cpu().numpy())
            plain = kv[j][: start[-1]]
            assert (np.abs(stored[j] - plain) <= (2.0**-4 if fp8 else 2.0**-8) * np.abs(plain)
                    + (2.0**-14 if fp8 else 2.0**-17)).all()
        for b, n in enumerate(new):
            cached[b] += n
            for j in (0, 1):
                held[j][b] = np.concatenate([held[j][b][: cached[b] - max(n, 0)],
                                             stored[j][start[b]:start[b + 1]]])
        assert lens.cpu().tolist() == cached
        # the same tokens in a cache of one block per request
        big = max(cached) + 1
        dense = [np.zeros((B, big, h_kv, 128)) for _ in range(2)]
        for j in (0, 1):
            for b in range(B):
                dense[j][b, : cached[b]] = held[j][b]
        ref = step.attend(qr.double().cpu().numpy(), *dense, np.arange(B)[:, None], start, cached,
                          scale=0.09, window=window, sinks=sinks)
        if fp8:
            ref = (ref[0], ref[1] + 2.0**-25 * ref[2] / HALF[dtype], ref[2], ref[3])
        _close(out, ref, dtype)
        if single and window:
            _close(dec, tuple(r[:B] for r in ref), dtype)


# ------------------------------------------------------------------ drawn cases


def _draw(seed):
    """Chunk lengths, cached lengths, heads, type, block, window and sinks."""
    rng = np.random.default_rng(1000 + seed)
    pick = lambda *x: x[int(rng.integers(len(x)))]  # noqa: E731
    B, most = pick(1, 2, 3, 5), pick(1, 3, 20, 150, 300)
    q_lens = rng.integers(0, most + 1, B).tolist()
    q_lens[0] = max(1, q_lens[0])
    lens = [n + int(rng.integers(0, pick(2, 130, 900))) for n in q_lens]
    h_kv = pick(1, 2, 3)
    h_q = h_kv * pick(1, 2, 3, 4, 7, 8, 12, 16)
    window = pick(0, 1, 2, int(rng.integers(1, 40)), int(rng.integers(40, 400)), 128, 2**31 - 1)
    sinks = pick(0, 1, 4, int(rng.integers(0, 300)), 128, 2**31 - 1) if window else 0
    return q_lens, lens, h_q, h_kv, pick("bf16", "fp16"), pick(8, 16, 32, 64, 128, 256), \
        window, sinks, pick(0, 1, 2, 3, 5, 8, 17)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seed", range(48))
def test_prefill_drawn(seed, fp8):
    q_lens, lens, h_q, h_kv, dtype, bs, window, sinks, splits = _draw(seed)
    x = _attn_case(q_lens, lens, h_q, h_kv, dtype, bs, 400 + seed, fp8=fp8)
    # The host's bounds need not be reached (the table must hold max_seq_len).
    x["max_len"] = min(x["max_len"] + seed % 3 * 100, x["table"].shape[1] * bs)
    x["max_q"] += seed % 4 * 5
    out, flag = _run_prefill(x, window=window or None, sinks=sinks, num_splits=splits)
    assert flag == 0
    ref = _plain_prefill(x, window=window, sinks=sinks)
    _close(out, _fp16_probs(ref, dtype) if fp8 else ref, dtype)
    again, _ = _run_prefill(x, window=window or None, sinks=sinks, num_splits=splits)
    assert torch.equal(again, out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seed", range(24))
def test_sinks_decode_drawn(seed, fp8):
    _, lens, h_q, h_kv, dtype, bs, window, sinks, splits = _draw(100 + seed)
    window, sinks = window or 77, sinks or 1
    x = _attn_case([1] * len(lens), lens, h_q, h_kv, dtype, bs, 500 + seed, fp8=fp8)
    fn = da.gqa_decode_fp8kv_sinks if fp8 else da.gqa_decode_sinks
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = fn(x["q"], *x["caches"], *(x["scales"] or []), x["table"], x["lens"], scale=0.09,
             max_seq_len=x["table"].shape[1] * bs, window=window, sinks=sinks,
             num_splits=splits, err_flag=flag)
    assert int(flag) == 0
    ref = _plain_prefill(x, scale=0.09, window=window, sinks=sinks)
    _close(out, _fp16_probs(ref, dtype) if fp8 else ref, dtype)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_of_an_empty_batch_and_of_empty_sequences(fp8):
    x = _attn_case([3, 2], [40, 50], 8, 2, "bf16", 16, 600, fp8=fp8)
    none = dict(x, start=_i32([0, 0, 0]))
    for splits in (1, 0, 3):
        out = torch.full_like(x["q"], 7.0)
        _, flag = _run_prefill(none, out=out, num_splits=splits)
        assert flag == 0 and bool((out == 7).all())
        # no rows at all
        got, flag = _run_prefill(dict(none, q=x["q"][:0]), num_splits=splits)
        assert flag == 0 and got.shape == (0, 8, 128)
        # rows of sequences that hold no token: zeros
        got, flag = _run_prefill(dict(x, lens=_i32([0, 0])), num_splits=splits)
        assert flag == 0 and bool((got == 0).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_uneven_batch_with_bad_sequences(fp8):
    """More pieces than SMs, taken in order of length: empty chunks, equal lengths,
    bad lengths and a chunk beyond the bound among them."""
    rng = np.random.default_rng(14)
    q_lens = rng.choice([0, 1, 1, 3, 40, 70], 90).tolist()
    q_lens[5], q_lens[40], q_lens[41], q_lens[89] = 40, 90, 1, 3
    lens = [n + int(rng.choice([0, 0, 130, rng.integers(0, 300)])) for n in q_lens]
    x = _attn_case(q_lens, lens, 8, 4, "bf16", 16, 615, fp8=fp8)
    ref = _plain_prefill(x, window=100, sinks=3)
    x["max_q"] = 70
    x["lens"][5], x["lens"][41] = -1, 2**31 - 1
    start = np.concatenate([[0], np.cumsum(q_lens)])
    out = torch.full_like(x["q"], 7.0)
    _, flag = _run_prefill(x, out=out, num_splits=1, window=100, sinks=3)
    assert flag == da.FLAG_BAD_SEQ_LEN
    for s in (5, 41):  # bad lengths: zeros
        assert bool((out[start[s]:start[s + 1]] == 0).all())
    assert bool((out[start[40]:start[41]] == 7).all())  # a longer chunk than said: left alone
    for s in (5, 40, 41):
        for a in ref:
            a[start[s]:start[s + 1]] = np.nan
    _close(out, _fp16_probs(ref, "bf16") if fp8 else ref, "bf16")


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_and_cache_write_past_32_bits(fp8):
    """A cache of more than 2^32 elements, used at its far end."""
    h_kv, bs, dtype = 4, 16, "bf16"
    nb = 2**32 // (bs * h_kv * 128) + 64
    kind = torch.uint8 if fp8 else TYPES[dtype]
    caches = [torch.empty((nb, bs, h_kv, 128), dtype=kind, device=DEV) for _ in range(2)]
    scales = [torch.full((h_kv,), 0.25, device=DEV) for _ in range(2)] if fp8 else None
    L = 40
    table = _i32([[nb - 1, nb - 40, nb - 7]])
    t = torch.arange(L, device=DEV)
    slots = (table[0].long()[t // bs] * bs + t % bs).int()
    assert int(slots.max()) * h_kv * 128 > 2**32
    g = _gen(601)
    q, k, v = (torch.randn((L, n, 128), generator=g, device=DEV).to(TYPES[dtype])
               for n in (8, h_kv, h_kv))
    rope = da.rope_table([0.0] * 64)  # no turn: the rows themselves
    fn = da.gqa_rope_append_fp8kv if fp8 else da.gqa_rope_append
    q = fn(q, k, v, *(scales or []), _i32(np.zeros((1, L))), rope, slots, *caches)
    for c, rows in zip(caches, (k, v)):
        got = c.view(-1, h_kv, 128)[slots.long()]
        want = (rows.float() / 0.25).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else rows
        assert torch.equal(got, want)
    small = [c[[nb - 1, nb - 40, nb - 7]].contiguous() for c in caches]
    x = dict(q=q, caches=caches, scales=scales, table=table, start=_i32([0, L]), lens=_i32([L]),
             max_q=L, max_len=L, dtype=dtype)
    y = dict(x, caches=small, table=_i32([[0, 1, 2]]))
    a, fa = _run_prefill(x)
    b, fb = _run_prefill(y)
    assert fa == fb == 0 and torch.equal(a, b)
    dec = da.gqa_decode_fp8kv_sinks if fp8 else da.gqa_decode_sinks
    da_, db = (dec(z["q"][-1:].contiguous(), *z["caches"], *(scales or []), z["table"], z["lens"],
                   scale=0.09, max_seq_len=L, window=9, sinks=3) for z in (x, y))
    assert torch.equal(da_, db)


def test_calls_on_two_streams_at_once():
    """Prefill, rotation, plan and decode calls in flight together give what they
    give alone."""
    cases = [_attn_case([200, 90, 1], [900, 90, 700], 16, 4, "bf16", 16, 610 + i, fp8=i % 2 == 1)
             for i in range(4)]
    alone = [_run_prefill(x, num_splits=2)[0] for x in cases]
    parts, rc, _, slots = _rope_case(700, 8, 2, "bf16", 16, False, 611)
    rope = da.rope_table([1e4 ** (-i / 64) for i in range(64)])
    pos = torch.arange(700, device=DEV, dtype=torch.int32)[None]
    rq = da.gqa_rope_append(*parts, pos, rope, slots, *rc)
    c0 = cases[0]
    decode = lambda: da.gqa_decode_sinks(  # noqa: E731
        c0["q"][:3], *c0["caches"], c0["table"], c0["lens"], scale=0.09, max_seq_len=900,
        window=64, sinks=4)
    dec = decode()
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    outs = []
    for rep in range(5):
        for i, (x, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                fn = da.gqa_prefill if x["scales"] is None else da.gqa_prefill_fp8kv
                outs.append((alone[i], fn(x["q"], *x["caches"], *(x["scales"] or []), x["table"],
                                          x["start"], x["lens"], scale=128 ** -0.5,
                                          max_q_len=x["max_q"], max_seq_len=x["max_len"],
                                          num_splits=2)))
                outs.append((rq, da.gqa_rope_append(*parts, pos, rope, slots,
                                                    *[c.clone() for c in rc])))
                outs.append((dec, decode()))
    torch.cuda.synchronize()
    for want, got in outs:
        assert torch.equal(want, got)


@pytest.mark.parametrize("decode", [False, True])
def test_workspaces_of_calls_on_a_given_stream_stay_theirs(decode):
    """A call on another stream frees its workspace when it returns, long before it
    runs: work on the current stream must not get that memory."""
    x = _attn_case([1, 1, 1], [900, 90, 700], 16, 4, "bf16", 16, 612)

    def call(**kw):
        if decode:
            return da.gqa_decode_sinks(x["q"], *x["caches"], x["table"], x["lens"], scale=0.1,
                                       max_seq_len=900, window=800, sinks=4, num_splits=10, **kw)
        return da.gqa_prefill(x["q"], *x["caches"], x["table"], x["start"], x["lens"], scale=0.1,
                              max_q_len=1, max_seq_len=900, num_splits=7, **kw)

    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # the call runs in some ms
    got = call(stream=s)
    size = max(da.gqa_prefill_workspace_size(3, 16, 7), da.gqa_workspace_size(3, 16, 10))
    spoil = [torch.full((size // 4,), float("nan"), device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(spoil) == 4


def test_a_whole_step_in_one_graph():
    """Plan, rotation with cache write, and 8-bit prefill captured together and
    replayed for several steps equal the same calls made one by one."""
    B, bs, M, T, h_q, h_kv = 3, 16, 30, 64, 8, 2
    rng = np.random.default_rng(12)
    rope = da.rope_table([1e4 ** (-i / 64) for i in range(64)])
    scales = [torch.full((h_kv,), 0.02, device=DEV) for _ in range(2)]

    def state():
        return dict(lens=_i32(np.zeros(B)), new=_i32(np.zeros(B)),
                    table=_i32(np.full((B, M), -1)), free=_i32(np.arange(B * M)),
                    count=_i32([B * M]),
                    caches=[torch.zeros((B * M, bs, h_kv, 128), dtype=torch.uint8, device=DEV)
                            for _ in range(2)],
                    qkv=torch.zeros((T, h_q + 2 * h_kv, 128), dtype=torch.bfloat16, device=DEV),
                    flag=torch.zeros(1, dtype=torch.int32, device=DEV))

    def run(s):
        p = da.paged_plan(s["lens"], s["new"], s["table"], s["free"], s["count"], block_size=bs,
                          max_tokens=T, seq_lens=s["lens"], free_count_out=s["count"],
                          err_flag=s["flag"])
        q, k, v = s["qkv"].split([h_q, h_kv, h_kv], 1)
        q = da.gqa_rope_append_fp8kv(q, k, v, *scales, p.positions[None], rope, p.slots,
                                     *s["caches"], err_flag=s["flag"])
        return da.gqa_prefill_fp8kv(q, *s["caches"], *scales, s["table"], p.q_start, s["lens"],
                                    scale=0.09, max_q_len=T, max_seq_len=M * bs,
                                    err_flag=s["flag"])

    a, b = state(), state()
    run(a)  # (a step of no token)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        out = run(a)
    for seed in range(6):
        new = _i32(rng.integers(1, 21, B))
        for s in (a, b):
            s["new"].copy_(new)
            s["qkv"].copy_(torch.randn(s["qkv"].shape, generator=_gen(seed), device=DEV))
        graph.replay()
        want = run(b)
        torch.cuda.synchronize()
        n = int(new.sum())
        assert int(a["flag"]) == int(b["flag"]) == 0
        assert torch.equal(out[:n], want[:n]) and bool((want[:n] != 0).any())
        for x, y in zip(a["caches"], b["caches"]):
            assert torch.equal(x, y)
        assert torch.equal(a["lens"], b["lens"]) and torch.equal(a["table"], b["table"])


def test_binding_refusals_and_what_it_takes():
    x = _attn_case([1, 1, 1], [30, 50, 64], 8, 2, "bf16", 16, 620)
    args = (x["q"], *x["caches"], x["table"], x["lens"])
    kw = dict(scale=0.09, max_seq_len=64)
    ref = da.gqa_decode(*args, **kw)
    # outputs of another shape with room, a workspace of any type, a flag and
    # lengths in pinned memory
    flat = torch.zeros(4, 8 * 128, dtype=torch.bfloat16, device=DEV)
    got = da.gqa_decode(*args, out=flat, **kw)
    assert got is flat and torch.equal(flat[:3].view_as(ref), ref) and bool((flat[3] == 0).all())
    ws = torch.empty(2**18, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32).pin_memory()
    lens = torch.tensor([30, 50, 65], dtype=torch.int32).pin_memory()
    da.gqa_decode(*args[:4], lens, num_splits=1, workspace=ws, err_flag=flag, **kw)
    torch.cuda.synchronize()
    assert int(flag) == da.FLAG_BAD_SEQ_LEN
    bad = [dict(out=flat[:2]), dict(out=ref.float()), dict(out=ref.cpu()),
           dict(out=torch.zeros(3, 8, 256, dtype=torch.bfloat16, device=DEV)[..., ::2]),
           dict(workspace=ws.cpu()), dict(workspace=3), dict(err_flag=torch.zeros(0, device=DEV)),
           dict(err_flag=torch.zeros(1, dtype=torch.int32)), dict(num_splits=2**40),
           dict(max_seq_len=2**31), dict(scale="x"), dict(stream="x"), dict(num_splits=1.5)]
    for b in bad:
        with pytest.raises((TypeError, ValueError)):
            da.gqa_decode(*args, **{**kw, **b})
        with pytest.raises((TypeError, ValueError)):
            da.gqa_prefill(*args[:4], x["start"], x["lens"], max_q_len=1, **{**kw, **b})
    with pytest.raises(da.DecAttnError):
        da.gqa_prefill(*args[:4], x["start"], x["lens"], max_q_len=1, num_splits=4,
                       workspace=ws[:16], **kw)
    with pytest.raises(ValueError):  # prefill writes rows of its own shape only
        da.gqa_prefill(*args[:4], x["start"], x["lens"], max_q_len=1, out=flat, **kw)
