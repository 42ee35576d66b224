"""Calls of the operators for long caches that their documentation allows, beside those of
test_long_cache_gpu.py, against the same plain forms in 64 bits with the same tolerances."""
import os

import numpy as np
import pytest
import torch

import gqa_mqa_mla_gb300 as da
from gqa_mqa_mla_gb300 import binding, build
from oracle import long_cache

from test_long_cache_gpu import (DEV, _attend, _bounds_of, _case, _close, _decode, _flag,
                                 _gen, _i32, _lists, _np, _same_choice, _values,
                                 _weights_close)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ queries over 8 bits


@pytest.mark.parametrize("kind", ["plain", "sinks", "blocks", "weights"])
@pytest.mark.parametrize("size", [2.0**-40, 2.0**18, 2.0**100])
@pytest.mark.parametrize("heads", [(8, 8), (8, 2), (28, 4), (16, 1), (32, 1)])
def test_bf16_queries_of_any_size_over_8_bits(heads, size, kind):
    """Far below and above fp16's range, heads of a group a factor of 16 apart."""
    x = _case([700, 65, 1], *heads, "bf16", 16, 300, fp8=True)
    x["q"] = x["q"].float() * size
    x["q"][:, 1::2] *= 16
    x["q"] = x["q"].bfloat16()
    scale, flag = 0.02 / size, _flag()
    lists = None
    w = x["weights"].clone()
    if kind == "plain":
        got = da.gqa_decode_fp8kv(x["q"], *x["caches"], *x["scales"], x["table"], x["lens"], scale=scale,
                                  max_seq_len=700, err_flag=flag)
    elif kind == "sinks":  # (a window behind 16 kept tokens: blocks 0 and 40 .. 43 of the longest)
        got = da.gqa_decode_fp8kv_sinks(x["q"], *x["caches"], *x["scales"], x["table"], x["lens"],
                                        scale=scale, max_seq_len=700, window=60, sinks=16, err_flag=flag)
        lists = np.full((3, heads[1], 5), -1)
        lists[0], lists[1, :, :5], lists[2, :, 0] = [0, 40, 41, 42, 43], range(5), 0
    elif kind == "blocks":
        lists = _lists(x, 30, 8, empty=False)
        got = _decode(x, "blocks", x["table"], x["lens"], _i32(lists), scale=scale, err_flag=flag)
    else:
        got = _decode(x, "weights", w, x["table"], x["lens"], scale=scale, err_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == 0
    ref, keys = _attend(x, scale, lists)
    _close(x, got, ref, keys, scale)
    if kind == "weights":
        _weights_close(x, w, x["weights"], ref, keys, scale)


@pytest.mark.parametrize("heads", [(8, 8), (8, 2), (32, 2)])
@pytest.mark.parametrize("kind", ["blocks", "weights"])
def test_strange_queries_over_8_bits_leave_the_other_heads_alone(heads, kind):
    """Zero queries attend to all tokens alike; infinite ones and NaN make their own rows
    NaN (where a score is not -inf); the other heads give the same bytes as without them."""
    x = _case([700, 65, 1], *heads, "bf16", 16, 305, fp8=True)
    lists = _lists(x, 30, 8, empty=False)

    def call():
        if kind == "blocks":
            return _decode(x, "blocks", x["table"], x["lens"], _i32(lists), scale=0.09)
        return _decode(x, "weights", x["weights"].clone(), x["table"], x["lens"], scale=0.09)

    plain = call()
    x["q"][:, 0] = 0
    zero = call()
    x["q"][:, 1, 7], x["q"][:, 2, 9] = float("inf"), float("nan")
    got = call()
    assert torch.equal(got[:, 3:], plain[:, 3:]) and torch.equal(zero[:, 1:], plain[:, 1:])
    assert bool(got[:, 2].isnan().all()) and torch.equal(got[:, 0], zero[:, 0])
    j = 1 // (heads[0] // heads[1])  # (the infinite query's KV head)
    for b, n in enumerate(x["n"]):
        t = [t for t in range(n) if kind != "blocks" or t // 16 in lists[b, j]]
        keys = _values(x)[0][x["table"][b].cpu().numpy()[np.array(t) // 16], np.array(t) % 16, j, 7]
        # (Where every score is -inf the row may be zeros: nothing has weight.)
        assert bool(got[b, 1].isnan().all()) or ((keys < 0).all() and bool((got[b, 1] == 0).all()))
    x["q"][:, 1:3] = 0
    ref, keys = _attend(x, 0.09, lists if kind == "blocks" else None)
    zero[:, 1:3] = torch.tensor(ref[0][:, 1:3], device=DEV).to(zero.dtype)
    _close(x, zero, ref, keys, 0.09)


# ------------------------------------------------------------------ a call that gave up


@pytest.mark.parametrize("limit_us", [200, 2000])
def test_a_split_that_gave_up_is_marked_in_every_row(limit_us):
    """(What the second launch does with such a split is tested with bad block ids, whose
    mark is the same.)"""
    flag, rows = binding.selftest_gave_up(limit_us)
    want = torch.arange(40.0)[:, None].repeat(1, 3)
    want[:, 1] = float("inf")
    assert flag == da.FLAG_TIMEOUT and torch.equal(rows, want)


# ------------------------------------------------------------------ selection: tables


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("first,last", [(2, 4), (0, 6), (6, 0)])
@pytest.mark.parametrize("lens", [[1000, 0, 90, 97, 2000], [70000, 30]])
def test_blocks_that_are_all_taken_always_need_no_scores(lens, first, last, fp8):
    x = _case(lens, 8, 2, "bf16", 16, 320, fp8=fp8)
    bounds = _bounds_of(x)
    need = da.gqa_select_workspace_size(len(lens), 2, x["max_len"], 16, 6)
    ws = torch.full((need,), 77, dtype=torch.uint8, device=DEV)
    _same_choice(x, bounds, count=6, first=first, last=last, workspace=ws)
    assert bool((ws == 77).all())


def test_selection_from_a_bad_table_with_nothing_to_choose():
    """A sequence of no more blocks than are listed: its table is checked as a longer
    one's is."""
    x = _case([400, 60, 80], 8, 2, "bf16", 16, 330)
    bounds = _bounds_of(x)
    for count in (5, 30):
        want = long_cache.select_blocks(_np(x["q"]), _np(bounds), x["table"].cpu().numpy(), x["n"],
                                        block_size=16, count=count, first=1, last=1)
        for at in (-1, bounds.shape[0]):
            table, flag = x["table"].clone(), _flag()
            table[1, 3] = at
            table[2, 6:] = -9  # (past the sequence: not looked at)
            got = da.gqa_select_blocks(x["q"], bounds, table, x["lens"], block_size=16, max_seq_len=400,
                                       count=count, err_flag=flag).cpu().numpy()
            assert int(flag) == da.FLAG_BAD_BLOCK and (got[1] == -1).all()
            assert np.array_equal(got[[0, 2]], want[[0, 2]])


# ------------------------------------------------------------------ the README's step


def _readme():
    """The code of the README's step over long caches, and of the weights and the eviction."""
    with open(os.path.join(build.ROOT, "README.md")) as f:
        text = f.read()
    text = text[text.index("A step over long caches"):text.index("From C:")]
    lines = [line[4:] for line in text.split("\n") if line.startswith("    ") or not line]
    code = "\n".join(lines).strip("\n").split("\n\n")
    return [c for c in code if c.strip()]


def test_the_readme_step_over_long_caches():
    """Run as it stands, over caches, bounds and weights that other sequences have used: after
    an eviction the bounds are those of the rows that are there, new tokens' positions count
    the evicted ones, and weights begin at 0."""
    step, evict = _readme()
    h_q, h_kv, bs, nb, longest, B = 4, 2, 16, 1200, 8400, 2
    g = _gen(380)
    freq = [1e4 ** (-i / 64) for i in range(64)]
    kv = [torch.randn((nb, bs, h_kv, 128), generator=g, device=DEV).bfloat16() for _ in "kv"]
    s = dict(da=da, torch=torch, k_cache=kv[0], v_cache=kv[1], longest=longest,
             rope=da.rope_table(freq), lens=_i32([0] * B), gone=_i32([0] * B), weighed=_i32([0] * B),
             table=_i32(np.full((B, longest // bs), -1)), free=_i32(np.random.default_rng(3).permutation(nb)),
             free_count=_i32([nb]), bounds=torch.randn((nb, 2, h_kv, 128), generator=g, device=DEV).bfloat16() * 9,
             weights=torch.rand((nb, h_kv, bs), generator=g, device=DEV) * 1e3)
    seen, scale = [0] * B, 128 ** -0.5
    for new in ([8300, 900], [1, 1], [3, 7000], [1, 450], [1, 1]):
        T = sum(new) + 5
        raw = [torch.randn((T, h, 128), generator=g, device=DEV).bfloat16() for h in (h_q, h_kv, h_kv)]
        before = s["weights"].clone()
        had = s["lens"].tolist()
        s.update(new=_i32(new), T=T, q=raw[0], k=raw[1], v=raw[2])
        exec(step, s)
        torch.cuda.synchronize()
        seen = [a + b for a, b in zip(seen, new)]
        assert s["lens"].tolist() == [a + b for a, b in zip(had, new)]
        # The newest tokens' queries, turned by all the tokens that their sequences have had.
        at = np.cumsum(new) - 1
        rows = _np(raw[0])[at]
        angle = np.outer([n - 1 for n in seen], freq)[:, None]
        a, b = rows[..., :64], rows[..., 64:]
        want = np.concatenate([a * np.cos(angle) - b * np.sin(angle), a * np.sin(angle) + b * np.cos(angle)], -1)
        # (each result rounded to bf16 once; its products and the sum in fp32)
        far = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
        assert (np.abs(_np(s["newest"]) - want) <= 2.0**-8 * np.abs(want) + 2.0**-21 * far).all()
        # The bounds of every block of the sequences.
        x = dict(q=s["newest"], caches=kv, scales=[], table=s["table"], lens=s["lens"], n=s["lens"].tolist(),
                 bs=bs, h_q=h_q, h_kv=h_kv, dtype="bf16", fp8=False, max_len=longest, weights=before)
        table, now = s["table"].cpu().numpy(), _np(s["bounds"])
        assert np.array_equal(now, long_cache.block_bounds(_np(kv[0]), table, None, x["n"], now))
        want = long_cache.select_blocks(_np(s["newest"]), now, table, x["n"], block_size=bs, count=128,
                                        first=1, last=2)
        assert np.array_equal(s["some"].cpu().numpy(), want)
        ref, keys = _attend(x, scale, want)
        _close(x, s["out"], ref, keys, scale)
        # Weights: those that the sequences' tokens had, 0 for the new ones.
        _decode(x, "weights", before, s["table"], s["lens"], scale=scale, weighed_lens=_i32(had))
        raw = [c.view(torch.int16).cpu().numpy() for c in kv]
        plain = long_cache.evict(*raw, before.cpu().numpy(), table, x["n"], keep=6144, recent=1024, limit=8192)
        exec(evict, s)
        torch.cuda.synchronize()
        ref, keys = _attend(dict(x, caches=[torch.tensor(r, device=DEV).view(torch.bfloat16) for r in raw]), scale)
        _close(x, s["out"], ref, keys, scale)
        assert s["lens"].tolist() == [min(n, 6144) if n > 8192 else n for n in x["n"]]
        for got, ref in zip([*(c.view(torch.int16) for c in kv), s["weights"]], plain):
            assert np.array_equal(got.cpu().numpy(), ref)
    assert s["gone"].tolist()[0] > 0 and s["gone"].tolist()[1] > 0


# ------------------------------------------------------------------ launch shapes


def _far_bound(x, blocks):
    """The case under a bound of `blocks` blocks a sequence."""
    table = torch.full((len(x["n"]), blocks), -1, dtype=torch.int32, device=DEV)
    table[:, : x["table"].shape[1]] = x["table"]
    x.update(table=table, max_len=blocks * x["bs"])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [(64, 8), (32, 8), (28, 4), (8, 8), (18, 6), (7, 7)])
def test_selection_by_ctas_of_several_heads(heads, dtype, fp8):
    """Bounds of far more tiles than the GPU has warps: CTAs take four (of 8 and 4 KV heads),
    two (of 6) or one (of 7) heads' scores."""
    x = _case([3000, 777, 0, 24, 1111], *heads, dtype, 8, 340, fp8=fp8)
    bounds = _bounds_of(x)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    _far_bound(x, 16 * (sms * 32 // (5 * heads[1]) + 2))
    for count, first, last in ((9, 1, 2), (90, 0, 0)):
        _same_choice(x, bounds, count=count, first=first, last=last)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fp8", [False, True])
def test_selection_by_many_ctas_for_one_row(dtype, fp8):
    """One sequence and KV head of 36000 blocks: more CTAs of scores than the choice has
    threads."""
    g = _gen(350)
    n = 36000
    mid = torch.randn((n, 1, 1, 128), generator=g, device=DEV)
    half = torch.rand((n, 1, 1, 128), generator=g, device=DEV) * 2
    bounds = torch.cat([mid - half, mid + half], 1)
    bounds = (bounds * 64).to(torch.float8_e4m3fn) if fp8 else bounds.to(getattr(torch, {"bf16": "bfloat16", "fp16": "float16"}[dtype]))
    table = torch.randperm(n, generator=g, device=DEV).int()[None].contiguous()
    q = torch.randn((1, 3, 128), generator=g, device=DEV).to(getattr(torch, {"bf16": "bfloat16", "fp16": "float16"}[dtype]))
    x = dict(q=q, table=table, lens=_i32([8 * n - 5]), n=[8 * n - 5], bs=8, max_len=8 * n)
    low, high = (_np(bounds[:, k, 0])[table[0].cpu().numpy()] for k in (0, 1))
    score = np.max([np.maximum(row * low, row * high).sum(-1) for row in _np(q)[0]], 0)
    for count in (130, 20000):
        got = da.gqa_select_blocks(q, bounds, table, x["lens"], block_size=8, max_seq_len=8 * n, count=count)
        s = score.copy()
        s[[0, -1]] = np.inf
        assert np.array_equal(got[0, 0].cpu().numpy(), np.sort(np.argsort(-s, kind="stable")[:count]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch", [257, 700])
def test_bounds_of_many_sequences(batch, fp8):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 60, batch).tolist()
    lens[3], lens[255], lens[256] = 200, 0, 33
    x = _case(lens, 2, 2, "bf16", 16, 360, fp8=fp8)
    first = [int(rng.integers(0, n + 2)) for n in lens]
    k = x["caches"][0]
    for f in (None, first):
        bounds, flag = torch.full((k.shape[0], 2, 2, 128), 3.0, device=DEV).to(k.dtype), _flag()
        before = _np(bounds)
        da.gqa_block_bounds(k, x["table"], x["lens"], bounds, max_seq_len=200, err_flag=flag,
                            first_lens=None if f is None else _i32(f))
        torch.cuda.synchronize()
        assert int(flag) == 0
        want = long_cache.block_bounds(_np(k), x["table"].cpu().numpy(), f, lens, before)
        assert np.array_equal(_np(bounds), want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [(2, 2), (8, 2), (34, 2)])
def test_weights_of_one_long_sequence_among_many(heads, fp8):
    """More sequences than the second launch has waves for: its CTAs take several runs of
    the long one's tokens."""
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 4, 400).tolist()
    lens[123] = 9001
    x = _case(lens, *heads, "bf16", 32, 370, fp8=fp8)
    w, flag = x["weights"].clone(), _flag()
    got = _decode(x, "weights", w, x["table"], x["lens"], scale=0.09, err_flag=flag)
    torch.cuda.synchronize()
    assert int(flag) == 0
    ref, keys = _attend(x, 0.09)
    _close(x, got, ref, keys, 0.09)
    _weights_close(x, w, x["weights"], ref, keys, 0.09)
