"""The operators for long caches on the GPU against their plain forms in 64 bits
(oracle/long_cache.py): bounds of blocks, choice of blocks, decode over the chosen
ones, decode that weighs tokens, eviction, and a run of them together.

Bounds, chosen blocks and evictions are exact.  Attention outputs, per element
(u = half a step of the 16-bit type, relative): the output's own rounding u |out|;
the probabilities' rounding u sum p |v| / sum p =: u A; a score error of D = 130
2^-24 |scale| sum |q| |k| (fp32 sums of 128 products, two more roundings) changes p
and the sum by D each, 2 D A; 2^-19 A for exp2, the sums and the division in fp32;
and for fp16 probabilities (an 8-bit cache's too) what falls below half of their
smallest step, 2^-25 sum |v| / sum e^(s - max).  From 17 heads a KV head on, a query
over an 8-bit cache is written in e4m3 terms that lose at most 2^-10 / 224 of its
largest value: D grows by that times |scale| sum |k|.

A weight p = 2^(s - lse), relative: 2 D (the score, and the sum); the base-two
logarithm of the sum, 2^-22, and twice the rounding of lse (one more where splits
are merged), 2^-24 (|s| + log2 n + 1) each, and that of s - lse, all times ln 2; two
steps of exp2 (2^-22); together 2 D + 2^-20 + 3 2^-24 (reach log2 e + log2 n + 1).
The sum of G heads and the old weight adds (G + 1) 2^-24 of the total."""
import threading

import numpy as np
import pytest
import torch

import gqa_mqa_mla_gb300 as da
from oracle import long_cache

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"bf16": 2.0**-8, "fp16": 2.0**-11}


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _flag():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _np(t):
    """float64 (codes: the values they stand for)."""
    return t.double().cpu().numpy()


def _bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def _case(lens, h_q, h_kv, dtype, bs, seed, fp8=False, spare=3, most=None):
    """Caches whose slots past the sequences are NaN, q, table, lengths, scales."""
    g = _gen(seed)
    need = [-(-n // bs) for n in lens]
    most = most or max(1, max(need))
    nb = sum(need) + spare
    ids = np.random.default_rng(seed).permutation(nb)
    table = np.full((len(lens), most), -1)
    used = np.zeros((nb, bs), bool)
    at = 0
    for b, n in enumerate(lens):
        table[b, : need[b]] = ids[at:at + need[b]]
        for t in range(n):
            used[table[b, t // bs], t % bs] = True
        at += need[b]
    gone = torch.tensor(~used, device=DEV)[:, :, None, None]
    caches, scales = [], []
    for k in range(2):
        x = torch.randn((nb, bs, h_kv, 128), generator=g, device=DEV)
        if k == 0:
            x += 0.5 * torch.randn((h_kv, 128), generator=g, device=DEV)
        x = x.masked_fill(gone, float("nan"))
        caches.append((x * 64).to(torch.float8_e4m3fn) if fp8 else x.to(TYPES[dtype]))
        if fp8:
            scales.append((torch.rand(h_kv, generator=g, device=DEV) + 0.5) / 64)
    return dict(q=torch.randn((len(lens), h_q, 128), generator=g, device=DEV).to(TYPES[dtype]),
                caches=caches, scales=scales, table=_i32(table), lens=_i32(lens), n=list(lens),
                max_len=max(lens), bs=bs, h_q=h_q, h_kv=h_kv, dtype=dtype, fp8=fp8,
                weights=torch.rand((nb, h_kv, bs), generator=g, device=DEV) * 4)


def _values(x):
    """The caches in 64 bits."""
    return [_np(c) * (s.double().cpu().numpy()[:, None] if x["fp8"] else 1.0)
            for c, s in zip(x["caches"], x["scales"] or [None, None])]


def _attend(x, scale, selected=None):
    k, v = _values(x)
    return long_cache.attend(_np(x["q"]), k, v, x["table"].cpu().numpy(), x["n"], scale=scale,
                             selected=selected), k


def _errors(x, ref, keys, scale):
    """2 D per row and head."""
    d = 130 * 2.0**-24 * ref[3]
    if x["fp8"] and x["h_q"] // x["h_kv"] > 16:
        far = np.nansum(np.abs(keys), -1).max()
        d = d + 2.0**-10 / 224 * np.abs(_np(x["q"])).max(-1) * abs(scale) * far
    return 2 * d


def _close(x, got, ref, keys, scale):
    out, spread, tiny = ref[:3]
    u = HALF[x["dtype"]]
    tol = u * np.abs(out) + (u + 2.0**-19 + _errors(x, ref, keys, scale)[..., None]) * spread
    if x["dtype"] == "fp16" or x["fp8"]:
        tol = tol + 2.0**-25 * tiny
    err = np.abs(_np(got) - out)
    assert np.isfinite(_np(got)).all()
    assert (err <= tol + 1e-30).all(), (float(err.max()), float((err / (tol + 1e-30)).max()))


def _decode(x, kind, *more, **kw):
    """gqa_decode_<kind> or its 8-bit form."""
    fn = getattr(da, ("gqa_decode_fp8kv_" if x["fp8"] else "gqa_decode_") + kind)
    return fn(x["q"], *x["caches"], *x["scales"], *more, max_seq_len=kw.pop("most", x["max_len"]),
              **kw)


HEADS = [(8, 8), (8, 2), (28, 4), (32, 2), (9, 1), (32, 1), (64, 1)]


# ------------------------------------------------------------------ bounds


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype,bs,h_kv,lens,first", [
    ("bf16", 16, 2, [1, 0, 40, 64, 65], None), ("fp16", 8, 3, [7, 8, 9, 100], None),
    ("bf16", 256, 1, [1, 255, 256, 700], None), ("bf16", 64, 5, [130, 1, 64], [129, 0, 63]),
    ("fp16", 32, 8, [500, 33, 32, 31], [400, 33, 40, 0]), ("bf16", 128, 32, [300], [299]),
    ("fp16", 16, 1, [5000, 3], [0, 2]),
])
def test_bounds(dtype, bs, h_kv, lens, first, fp8):
    x = _case(lens, h_kv, h_kv, dtype, bs, 1 + bs, fp8=fp8)
    k = x["caches"][0]
    before = torch.full((k.shape[0], 2, h_kv, 128), 7.0, device=DEV).to(k.dtype)
    bounds, flag = before.clone(), _flag()
    got = da.gqa_block_bounds(k, x["table"], x["lens"], bounds, max_seq_len=x["max_len"],
                              first_lens=None if first is None else _i32(first), err_flag=flag)
    torch.cuda.synchronize()
    want = long_cache.block_bounds(_np(k), x["table"].cpu().numpy(), first, lens, _np(before))
    assert got.data_ptr() == bounds.data_ptr() and int(flag) == 0
    assert np.array_equal(_np(bounds), want)


@pytest.mark.parametrize("fp8", [False, True])
def test_bounds_of_values_that_are_not_finite(fp8):
    """NaN of either sign makes both bounds of its dimension NaN; infinities and zeros
    of either sign are values.  uint8 codes give the same bytes as float8."""
    x = _case([40, 16], 2, 2, "fp16", 16, 3, fp8=fp8)
    k = x["caches"][0]
    raw = k.view(torch.uint8 if fp8 else torch.int16)
    t = x["table"].cpu().numpy()
    nan = [0x7F, 0xFF] if fp8 else [0x7E00, -0x200]
    raw[t[0, 0], 3, 0, 5], raw[t[0, 1], 15, 1, 6] = nan
    raw[t[0, 2], 0, 0, :4] = torch.tensor([0x00, 0x80, 0x7E, 0xFE] if fp8 else [0, -0x8000, 0x7C00, -0x400],
                                          dtype=raw.dtype, device=DEV)
    bounds = torch.zeros((k.shape[0], 2, 2, 128), device=DEV).to(k.dtype)
    da.gqa_block_bounds(k, x["table"], x["lens"], bounds, max_seq_len=40)
    want = long_cache.block_bounds(_np(k), t, None, x["n"], np.zeros(bounds.shape))
    assert np.isnan(want).sum() == 4 and np.array_equal(_np(bounds), want, equal_nan=True)
    if fp8:
        again = torch.zeros(bounds.shape, dtype=torch.uint8, device=DEV)
        da.gqa_block_bounds(raw, x["table"], x["lens"], again, max_seq_len=40)
        assert torch.equal(again, bounds.view(torch.uint8))


def test_bounds_leave_bad_sequences_out():
    x = _case([40, 40, 40, 33], 2, 2, "bf16", 16, 4)
    k = x["caches"][0]
    for lens, first, table, flag_is, done in [
        ([40, 41, 40, 33], None, None, da.FLAG_BAD_SEQ_LEN, [0, 2, 3]),
        ([40, -1, 40, 33], None, None, da.FLAG_BAD_SEQ_LEN, [0, 2, 3]),
        ([40, 40, 40, 33], [0, -1, 0, 0], None, da.FLAG_BAD_SEQ_LEN, [0, 2, 3]),
        ([40, 40, 40, 33], None, (1, 1, k.shape[0]), da.FLAG_BAD_BLOCK, None),
        ([40, 40, 40, 33], None, (1, 1, -2), da.FLAG_BAD_BLOCK, None),
    ]:
        t = x["table"].clone()
        if table:
            t[table[0], table[1]] = table[2]
        flag = _flag()
        bounds = torch.full((k.shape[0], 2, 2, 128), 3.0, device=DEV).bfloat16()
        da.gqa_block_bounds(k, t, _i32(lens), bounds, max_seq_len=40, err_flag=flag,
                            first_lens=None if first is None else _i32(first))
        torch.cuda.synchronize()
        assert int(flag) == flag_is
        tn = x["table"].cpu().numpy()
        some = [(b, c) for b in range(4) for c in range(3)]
        some = [(b, c) for b, c in some if (b in done if done else (b, c) != (1, 1))]
        want = np.full(bounds.shape, 3.0)
        for b, c in some:
            keys = _np(k)[tn[b, c], : min(16, x["n"][b] - 16 * c)]
            want[tn[b, c], 0], want[tn[b, c], 1] = keys.min(0), keys.max(0)
        assert np.array_equal(_np(bounds), want)


# ------------------------------------------------------------------ selection


def _bounds_of(x):
    k = x["caches"][0]
    bounds = torch.zeros((k.shape[0], 2, x["h_kv"], 128), device=DEV).to(k.dtype)
    return da.gqa_block_bounds(k, x["table"], x["lens"], bounds, max_seq_len=x["max_len"])


def _same_choice(x, bounds, q=None, **kw):
    q = x["q"] if q is None else q
    flag = _flag()
    got = da.gqa_select_blocks(q, bounds, x["table"], x["lens"], block_size=x["bs"],
                               max_seq_len=x["max_len"], err_flag=flag, **kw)
    torch.cuda.synchronize()
    want = long_cache.select_blocks(_np(q), _np(bounds), x["table"].cpu().numpy(), x["n"],
                                    block_size=x["bs"], count=kw["count"],
                                    first=kw.get("first", 1), last=kw.get("last", 1))
    assert int(flag) == 0
    assert np.array_equal(got.cpu().numpy(), want), (got.cpu().numpy(), want)
    return got


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype,bs,lens,count,first,last", [
    ("bf16", 16, [1000, 0, 1, 63, 64, 700], 5, 1, 1), ("fp16", 8, [777, 640, 80], 10, 0, 0),
    ("bf16", 32, [1500, 40], 4, 2, 2), ("fp16", 64, [2000, 3000], 17, 0, 3),
    ("bf16", 256, [5000], 3, 1, 0), ("bf16", 8, [300, 24], 1, 0, 0),
])
def test_selection(heads, dtype, bs, lens, count, first, last, fp8):
    x = _case(lens, *heads, dtype, bs, 11 + count, fp8=fp8)
    _same_choice(x, _bounds_of(x), count=count, first=first, last=last)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_selection_from_many_blocks(dtype, fp8):
    """Thousands of blocks whose scores lie close together."""
    x = _case([24000, 20001], 8, 2, dtype, 8, 5, fp8=fp8)
    bounds = _bounds_of(x)
    for count in (7, 500, 2400):
        _same_choice(x, bounds, count=count)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("alike", [3, 40, 400])
def test_selection_of_equal_blocks_takes_the_earliest(alike, fp8):
    """Blocks with the same bounds: `alike` of them around the cut (more than a warp
    orders, and all)."""
    x = _case([3200], 8, 2, "bf16", 8, 6, fp8=fp8)
    bounds = _bounds_of(x)
    t = x["table"][0].long()
    at = torch.arange(0, 400, 400 // alike, device=DEV)[:alike]
    view = bounds.view(torch.uint8) if fp8 else bounds
    view[t[at]] = view[t[at[0]]].clone()
    for count in (3, 20, 200, 399):
        _same_choice(x, bounds, count=count)
    view.zero_()
    _same_choice(x, bounds, count=50)
    _same_choice(x, bounds, count=50, first=0, last=0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("blocks", [500, 5000, 41000, 330000])
def test_selection_among_repeated_blocks(blocks, fp8):
    """Long tables (one CTA, a cluster, slices past a CTA's and a cluster's shared memory)
    over few distinct blocks, so that every cut falls among equals."""
    g, rng = _gen(blocks), np.random.default_rng(blocks)
    q = torch.randn((2, 4, 128), generator=g, device=DEV).bfloat16()
    lo, hi = -torch.rand((50, 1, 2, 128), generator=g, device=DEV), torch.rand((50, 1, 2, 128), generator=g, device=DEV)
    bounds = (torch.cat([lo, hi], 1) * 4).to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
    table = rng.integers(0, 50, (2, blocks))
    lens = [8 * blocks - 3, 8 * (blocks // 2)]
    for count, first, last in ((7, 1, 1), (blocks // 3, 0, 2), (blocks // 2 + 5, 1, 0)):
        got = da.gqa_select_blocks(q, bounds, _i32(table), _i32(lens), block_size=8, count=count,
                                   max_seq_len=8 * blocks, first=first, last=last).cpu().numpy()
        for b, n in enumerate((blocks, blocks // 2)):
            for j in range(2):
                if n <= count:
                    want = np.concatenate([np.arange(n), np.full(count - n, -1)])
                else:
                    s = np.array([long_cache.block_score(_np(q)[b, 2 * j:2 * j + 2], *_np(bounds)[i, :, j])
                                  for i in range(50)])[table[b, :n]]
                    s[:first], s[n - last:] = np.inf, np.inf
                    want = np.sort(np.argsort(-s, kind="stable")[:count])
                assert np.array_equal(got[b, j], want)


@pytest.mark.parametrize("fp8", [False, True])
def test_selection_of_nearly_equal_blocks(fp8):
    """Scores that differ by less than 32 bits hold: one large product and a small
    one that only 64 bits tell apart."""
    x = _case([1600], 2, 1, "bf16", 8, 7, fp8=fp8)
    n = 200
    bounds = torch.zeros((x["caches"][0].shape[0], 2, 1, 128), device=DEV)
    t = x["table"][0].long()
    rng = np.random.default_rng(0)
    bounds[:, :, 0, 0] = 256.0
    small = torch.tensor(rng.permutation(n) // 2, dtype=torch.float32, device=DEV)  # pairs of equals
    bounds[t, :, 0, 1] = ((small % 16 + 16) * 2.0 ** (torch.div(small, 16, rounding_mode="floor") - 8))[:, None]
    b = bounds.to(x["caches"][0].dtype)
    q = torch.zeros_like(x["q"])
    q[:, :, 0], q[:, :, 1] = 256.0, 2.0**-12
    for count in (3, 60, 111, 150):
        _same_choice(x, b, q=q, count=count)


@pytest.mark.parametrize("lens", [[1600], [40000]])  # (one CTA, a cluster)
@pytest.mark.parametrize("step", [2.0**-5, 2.0**-12, 0.0])
@pytest.mark.parametrize("alike", [2, 9, 32])
def test_selection_where_a_few_are_nearly_equal(alike, step, lens):
    """`alike` blocks around the cut, the others surely in or out.  Their scores are 2^16
    plus whole steps, in pairs: within the products' common error (2^-16 of 256 x 512);
    steps of 2^-5 are told apart by a 32-bit sum with its own error (11 x 2^-24 of 2^16)
    from the third on, those of 2^-12 in 64 bits only; equals go by their places."""
    x = _case(lens, 2, 1, "bf16", 8, 9)
    n = lens[0] // 8
    rng = np.random.default_rng(alike)
    order = rng.permutation(n)
    above, close = order[: n // 3], np.sort(order[n // 3 : n // 3 + alike])
    small = np.zeros(n)
    large = np.full(n, 128.0)
    large[above] = 512.0
    large[close] = 256.0
    small[close] = rng.permutation(alike) // 2 * 1.0  # (pairs of equals)
    bounds = torch.zeros((x["caches"][0].shape[0], 2, 1, 128), device=DEV)
    t = x["table"][0].long()
    bounds[t, :, 0, 0] = torch.tensor(large, dtype=torch.float32, device=DEV)[:, None]
    bounds[t, :, 0, 1] = torch.tensor(small, dtype=torch.float32, device=DEV)[:, None]
    q = torch.zeros_like(x["q"])
    q[:, 0, 0], q[:, 0, 1] = 256.0, step
    q[:, 1, 0], q[:, 1, 2] = 128.0, 1.0
    for k in sorted({1, alike // 2, alike - 1}):
        _same_choice(x, bounds.bfloat16(), q=q, count=n // 3 + k, first=0, last=0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fp8", [False, True])
def test_selection_by_values_that_are_not_finite(fp8, dtype):
    """NaN and infinities in bounds and queries; sums past 32 bits' range or below its
    normal one; NaN is +inf."""
    for seed, what in enumerate(["nan", "inf", "-inf", "q nan", "q inf", "huge", "tiny", "smallest"]):
        x = _case([800, 640], 8, 2, dtype, 16, 20 + seed, fp8=fp8)
        bounds, q = _bounds_of(x), x["q"].clone()
        t = x["table"].cpu().numpy()
        view = bounds.view(torch.uint8) if fp8 else bounds
        if what in ("huge", "tiny", "smallest") and dtype == "fp16":
            q *= {"huge": 1e4, "tiny": 2.0**-14, "smallest": 2.0**-20}[what]
            if what == "smallest" and not fp8:
                bounds *= 2.0**-16
        elif what == "nan":
            view[int(t[0, 7]), :, 0, 3] = 0x7F if fp8 else float("nan")
            view[int(t[1, 9]), 0, 1, 3] = 0xFF if fp8 else float("nan")
        elif what in ("inf", "-inf") and not fp8:
            for c in (3, 11, 12, 13):
                bounds[int(t[0, c]), 1 if what == "inf" else 0, :, c] = float(what)
        elif what == "q nan":
            q[0, 1, 5] = float("nan")
        elif what == "q inf":
            q[0, 1, 5], q[1, 7, 0] = float("inf"), -float("inf")
        elif what == "huge":
            q *= 1e37
        elif what == "tiny":
            q *= 2.0**-120
        elif what == "smallest":  # products below 32 bits' normal range
            q *= 2.0**-124
            if not fp8:
                bounds *= 2.0**-14
        with np.errstate(over="ignore", invalid="ignore"):
            _same_choice(x, bounds, q=q, count=6)


def test_selection_flags():
    x = _case([400, 300, 350], 8, 2, "bf16", 16, 30)
    bounds = _bounds_of(x)
    for lens, at, flag_is in [([400, 401, 350], None, da.FLAG_BAD_SEQ_LEN),
                              ([400, -3, 350], None, da.FLAG_BAD_SEQ_LEN),
                              ([400, 300, 350], -1, da.FLAG_BAD_BLOCK),
                              ([400, 300, 350], bounds.shape[0], da.FLAG_BAD_BLOCK)]:
        table, flag = x["table"].clone(), _flag()
        if at is not None:
            table[1, 4] = at
        got = da.gqa_select_blocks(x["q"], bounds, table, _i32(lens), block_size=16, max_seq_len=400,
                                   count=5, err_flag=flag).cpu().numpy()
        assert int(flag) == flag_is and (got[1] == -1).all()
        want = long_cache.select_blocks(_np(x["q"]), _np(bounds), x["table"].cpu().numpy(), x["n"],
                                        block_size=16, count=5, first=1, last=1)
        assert np.array_equal(got[[0, 2]], want[[0, 2]])


def test_selection_workspace_and_out():
    x = _case([400, 300], 8, 2, "fp16", 16, 31)
    bounds = _bounds_of(x)
    need = da.gqa_select_workspace_size(2, 2, 400, 16, 5)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    out = torch.full((2, 2, 5), 9, dtype=torch.int32, device=DEV)
    a = (x["q"], bounds, x["table"], x["lens"])
    kw = dict(block_size=16, max_seq_len=400, count=5)
    got = da.gqa_select_blocks(*a, workspace=ws, out=out, **kw)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, da.gqa_select_blocks(*a, **kw))
    with pytest.raises(da.DecAttnError, match="workspace"):
        da.gqa_select_blocks(*a, workspace=ws[:-1], **kw)
    assert da.gqa_select_workspace_size(2, 2, 400, 16, 25) == 0
    got = da.gqa_select_blocks(*a, block_size=16, max_seq_len=400, count=25)
    assert got[0, 0].tolist() == list(range(25)) and got[1, 1, 18:].tolist() == [18] + [-1] * 6


# ------------------------------------------------------------------ decode over blocks


def _lists(x, count, seed, empty=True):
    """Some ascending blocks for each sequence and KV head; one list is empty."""
    rng = np.random.default_rng(seed)
    out = np.full((len(x["n"]), x["h_kv"], count), -1)
    for b, n in enumerate(x["n"]):
        blocks = -(-n // x["bs"])
        for j in range(x["h_kv"]):
            k = min(count, int(rng.integers(0 if empty else 1, blocks + 1))) if blocks else 0
            out[b, j, :k] = np.sort(rng.permutation(blocks)[:k])
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("splits", [1, 0, 3, 9])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype,bs,lens,count", [
    ("bf16", 16, [1000, 0, 1, 63, 64, 700], 37), ("fp16", 8, [333, 80, 9], 41),
    ("bf16", 256, [2000, 255, 256], 4), ("fp16", 64, [1300, 65], 12), ("bf16", 32, [64], 1),
    ("bf16", 128, [900, 129], 9),
])
def test_decode_over_blocks(heads, dtype, bs, lens, count, splits, fp8):
    x = _case(lens, *heads, dtype, bs, 40 + count, fp8=fp8)
    lists = _lists(x, count, count)
    table = x["table"].clone()  # blocks that no head lists may be gone
    for b, n in enumerate(lens):
        for t in range(-(-n // bs)):
            if not (lists[b] == t).any():
                table[b, t] = -5
    flag = _flag()
    got = _decode(x, "blocks", table, x["lens"], _i32(lists), scale=0.09, num_splits=splits,
                  err_flag=flag)
    torch.cuda.synchronize()
    ref, keys = _attend(x, 0.09, lists)
    assert int(flag) == 0
    _close(x, got, ref, keys, 0.09)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [(8, 8), (8, 2), (32, 2), (32, 1)])
def test_all_blocks_listed_is_plain_decode(heads, fp8):
    """The same bytes as gqa_decode with the same splits, a long list included (MHA over
    an 8-bit cache, which another consumer takes: attention over the same tokens)."""
    x = _case([5000, 3000, 17], *heads, "bf16", 8, 50, fp8=fp8)
    every = np.full((3, heads[1], 700), -1)
    for b, n in enumerate(x["n"]):
        every[b, :, : -(-n // 8)] = np.arange(-(-n // 8))
    plain = da.gqa_decode_fp8kv if fp8 else da.gqa_decode
    for splits in (1, 9, 20):
        want = plain(x["q"], *x["caches"], *x["scales"], x["table"], x["lens"], scale=0.1,
                     max_seq_len=5000, num_splits=splits)
        got = _decode(x, "blocks", x["table"], x["lens"], _i32(every), scale=0.1, num_splits=splits)
        if fp8 and heads == (8, 8):
            ref, keys = _attend(x, 0.1)
            _close(x, got, ref, keys, 0.1)
        else:
            assert torch.equal(got, want)


@pytest.mark.parametrize("heads", [(8, 8), (8, 2), (32, 1)])
@pytest.mark.parametrize("splits", [1, 2, 10])
def test_lists_that_are_wrong(heads, splits):
    """A block twice, in the wrong order, past the sequence, behind the end of the list,
    and a bad block id: that head's rows are zeros, the others as they were."""
    h_q, h_kv = heads
    x = _case([500, 400], h_q, h_kv, "bf16", 16, 60)
    good = np.full((2, h_kv, 50), -1)
    good[0, :, :30], good[1, :, :25] = np.arange(30), np.arange(25)
    ref, keys = _attend(x, 0.1, good)
    g, j = h_q // h_kv, h_kv - 1
    for wrong in ("twice", "order", "past", "behind", "id"):
        lists, table = good.copy(), x["table"].clone()
        if wrong == "twice":
            lists[0, j, 7] = 6
        elif wrong == "order":
            lists[0, j, 7] = 2
        elif wrong == "past":
            lists[0, j, 30] = 32
        elif wrong == "behind":
            lists[0, j, 40] = 31
        else:
            table[0, 12] = x["caches"][0].shape[0]
            lists[0, :j, 12:] = -1
        flag = _flag()
        got = _decode(x, "blocks", table, x["lens"], _i32(lists), scale=0.1, num_splits=splits,
                      err_flag=flag)
        torch.cuda.synchronize()
        assert int(flag) == da.FLAG_BAD_BLOCK, wrong
        assert bool((got[0, j * g:] == 0).all()) and bool((got[1] != 0).any()), wrong
        if wrong != "id":
            keep = got.clone()
            keep[0, j * g:] = torch.tensor(ref[0][0, j * g:], device=DEV).to(keep.dtype)
            _close(x, keep, ref, keys, 0.1)
    flag = _flag()
    got = _decode(x, "blocks", x["table"], _i32([501, 400]), _i32(good), scale=0.1, err_flag=flag,
                  num_splits=splits)
    torch.cuda.synchronize()
    assert int(flag) == da.FLAG_BAD_SEQ_LEN and bool((got[0] == 0).all())


# ------------------------------------------------------------------ weights


def _weigh(x, p, before, weighed=None, decay=1.0):
    return long_cache.add_weights(before, p, x["table"].cpu().numpy(), x["n"], weighed,
                                  decay=decay)


def _weights_close(x, got, before, ref, keys, scale, weighed=None, decay=1.0):
    g = x["h_q"] // x["h_kv"]
    want = _weigh(x, ref[4], _np(before), weighed, decay)
    rel = _errors(x, ref, keys, scale) + 2.0**-20 + 3 * 2.0**-24 * (
        1.4427 * ref[3] + np.log2(np.maximum(1, x["n"]))[:, None] + 1)
    tol = _weigh(x, [p * r[:, None] for p, r in zip(ref[4], rel)], np.zeros(tuple(before.shape)))
    tol = tol + (g + 1) * 2.0**-24 * np.abs(want) + g * 2.0**-125
    t = x["table"].cpu().numpy()
    live = np.zeros(tuple(before.shape), bool)
    for b, n in enumerate(x["n"]):
        for c in range(-(-n // x["bs"])):
            live[t[b, c], :, : n - c * x["bs"]] = True
    err = np.abs(_np(got) - want)
    assert (err[live] <= tol[live]).all(), float((err[live] / tol[live]).max())
    assert np.array_equal(_np(got)[~live], _np(before)[~live], equal_nan=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("splits", [1, 0, 5])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype,bs,lens", [
    ("bf16", 16, [1000, 0, 1, 63, 64, 700]), ("fp16", 8, [333, 80, 9]),
    ("bf16", 256, [2000, 255, 257]), ("fp16", 64, [1300, 65]), ("bf16", 32, [5]),
])
def test_decode_with_weights(heads, dtype, bs, lens, splits, fp8):
    x = _case(lens, *heads, dtype, bs, 70 + bs, fp8=fp8)
    before, flag = x["weights"].clone(), _flag()
    for b, n in enumerate(lens):  # the newest token's slot holds what it held before
        if n:
            before[int(x["table"][b, (n - 1) // bs]), :, (n - 1) % bs] = float("nan")
    w = before.clone()
    got = _decode(x, "weights", w, x["table"], x["lens"], scale=0.09, num_splits=splits,
                  err_flag=flag)
    torch.cuda.synchronize()
    ref, keys = _attend(x, 0.09)
    assert int(flag) == 0
    _close(x, got, ref, keys, 0.09)
    _weights_close(x, w, before, ref, keys, 0.09)


@pytest.mark.parametrize("heads", [(8, 8), (8, 2), (32, 1)])
@pytest.mark.parametrize("fp8", [False, True])
def test_weights_decay_and_new_tokens(heads, fp8):
    x = _case([300, 200, 100], *heads, "bf16", 16, 90, fp8=fp8)
    ref, keys = _attend(x, 0.1)
    for weighed, decay in [([0, 150, 100], 1.0), ([-5, 1 << 30, 7], 0.5), (None, 0.0)]:
        before = x["weights"].clone()
        w = before.clone()
        _decode(x, "weights", w, x["table"], x["lens"], scale=0.1, decay=decay,
                weighed_lens=None if weighed is None else _i32(weighed))
        _weights_close(x, w, before, ref, keys, 0.1, weighed, decay)


@pytest.mark.parametrize("heads", [(8, 8), (8, 2), (32, 1)])
@pytest.mark.parametrize("splits", [1, 3])
def test_weights_output_is_plain_decode(heads, splits):
    x = _case([1000, 321, 64], *heads, "bf16", 16, 91)
    want = da.gqa_decode(x["q"], *x["caches"], x["table"], x["lens"], scale=0.1, max_seq_len=1000,
                         num_splits=splits)
    w = x["weights"].clone()
    assert torch.equal(_decode(x, "weights", w, x["table"], x["lens"], scale=0.1,
                               num_splits=splits), want)
    again = x["weights"].clone()  # the order of the sums is always the same
    _decode(x, "weights", again, x["table"], x["lens"], scale=0.1, num_splits=splits)
    assert torch.equal(again, w)


@pytest.mark.parametrize("heads", [(8, 8), (8, 2), (32, 1)])
@pytest.mark.parametrize("splits", [1, 3])
def test_weights_of_rows_that_are_not_numbers(heads, splits):
    """A NaN query: its KV head's weights are NaN.  Scores of -inf alone: zero rows that
    add nothing.  Bad data: weights as they were."""
    h_q, h_kv = heads
    x = _case([300, 200, 260], h_q, h_kv, "bf16", 16, 92)
    x["q"][0, 0, 3] = float("nan")
    t = x["table"].cpu().numpy()
    for c in range(13):
        x["caches"][0][int(t[1, c]), :, :, 0] = -float("inf")
    x["q"][1, :, 0] = x["q"][1, :, 0].abs() + 1
    for bad_id, lens, flag_is in [(None, [300, 200, -1], da.FLAG_BAD_SEQ_LEN),
                                  (-3, [300, 200, 260], da.FLAG_BAD_BLOCK)]:
        table = x["table"].clone()
        if bad_id is not None:
            table[2, 9] = bad_id
        w, flag = x["weights"].clone(), _flag()
        got = _decode(x, "weights", w, table, _i32(lens), scale=0.1, num_splits=splits,
                      err_flag=flag)
        torch.cuda.synchronize()
        assert int(flag) == flag_is
        assert bool(got[0, 0].isnan().all()) and bool((got[1:] == 0).all())
        ids = torch.tensor(t[0, :19], device=DEV).long()
        assert bool(w[ids, 0].flatten()[:300].isnan().all())
        ids = torch.tensor(t[1, :13], device=DEV).long()
        a, b = (v[ids].permute(1, 0, 2).reshape(h_kv, -1) for v in (w, x["weights"]))
        assert torch.equal(a[:, :199], b[:, :199]) and bool((a[:, 199] == 0).all())
        ids = torch.tensor(t[2, :17], device=DEV).long()
        assert torch.equal(w[ids], x["weights"][ids])


# ------------------------------------------------------------------ eviction


def _evict(x, **kw):
    k, v, w = x["caches"][0].clone(), x["caches"][1].clone(), x["weights"].clone()
    flag = _flag()
    e = da.gqa_kv_evict(k, v, w, kw.pop("table", x["table"]), kw.pop("lens", x["lens"]),
                        max_seq_len=kw.pop("most", x["max_len"]), err_flag=flag, **kw)
    torch.cuda.synchronize()
    return k, v, w, e, int(flag)


def _same_eviction(x, keep, recent, limit, **kw):
    k, v, w, e, flag = _evict(x, keep=keep, recent=recent, limit=limit, **kw)
    raw = [c.view(torch.uint8 if x["fp8"] else torch.int16).cpu().numpy() for c in x["caches"]]
    bits = x["weights"].cpu().numpy()
    want = long_cache.evict(*raw, bits, x["table"].cpu().numpy(), x["n"], keep=keep, recent=recent,
                            limit=limit)
    assert flag == 0
    assert np.array_equal(e.kept.cpu().numpy(), want[4])
    assert e.new_lens.tolist() == want[3].tolist()
    for got, ref in zip((k, v), want):
        assert np.array_equal(got.view(torch.uint8 if x["fp8"] else torch.int16).cpu().numpy(), ref)
    assert np.array_equal(w.view(torch.int32).cpu().numpy(), want[2].view(np.int32))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs,h_kv,lens,keep,recent,limit", [
    (16, 2, [300, 0, 1, 100, 101, 99], 100, 20, 100), (8, 3, [77, 200], 33, 33, 40),
    (256, 1, [1000, 256, 257], 250, 0, 256), (64, 8, [129, 500], 128, 1, 128),
    (32, 5, [40, 90], 1, 0, 1), (32, 5, [40, 90], 1, 1, 60), (16, 32, [2000], 1111, 10, 1500),
    (128, 2, [5000, 4000], 3999, 100, 3999),
])
def test_eviction(bs, h_kv, lens, keep, recent, limit, fp8):
    x = _case(lens, h_kv, h_kv, "bf16", bs, 100 + bs, fp8=fp8)
    x["weights"].copy_((x["weights"] * 3).exp())
    _same_eviction(x, keep, recent, limit)


def test_eviction_by_equal_and_strange_weights():
    """Equal weights go by position; -0 is 0; NaN, infinities and negative weights."""
    x = _case([900, 700], 2, 2, "fp16", 16, 130)
    plain = x["weights"].clone()
    for what in ("zero", "few", "strange"):
        w = x["weights"]
        if what == "zero":
            w.zero_()
            w[::2] = -0.0
        elif what == "few":
            w.copy_((plain * 2).floor())
        else:
            w.copy_(plain - 2)
            for k, v in enumerate([float("nan"), -float("nan"), float("inf"), -float("inf"), 0.0, -0.0]):
                w[k::9, :, k] = v
        for keep, recent in ((300, 50), (600, 0), (2, 1)):
            _same_eviction(x, keep, recent, keep)


@pytest.mark.parametrize("batch", [1, 40])
def test_eviction_from_long_sequences(batch):
    """More tokens than the weights that a CTA's shared memory holds: a cluster's, with
    few and with many sequences; and, by the host's bound, one CTA without."""
    x = _case([60000, 300, 5][:min(3, batch)] + [5] * (batch - 3), 2, 2, "bf16", 64, 131, fp8=True,
              most=6720)
    x["weights"].copy_((x["weights"] * 8).floor())
    for most in (60000, 430000):
        _same_eviction(x, 2500, 100, 2500, most=most)
        _same_eviction(x, 55000, 0, 55000, most=most)
        _same_eviction(x, 4000, 4000, 5000, most=most)


def test_eviction_flags():
    x = _case([300, 310, 290], 2, 2, "bf16", 16, 132)
    want = _evict(x, keep=100, recent=10)
    for lens, at, flag_is in [([300, 401, 290], None, da.FLAG_BAD_SEQ_LEN),
                              ([300, -1, 290], None, da.FLAG_BAD_SEQ_LEN),
                              ([300, 310, 290], -1, da.FLAG_BAD_BLOCK),
                              ([300, 310, 290], 4000, da.FLAG_BAD_BLOCK)]:
        table = x["table"].clone()
        if at is not None:
            table[1, 19] = at
        kw = dict(lens=_i32(lens), table=table)
        k, v, w, e, flag = _evict(x, keep=100, recent=10, most=310, **kw)
        assert flag == flag_is and e.new_lens.tolist() == [-200, 0, -190]
        assert bool((e.kept[1] == -1).all()) and torch.equal(e.kept[::2], want[3].kept[::2])
        ids = x["table"][1, :20].long()
        other = x["table"][0, :19].long()
        for got, ref, had in zip((k, v, w), want, [*x["caches"], x["weights"]]):
            assert np.array_equal(_bytes(got[ids]), _bytes(had[ids]))
            assert np.array_equal(_bytes(got[other]), _bytes(ref[other]))


# ------------------------------------------------------------------ streams, graphs, bounds


def _calls_of(x, **kw):
    """Each operator's call on x with fresh outputs, as a function of the stream, and the
    tensors that it returns or updates."""
    bounds, weights = _bounds_of(x), x["weights"]
    lists = _i32(_lists(x, 9, 3, empty=False))
    ws = torch.empty(da.gqa_weights_workspace_size(len(x["n"]), x["h_q"], x["max_len"], 4) + (1 << 20),
                     dtype=torch.uint8, device=DEV)

    def select(**k):
        return [da.gqa_select_blocks(x["q"], bounds, x["table"], x["lens"], block_size=x["bs"],
                                     max_seq_len=x["max_len"], count=6, workspace=ws, **kw, **k)]

    def blocks(**k):
        return [_decode(x, "blocks", x["table"], x["lens"], lists, scale=0.1, num_splits=3,
                        workspace=ws, **kw, **k)]

    def weighed(**k):
        w = weights.clone()
        return [_decode(x, "weights", w, x["table"], x["lens"], scale=0.1, num_splits=4, workspace=ws,
                        **kw, **k), w]

    def evict(**k):
        c = [t.clone() for t in x["caches"]]
        w = weights.clone()
        e = da.gqa_kv_evict(*c, w, x["table"], x["lens"], max_seq_len=x["max_len"], keep=90, recent=9,
                            limit=100, **kw, **k)
        return [*(t.view(torch.uint8) for t in c), w, *e]

    def bound(**k):
        b = torch.zeros_like(bounds)
        return [da.gqa_block_bounds(x["caches"][0], x["table"], x["lens"], b, max_seq_len=x["max_len"],
                                    **kw, **k).view(torch.uint8)]

    return select, blocks, weighed, evict, bound


@pytest.mark.parametrize("heads", [(8, 2), (32, 1)])
@pytest.mark.parametrize("fp8", [False, True])
def test_captured_calls_share_a_workspace(heads, fp8):
    """Two graphs whose calls use the same workspace, replayed in turn over new queries."""
    x = _case([700, 333, 100], *heads, "bf16", 16, 150, fp8=fp8)
    y = _case([64, 900, 512], *heads, "bf16", 16, 151, fp8=fp8)
    calls = [_calls_of(x), _calls_of(y)]
    for fns in calls:
        for fn in fns:
            fn()
    torch.cuda.synchronize()
    graphs, outs, stream = [], [], torch.cuda.Stream()
    for fns in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            outs.append([t for fn in fns for t in fn()])
    for seed in (1, 2):
        for z, graph, out, fns in zip((x, y), graphs, outs, calls):
            z["q"].copy_(torch.randn(z["q"].shape, generator=_gen(seed), device=DEV))
            graph.replay()
            torch.cuda.synchronize()
            for got, want in zip(out, [t for fn in fns for t in fn()]):
                assert torch.equal(got.view(torch.int32) if got.dtype == torch.float32 else got,
                                   want.view(torch.int32) if want.dtype == torch.float32 else want)


def test_calls_on_another_stream():
    """On a given stream, and under one: the results of the default stream's calls; what is
    returned may be dropped while it is in use."""
    x = _case([700, 333, 100], 8, 2, "bf16", 16, 152)
    want = [t for fn in _calls_of(x) for t in fn()]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for handle in (stream, stream.cuda_stream):
        stream.wait_stream(torch.cuda.current_stream())
        fns = _calls_of(x)
        torch.cuda.synchronize()
        got = []
        for fn in fns:
            r = fn(stream=handle) if fn.__name__ in ("select", "blocks") else None
            if r is None:
                with torch.cuda.stream(stream):
                    r = fn()
            got += r
        torch.cuda.current_stream().wait_stream(stream)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("heads", [(8, 8), (8, 2), (32, 1)])
def test_a_bound_far_above_the_lengths(heads):
    """max_seq_len as a captured step has it (short sequences, a long bound) changes no
    result."""
    x = _case([700, 333, 1, 0], *heads, "bf16", 16, 153, most=4096)
    bounds = _bounds_of(x)
    x["max_len"] = 65536
    assert torch.equal(bounds, _bounds_of(x))
    _same_choice(x, bounds, count=6)
    lists = _lists(x, 30, 4)
    got = _decode(x, "blocks", x["table"], x["lens"], _i32(lists), scale=0.1)
    ref, keys = _attend(x, 0.1, lists)
    _close(x, got, ref, keys, 0.1)
    before, w = x["weights"].clone(), x["weights"].clone()
    got = _decode(x, "weights", w, x["table"], x["lens"], scale=0.1)
    ref, keys = _attend(x, 0.1)
    _close(x, got, ref, keys, 0.1)
    _weights_close(x, w, before, ref, keys, 0.1)
    if heads[0] != 32:
        _same_eviction(x, 300, 20, 320)


def test_calls_of_different_sizes_from_threads():
    """Choices and evictions that need little and much shared memory, at the same time, each
    on a stream of its own: every result as alone."""
    jobs, failed = [], []
    for i, (n, bs) in enumerate([(500, 16), (60000, 8), (9000, 8), (33000, 16)]):
        x = _case([n, n // 3], 2, 1, "bf16", bs, 160 + i, fp8=True)
        bounds = _bounds_of(x)

        def both(x=x, bounds=bounds):
            some = da.gqa_select_blocks(x["q"], bounds, x["table"], x["lens"], block_size=x["bs"],
                                        max_seq_len=x["max_len"], count=9)
            c, w = [t.clone() for t in x["caches"]], x["weights"].clone()
            e = da.gqa_kv_evict(*c, w, x["table"], x["lens"], max_seq_len=x["max_len"], keep=300,
                                recent=20)
            return [some, *(t.view(torch.uint8) for t in c), w.view(torch.int32), *e]

        jobs.append((both, [t.clone() for t in both()]))
    torch.cuda.synchronize()

    def work(both, want):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(30):
                    got = both()
                stream.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want))
                stream.synchronize()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


@pytest.mark.parametrize("heads", [(16, 8), (64, 1)])
def test_blocks_far_into_a_large_cache(heads):
    """Sequences whose blocks lie past 2^31 elements of the cache: the same results as those
    of the same sequences in a small one."""
    h_q, h_kv = heads
    x = _case([300, 77], h_q, h_kv, "bf16", 256, 170, spare=0)
    nb = (1 << 31) // (256 * h_kv * 128) + 9
    far = torch.tensor([nb - 1, nb - 4, nb - 2], dtype=torch.int32, device=DEV)
    y = dict(x)
    y["table"] = torch.where(x["table"] >= 0, far[x["table"].clamp(min=0).long()], -1)
    y["caches"] = [torch.empty((nb, *c.shape[1:]), dtype=c.dtype, device=DEV) for c in x["caches"]]
    y["weights"] = torch.empty((nb, *x["weights"].shape[1:]), device=DEV)
    for a, b in zip([*x["caches"], x["weights"]], [*y["caches"], y["weights"]]):
        b[far.long()] = a
    bounds = [torch.zeros((z["caches"][0].shape[0], 2, h_kv, 128), dtype=torch.bfloat16, device=DEV)
              for z in (x, y)]
    lists = _i32(_lists(x, 2, 5, empty=False))
    results = []
    for z, b in zip((x, y), bounds):
        flag = _flag()
        rows = torch.arange(3, device=DEV) if z is x else far.long()
        da.gqa_block_bounds(z["caches"][0], z["table"], z["lens"], b, max_seq_len=300, err_flag=flag)
        r = [b[rows].view(torch.int16),
             da.gqa_select_blocks(z["q"], b, z["table"], z["lens"], block_size=256, max_seq_len=300,
                                  count=1, first=0, last=0, err_flag=flag),
             _decode(z, "blocks", z["table"], z["lens"], lists, scale=0.1, err_flag=flag),
             _decode(z, "weights", z["weights"], z["table"], z["lens"], scale=0.1, err_flag=flag)]
        r.append(z["weights"][rows].clone())
        e = da.gqa_kv_evict(*z["caches"], z["weights"], z["table"], z["lens"], max_seq_len=300, keep=70,
                            recent=9, err_flag=flag)
        r += [e.kept, e.new_lens, z["weights"][rows]] + [c[rows].view(torch.int16) for c in z["caches"]]
        assert int(flag) == 0
        results.append(r)
    for a, b in zip(*results):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_a_run_of_steps_with_eviction_and_selection(fp8, captured):
    """Prompts, then single tokens: plan, cache write, bounds, choice, decode over the
    chosen blocks, decode with weights, and every few steps an eviction whose blocks
    the plan takes back.  Each step equals the plain forms on the cache it found;
    captured, a step's launches are one graph that is replayed."""
    h_q, h_kv, bs, M, B, nb, T = 8, 2, 16, 24, 3, 64, 320
    g = _gen(200)
    rope = da.rope_table([1e4 ** (-i / 64) for i in range(64)])
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    caches = [torch.full((nb, bs, h_kv, 128), float("nan"), device=DEV).to(kind) for _ in "kv"]
    scales = [torch.tensor([1 / 64, 1 / 32], device=DEV) for _ in "kv"] if fp8 else []
    bounds = torch.zeros((nb, 2, h_kv, 128), device=DEV).to(kind)
    weights = torch.full((nb, h_kv, bs), float("nan"), device=DEV)
    lens, table, had = _i32([0] * B), _i32(np.full((B, M), -1)), _i32([0] * B)
    free, count = _i32(np.random.default_rng(1).permutation(nb)), _i32([nb])
    new, flag = _i32([0] * B), _flag()
    qkv = torch.zeros((T, (h_q + 2 * h_kv) * 128), device=DEV).bfloat16()
    out = {}

    def step():
        had.copy_(lens)
        p = da.paged_plan(lens, new, table, free, count, block_size=bs, max_tokens=T, seq_lens=lens,
                          free_count_out=count, err_flag=flag)
        q, k, v = (x.view(T, -1, 128) for x in qkv.split([h_q * 128, h_kv * 128, h_kv * 128], 1))
        turn = da.gqa_rope_append_fp8kv if fp8 else da.gqa_rope_append
        qr = turn(q, k, v, *scales, p.positions, rope, p.slots, *caches, err_flag=flag)
        rows = qr.index_select(0, (p.q_start[1:] - 1).clamp(min=0).long())
        da.gqa_block_bounds(caches[0], table, lens, bounds, first_lens=had, max_seq_len=M * bs,
                            err_flag=flag)
        some = da.gqa_select_blocks(rows, bounds, table, lens, block_size=bs, max_seq_len=M * bs,
                                    count=6, first=1, last=2, err_flag=flag)
        fn = da.gqa_decode_fp8kv_blocks if fp8 else da.gqa_decode_blocks
        sparse = fn(rows, *caches, *scales, table, lens, some, scale=0.09, max_seq_len=M * bs,
                    err_flag=flag)
        fn = da.gqa_decode_fp8kv_weights if fp8 else da.gqa_decode_weights
        dense = fn(rows, *caches, *scales, weights, table, lens, scale=0.09, max_seq_len=M * bs,
                   weighed_lens=had, err_flag=flag)
        out.update(rows=rows, some=some, sparse=sparse, dense=dense)

    def evict():
        e = da.gqa_kv_evict(*caches, weights, table, lens, max_seq_len=M * bs, keep=150, recent=30,
                            limit=180, err_flag=flag)
        da.paged_plan(lens, e.new_lens, table, free, count, block_size=bs, max_tokens=0,
                      seq_lens=lens, free_count_out=count, err_flag=flag)
        da.gqa_block_bounds(caches[0], table, lens, bounds, max_seq_len=M * bs, err_flag=flag)
        out.update(moved=e.new_lens, kept=e.kept)

    graphs = {}
    if captured:
        stream = torch.cuda.Stream()
        for fn in (step, evict):
            fn()  # (empty sequences: no state changes; loads every kernel)
            torch.cuda.synchronize()
            graphs[fn] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[fn], stream=stream):
                fn()

    def x_now():
        return dict(q=out["rows"], caches=caches, scales=scales, table=table, lens=lens,
                    n=lens.tolist(), bs=bs, h_q=h_q, h_kv=h_kv, dtype="bf16", fp8=fp8)

    for i in range(14):
        new.copy_(_i32([160, 40, 90] if i == 0 else [8, 1, 13] if i < 5 else [1, 1, 1]))
        qkv.copy_(torch.randn(qkv.shape, generator=g, device=DEV))
        before, n_before = weights.clone(), had.tolist()
        graphs[step].replay() if captured else step()
        torch.cuda.synchronize()
        assert int(flag) == 0
        x = x_now()
        want = long_cache.select_blocks(_np(out["rows"]), _np(bounds), table.cpu().numpy(), x["n"],
                                        block_size=bs, count=6, first=1, last=2)
        assert np.array_equal(out["some"].cpu().numpy(), want)
        ref, keys = _attend(x, 0.09, want)
        _close(x, out["sparse"], ref, keys, 0.09)
        ref, keys = _attend(x, 0.09)
        _close(x, out["dense"], ref, keys, 0.09)
        _weights_close(x, weights, before, ref, keys, 0.09, weighed=had.tolist())
        if i % 4 == 3:
            raw = [c.view(torch.uint8 if fp8 else torch.int16).cpu().numpy() for c in caches]
            plain = long_cache.evict(*raw, weights.cpu().numpy(), table.cpu().numpy(), x["n"], keep=150,
                                     recent=30, limit=180)
            low = int(count)
            graphs[evict].replay() if captured else evict()
            torch.cuda.synchronize()
            assert int(flag) == 0 and np.array_equal(out["kept"].cpu().numpy(), plain[4])
            assert lens.tolist() == [n + m for n, m in zip(x["n"], plain[3])]
            assert int(count) == low + sum(-(-n // bs) - -(-(n + int(m)) // bs)
                                           for n, m in zip(x["n"], plain[3]))
            for c, ref in zip([*caches, weights], plain):
                view = {1: torch.uint8, 2: torch.int16, 4: torch.float32}[c.element_size()]
                assert np.array_equal(c.view(view).cpu().numpy(), ref, equal_nan=view.is_floating_point)
    assert max(lens.tolist()) <= 200 and int(count) > 20
