"""What the attention kernels make of NaN and infinity that a row sees, on the
GPU against the definition in 64 bits: a NaN in a query or in a key of its, or an
infinite score, makes the whole row NaN, and one in a value the value's dimension;
a score of -inf has weight 0.  (What no row sees may hold anything: the other
tests.)  Tolerances of the finite rows as in test_step_ops_gpu.py."""
import numpy as np
import pytest
import torch

import gqa_mqa_mla_gb300 as da
from oracle import step

from test_step_ops_gpu import DEV, HALF, _attn_case, _close, _fp16_probs, _run_prefill

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def _values(x):
    """The caches' values in 64 bits, NaN and infinities as they are."""
    if x["scales"] is None:
        return [c.double().cpu().numpy() for c in x["caches"]]
    return [(c.view(torch.float8_e4m3fn).double() * s.double()[:, None]).cpu().numpy()
            for c, s in zip(x["caches"], x["scales"])]


def _defined(x, **kw):
    with np.errstate(all="ignore"):
        return step.attend(x["q"].double().cpu().numpy(), *_values(x), x["table"].cpu().numpy(),
                           x["start"].cpu().numpy(), x["lens"].cpu().numpy(), **kw)


def _slot(x, b, t):
    bs = x["caches"][0].shape[1]
    return int(x["table"][b, t // bs]), t % bs


def _spoil(x, what):
    """Puts one value that is not finite where rows see it."""
    fp8 = x["scales"] is not None
    last = int(x["start"][1]) - 1  # the first sequence's last row
    if what in ("q nan", "q inf", "q -inf"):
        x["q"][last, 1, 77] = float(what[2:])
        x["q"][0, 0, 3] = NAN  # and the first row's first head
        return
    kind, value, t = what.split()
    t = int(x["lens"][0]) - 2 if t == "late" else int(t)
    blk, at = _slot(x, 0, t)
    x["caches"][0 if kind == "k" else 1][blk, at, 0, 5] = 0x7F if fp8 else float(value)


def _agrees(got, ref, clean, dtype, what):
    """NaN and infinities where the definition has them; the rest within the
    tolerance (whose score error is the clean data's: an infinite key has no
    error of its own)."""
    out = ref[0]
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(out)), (what, int(np.isnan(g).sum()),
                                                       int(np.isnan(out).sum()))
    assert np.isnan(out).any() or np.isinf(out).any() or "inf" in what
    big = np.isinf(out)
    assert np.array_equal(g[big], out[big]), what
    keep = np.isfinite(out)
    r = [np.where(keep, a, np.nan) for a in ref[:3]]
    # (0 times an infinite value: nothing is left of it.)
    r[1], r[2] = (np.where(np.isfinite(a), a, c) for a, c in zip(r[1:], clean[1:3]))
    _close(torch.from_numpy(np.where(keep, g, 0.0)), (r[0], r[1], r[2], clean[3]), dtype, what)


# (An 8-bit cache holds no infinity.)
WHAT = [(w, fp8) for w in ("q nan", "q inf", "q -inf", "k nan 0", "k nan late", "k inf 2",
                           "k -inf 2", "v nan 0", "v inf 0")
        for fp8 in (False, True) if not (fp8 and "inf" in w)]

CHUNKS = [
    # q_lens, lens, h_q, h_kv, dtype, block, window, sinks
    ([40, 3, 130], [400, 300, 130], 8, 2, "bf16", 16, 0, 0),
    ([3, 5], [700, 90], 64, 1, "fp16", 64, 0, 0),
    ([50, 3, 200], [400, 900, 333], 8, 2, "fp16", 16, 60, 4),
    ([260], [300], 4, 4, "bf16", 8, 0, 0),
]


@pytest.mark.parametrize("what,fp8", WHAT)
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_prefill_passes_on_what_is_not_finite(case, what, fp8):
    q_lens, lens, h_q, h_kv, dtype, bs, window, sinks = CHUNKS[case]
    x = _attn_case(q_lens, lens, h_q, h_kv, dtype, bs, 700 + case, fp8=fp8)
    kw = dict(scale=0.09, window=window, sinks=sinks)
    clean = _defined(x, **kw)
    _spoil(x, what)
    ref = _defined(x, **kw)
    if fp8:
        ref, clean = (_fp16_probs(r, dtype) for r in (ref, clean))
    for splits in (1, 3):
        out, flag = _run_prefill(x, scale=0.09, window=window or None, sinks=sinks,
                                 num_splits=splits)
        assert flag == 0
        _agrees(out, ref, clean, dtype, f"{what}, {splits} splits")


DECODE = [
    # lens, h_q, h_kv, dtype, block, window, sinks
    ([1000, 64, 500, 129], 16, 2, "bf16", 16, 900, 4),
    ([700, 64], 8, 8, "fp16", 8, 600, 64),
    ([900, 129], 32, 2, "fp16", 64, 800, 66),
    ([1000, 900], 64, 1, "bf16", 16, 800, 130),
    ([700, 300], 33, 1, "fp16", 256, 600, 3),
]


@pytest.mark.parametrize("what,fp8", WHAT)
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode_passes_on_what_is_not_finite(case, what, fp8):
    """With a window and sinks (one split, a cluster of them, a launch that joins
    them), and without."""
    lens, h_q, h_kv, dtype, bs, window, sinks = DECODE[case]
    x = _attn_case([1] * len(lens), lens, h_q, h_kv, dtype, bs, 750 + case, fp8=fp8)
    full = _defined(x, scale=0.09)
    clean = _defined(x, scale=0.09, window=window, sinks=sinks)
    _spoil(x, what)
    if what == "k nan late":
        assert int(x["lens"][0]) - 2 > int(x["lens"][0]) - window
    fn = da.gqa_decode if not fp8 else da.gqa_decode_fp8kv
    for w, n, c in ((window, sinks, clean), (0, 0, full)):
        ref = _defined(x, scale=0.09, window=w, sinks=n)
        if fp8:
            ref, c = ((r[0], r[1] + 2.0**-25 * r[2] / HALF[dtype], r[2], r[3]) for r in (ref, c))
        for splits in (1, 4, 10):
            out = fn(x["q"], *x["caches"], *(x["scales"] or []), x["table"], x["lens"], scale=0.09,
                     max_seq_len=x["max_len"], window=w or None, sinks=n, num_splits=splits)
            _agrees(out, ref, c, dtype, f"{what}, window {w}, {splits} splits")


def test_scores_of_minus_infinity_alone_see_nothing():
    """A row all of whose scores are -inf has no weight to give: zeros, as a row
    that sees nothing; a stretch of the cache without weight does not disturb the
    rest (16-bit caches: e4m3 has no infinity)."""
    for h_q, h_kv in ((8, 2), (8, 8), (64, 1)):
        x = _attn_case([1, 1], [600, 600], h_q, h_kv, "bf16", 16, 795)
        x["q"].abs_()
        bs = 16
        for b, (lo, hi) in enumerate([(0, 600), (64, 448)]):
            t = torch.arange(lo, hi, device=DEV)
            x["caches"][0][x["table"][b][t // bs].long(), t % bs, :, 9] = -INF
        want = _defined(x, scale=0.09)
        for splits in (1, 4, 10):
            for fn in ("decode", "prefill", "sinks"):
                if fn == "prefill":
                    out, _ = _run_prefill(x, scale=0.09, num_splits=splits)
                else:
                    kw = dict(window=590, sinks=10) if fn == "sinks" else {}
                    out = da.gqa_decode(x["q"], *x["caches"], x["table"], x["lens"], scale=0.09,
                                        max_seq_len=600, num_splits=splits, **kw)
                assert bool((out[0] == 0).all()), (fn, splits)
                got, ref = out[1].double().cpu().numpy(), want[0][1]
                # u |out| + (u + 2^-10) A, A = sum p |v| / sum p <= the spread
                tol = 2.0**-8 * np.abs(ref) + (2.0**-8 + 2.0**-10) * want[1][1]
                assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all(), (fn, splits)


@pytest.mark.parametrize("value", [INF, -INF])
def test_infinite_queries_over_an_8_bit_cache(value):
    """They have no e4m3 terms; their rows are NaN, the others what they are."""
    for case, (q_lens, lens, h_q, h_kv, dtype, bs, window, sinks) in enumerate(CHUNKS):
        x = _attn_case(q_lens, lens, h_q, h_kv, dtype, bs, 770 + case, fp8=True)
        kw = dict(scale=0.09, window=window or None, sinks=sinks)
        for splits in (1, 3):
            good, _ = _run_prefill(x, num_splits=splits, **kw)
            q = x["q"].clone()
            q[q_lens[0] - 1, 1, 77], q[-1, 0, 0] = value, -value
            out, flag = _run_prefill(dict(x, q=q), num_splits=splits, **kw)
            bad = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
            bad[q_lens[0] - 1, 1] = bad[-1, 0] = True
            assert flag == 0 and bool(out[bad].isnan().all())
            assert torch.equal(out[~bad], good[~bad])
    for case, (lens, h_q, h_kv, dtype, bs, window, sinks) in enumerate(DECODE):
        x = _attn_case([1] * len(lens), lens, h_q, h_kv, dtype, bs, 780 + case, fp8=True)
        q = x["q"].clone()
        q[0, 1, 77] = value
        for kw in (dict(window=window, sinks=sinks), {}):
            for splits in (1, 4):
                good, out = (da.gqa_decode_fp8kv(y, *x["caches"], *x["scales"], x["table"], x["lens"],
                                                 scale=0.09, max_seq_len=x["max_len"],
                                                 num_splits=splits, **kw) for y in (x["q"], q))
                assert bool(out[0, 1].isnan().all()) and torch.equal(out[1:], good[1:])
                rest = [h for h in range(h_q) if h != 1]
                assert torch.equal(out[0, rest], good[0, rest])


@pytest.mark.parametrize("splits", [1, 3])
def test_scales_of_an_8_bit_cache_that_are_not_finite(splits):
    """A head whose K or V scale is NaN gives NaN, in chunks and in decode; the
    others what they are."""
    for j in (0, 1):
        x = _attn_case([40, 3], [400, 300], 6, 3, "bf16", 16, 790, fp8=True)
        good, _ = _run_prefill(x, num_splits=splits)
        x["scales"][j][1] = NAN
        out, flag = _run_prefill(x, num_splits=splits)
        assert flag == 0 and bool(out[:, 2:4].isnan().all())
        assert torch.equal(out[:, :2], good[:, :2]) and torch.equal(out[:, 4:], good[:, 4:])
        out = da.gqa_decode_fp8kv_sinks(x["q"][[39, 42]], *x["caches"], *x["scales"], x["table"],
                                        x["lens"], scale=0.1, max_seq_len=400, window=300, sinks=4,
                                        num_splits=splits)
        assert bool(out[:, 2:4].isnan().all()) and bool(out[:, [0, 1, 4, 5]].isfinite().all())
