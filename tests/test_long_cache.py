"""The operators for long caches without a GPU: refusals of the C ABI and of the
binding, planners and workspace sizes, and the plain forms themselves."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gqa_mqa_mla_gb300 as da
from gqa_mqa_mla_gb300 import binding, build
from oracle import long_cache

FAKE = 0x100000
INVALID, UNSUPPORTED, WORKSPACE = (binding.DECATTN_ERR_INVALID_ARG,
                                   binding.DECATTN_ERR_UNSUPPORTED,
                                   binding.DECATTN_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def _launch(kw):
    if kw is None:
        return None
    d = dict(batch=2, num_blocks=64, block_size=16, max_blocks_per_seq=16, max_seq_len=256,
             num_splits=1, dtype=binding.DECATTN_BF16, workspace=None, workspace_bytes=0,
             err_flag=None, stream=None)
    d.update(kw)
    return ctypes.byref(binding.Launch(**d))


# What every call refuses of its launch block.
LAUNCHES = [
    (dict(L=None), INVALID), (dict(L=dict(batch=0)), INVALID), (dict(L=dict(num_blocks=0)), INVALID),
    (dict(L=dict(block_size=12)), INVALID), (dict(L=dict(block_size=4)), UNSUPPORTED),
    (dict(L=dict(block_size=512)), UNSUPPORTED), (dict(L=dict(dtype=5)), INVALID),
    (dict(L=dict(max_seq_len=-1)), INVALID), (dict(L=dict(max_seq_len=257)), INVALID),
    (dict(L=dict(num_blocks=1 << 28)), UNSUPPORTED), (dict(L=dict(err_flag=FAKE + 2)), INVALID),
    (dict(L=dict(max_seq_len=0x7fffffff, max_blocks_per_seq=1 << 27)), UNSUPPORTED),
]


@pytest.mark.parametrize("case,expect", LAUNCHES + [
    (dict(k=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(bt=None), INVALID),
    (dict(bt=FAKE + 2), INVALID), (dict(first=FAKE + 1), INVALID), (dict(lens=None), INVALID),
    (dict(lens=FAKE + 2), INVALID), (dict(bounds=None), INVALID), (dict(bounds=FAKE + 4), INVALID),
    (dict(bounds=FAKE), INVALID), (dict(h_kv=0), INVALID), (dict(h_kv=1025), INVALID),
    (dict(kv_bytes=4), INVALID), (dict(d=64), UNSUPPORTED),
])
def test_bounds_host_checks(lib, case, expect):
    a = dict(k=FAKE, bt=FAKE, first=None, lens=FAKE, bounds=2 * FAKE, h_kv=2, d=128, kv_bytes=2, L={})
    a.update(case)
    assert lib.gqa_block_bounds(a["k"], a["bt"], a["first"], a["lens"], a["bounds"], a["h_kv"],
                                a["d"], a["kv_bytes"], _launch(a["L"])) == expect


@pytest.mark.parametrize("case,expect", LAUNCHES + [
    (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(bounds=None), INVALID),
    (dict(bt=FAKE + 1), INVALID), (dict(lens=None), INVALID), (dict(out=None), INVALID),
    (dict(out=FAKE + 2), INVALID), (dict(h_q=9), INVALID), (dict(h_kv=0), INVALID),
    (dict(h_q=130), UNSUPPORTED), (dict(d=64), UNSUPPORTED), (dict(kv_bytes=0), INVALID),
    (dict(count=0), INVALID), (dict(first=-1), INVALID), (dict(last=-1), INVALID),
    (dict(first=3, last=3), INVALID), (dict(first=0x7fffffff, last=0x7fffffff), INVALID),
    (dict(L=dict(batch=65536)), UNSUPPORTED),
    (dict(), WORKSPACE),
    (dict(L=dict(workspace=FAKE, workspace_bytes=100)), WORKSPACE),
    (dict(L=dict(workspace=FAKE + 8, workspace_bytes=1 << 20)), INVALID),
])
def test_selection_host_checks(lib, case, expect):
    a = dict(q=FAKE, bounds=FAKE, bt=FAKE, lens=FAKE, out=FAKE, h_q=8, h_kv=2, d=128, kv_bytes=2,
             count=5, first=1, last=1, L={})
    a.update(case)
    assert lib.gqa_select_blocks(a["q"], a["bounds"], a["bt"], a["lens"], a["out"], a["h_q"],
                                 a["h_kv"], a["d"], a["kv_bytes"], a["count"], a["first"],
                                 a["last"], _launch(a["L"])) == expect


DECODE = LAUNCHES + [
    (dict(q=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v=None), INVALID),
    (dict(bt=None), INVALID), (dict(lens=FAKE + 2), INVALID), (dict(out=None), INVALID),
    (dict(h_q=9), INVALID), (dict(h_q=130), UNSUPPORTED), (dict(d=64), UNSUPPORTED),
    (dict(scale=float("inf")), INVALID), (dict(L=dict(num_splits=257)), INVALID),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case,expect", DECODE + [
    (dict(some=None), INVALID), (dict(some=FAKE + 2), INVALID), (dict(count=0), INVALID),
    (dict(L=dict(num_splits=2)), WORKSPACE),
])
def test_blocks_host_checks(lib, fp8, case, expect):
    a = dict(q=FAKE, k=FAKE, v=FAKE, bt=FAKE, lens=FAKE, some=FAKE, out=FAKE, h_q=8, h_kv=2, d=128,
             scale=0.1, count=9, L={})
    a.update(case)
    fn = lib.gqa_decode_fp8kv_blocks if fp8 else lib.gqa_decode_blocks
    assert fn(a["q"], a["k"], a["v"], *([FAKE, FAKE] if fp8 else []), a["bt"], a["lens"], a["some"],
              a["out"], a["h_q"], a["h_kv"], a["d"], a["scale"], a["count"],
              _launch(a["L"])) == expect


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case,expect", DECODE + [
    (dict(weights=None), INVALID), (dict(weights=FAKE + 8), INVALID), (dict(weighed=FAKE + 2), INVALID),
    (dict(decay=float("nan")), INVALID),
    (dict(), WORKSPACE),  # even with one split: the scores
    (dict(L=dict(workspace=FAKE, workspace_bytes=2 * 8 * 256 * 4)), WORKSPACE),
])
def test_weights_host_checks(lib, fp8, case, expect):
    a = dict(q=FAKE, k=FAKE, v=FAKE, bt=FAKE, lens=FAKE, weighed=None, weights=FAKE, out=FAKE, h_q=8,
             h_kv=2, d=128, scale=0.1, decay=1.0, L={})
    a.update(case)
    fn = lib.gqa_decode_fp8kv_weights if fp8 else lib.gqa_decode_weights
    assert fn(a["q"], a["k"], a["v"], *([FAKE, FAKE] if fp8 else []), a["bt"], a["lens"],
              a["weighed"], a["weights"], a["out"], a["h_q"], a["h_kv"], a["d"], a["scale"],
              a["decay"], _launch(a["L"])) == expect


@pytest.mark.parametrize("case,expect", LAUNCHES + [
    (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID), (dict(v=FAKE), INVALID),
    (dict(weights=FAKE + 4), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID),
    (dict(new=None), INVALID), (dict(new=FAKE), INVALID), (dict(kept=FAKE + 1), INVALID),
    (dict(h_kv=0), INVALID), (dict(d=64), UNSUPPORTED), (dict(kv_bytes=3), INVALID),
    (dict(keep=0), INVALID), (dict(recent=-1), INVALID), (dict(recent=101), INVALID),
    (dict(limit=99), INVALID), (dict(L=dict(batch=65536)), UNSUPPORTED),
])
def test_eviction_host_checks(lib, case, expect):
    a = dict(k=FAKE, v=2 * FAKE, weights=FAKE, bt=FAKE, lens=FAKE, new=2 * FAKE, kept=FAKE, h_kv=2,
             d=128, kv_bytes=2, keep=100, recent=10, limit=120, L={})
    a.update(case)
    assert lib.gqa_kv_evict(a["k"], a["v"], a["weights"], a["bt"], a["lens"], a["new"], a["kept"],
                            a["h_kv"], a["d"], a["kv_bytes"], a["keep"], a["recent"], a["limit"],
                            _launch(a["L"])) == expect


@pytest.mark.parametrize("many", [0x7fffffff, 0x7fffffff - 65535])
def test_lists_past_32_bit_steps_are_refused(lib, many):
    L = _launch({})
    assert lib.gqa_select_blocks(FAKE, FAKE, FAKE, FAKE, FAKE, 8, 2, 128, 2, many, 1, 1,
                                 L) == UNSUPPORTED
    assert lib.gqa_decode_blocks(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 8, 2, 128, 0.1, many,
                                 L) == UNSUPPORTED
    assert lib.gqa_decode_fp8kv_blocks(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 8, 2,
                                       128, 0.1, many, L) == UNSUPPORTED
    assert lib.gqa_kv_evict(FAKE, 2 * FAKE, FAKE, FAKE, FAKE, 2 * FAKE, FAKE, 2, 128, 2, many, 0,
                            many, L) == UNSUPPORTED


def test_sizes_and_splits(lib):
    assert da.gqa_select_workspace_size(2, 4, 1000, 16, 63) == 0
    assert da.gqa_select_workspace_size(2, 4, 1000, 16, 62) >= 8 * 63 * 12
    assert da.gqa_select_workspace_size(2, 4, 1000, 12, 5) == 0
    assert da.gqa_select_workspace_size(1, 1, (1 << 31) - 70000, 8, 5) > 12 << 28
    for splits in (1, 7):
        rows = 3 * 12
        need = rows * splits * 4 + rows * 1024 * 4 + (rows * splits * 512 if splits > 1 else 0)
        got = da.gqa_weights_workspace_size(3, 12, 1000, splits)
        assert need <= got <= need + 3 * 256
    assert da.gqa_weights_workspace_size(3, 12, 1000, 0) == 0
    assert da.gqa_weights_workspace_size(1, 1, 0, 1) > 0
    for B, h_q, h_kv, most, count, bs, kv in [(32, 64, 8, 32768, 128, 16, 2), (1, 32, 1, 32768, 33, 64, 1),
                                              (4, 8, 8, 500, 1000, 8, 2), (1, 8, 2, 0, 1, 16, 1)]:
        got = da.gqa_blocks_plan_splits(B, h_q, h_kv, most, count, bs, kv, num_sms=152)
        span = min(most, count * bs)
        assert 1 <= got <= max(1, -(-span // 64))
    for B, h_q, h_kv, most, kv in [(64, 64, 8, 8192, 2), (7, 32, 32, 5000, 1), (1, 32, 1, 32768, 1), (1, 8, 2, 0, 2)]:
        got = da.gqa_weights_plan_splits(B, h_q, h_kv, most, kv, num_sms=152)
        assert 1 <= got <= max(1, -(-most // 64))
        if h_q != h_kv:
            plain = da.gqa_plan_splits if kv == 2 else da.gqa_fp8_plan_splits
            assert got == plain(B, h_q, h_kv, most, num_sms=152)
    with pytest.raises(da.DecAttnError):
        da.gqa_blocks_plan_splits(1, 8, 2, 100, 0, 16)
    with pytest.raises(da.DecAttnError):
        da.gqa_weights_plan_splits(1, 8, 2, 100, 3)


# ------------------------------------------------------------------ the binding's refusals


def _tensors(**kw):
    d = dict(q=torch.zeros(3, 8, 128, dtype=torch.bfloat16), k=torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16),
             v=torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16), w=torch.zeros(4, 2, 16),
             bounds=torch.zeros(4, 2, 2, 128, dtype=torch.bfloat16),
             table=torch.zeros(3, 4, dtype=torch.int32), lens=torch.zeros(3, dtype=torch.int32),
             some=torch.zeros(3, 2, 5, dtype=torch.int32))
    d.update(kw)
    return d


def _calls(x):
    kw = dict(max_seq_len=64)
    return dict(
        bounds=lambda **k: da.gqa_block_bounds(x["k"], x["table"], x["lens"], x["bounds"], **kw, **k),
        select=lambda **k: da.gqa_select_blocks(x["q"], x["bounds"], x["table"], x["lens"],
                                                **{**kw, "block_size": 16, "count": 2, **k}),
        blocks=lambda **k: da.gqa_decode_blocks(x["q"], x["k"], x["v"], x["table"], x["lens"], x["some"],
                                                scale=0.1, **kw, **k),
        weights=lambda **k: da.gqa_decode_weights(x["q"], x["k"], x["v"], x["w"], x["table"], x["lens"],
                                                  scale=0.1, **kw, **k),
        evict=lambda **k: da.gqa_kv_evict(x["k"], x["v"], x["w"], x["table"], x["lens"],
                                          **{**kw, "keep": 5, "recent": 1, **k}))


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


BAD = [
    # call, replaced tensors, arguments, exception, text
    ("bounds", dict(k=torch.zeros(4, 16, 2, 128)), {}, TypeError, "k_cache"),
    ("bounds", dict(k=torch.zeros(4, 16, 256, dtype=torch.bfloat16)), {}, ValueError, "4 dims"),
    ("bounds", dict(bounds=torch.zeros(4, 2, 2, 128, dtype=torch.float16)), {}, TypeError, "k_cache's type"),
    ("bounds", dict(bounds=torch.zeros(4, 2, 2, 128, dtype=torch.uint8)), {}, TypeError, "k_cache's type"),
    ("bounds", dict(bounds=torch.zeros(3, 2, 2, 128, dtype=torch.bfloat16)), {}, ValueError, "bounds must be"),
    ("bounds", dict(bounds=torch.zeros(4, 2, 128, 2, dtype=torch.bfloat16).transpose(2, 3)), {}, ValueError,
     "contiguous"),
    ("select", dict(bounds=torch.zeros(4, 2, 2, 128, dtype=torch.float16)), {}, TypeError, "bounds"),
    ("select", dict(bounds=torch.zeros(4, 2, 2, 64, dtype=torch.bfloat16)), {}, ValueError, "bounds must be"),
    ("select", dict(bounds=torch.zeros(4, 2, 3, 128, dtype=torch.bfloat16)), {}, ValueError, "multiple of h_kv"),
    ("select", dict(q=torch.zeros(3, 8, 128)), {}, TypeError, "q must be"),
    ("select", dict(table=_i32(2, 4)), {}, ValueError, "an entry for each of the 3 rows"),
    ("select", dict(lens=_i32(2)), {}, ValueError, "an entry for each of the 3 rows"),
    ("blocks", dict(some=_i32(2, 2, 5)), {}, ValueError, "CUDA|selected must be"),
    ("blocks", dict(table=_i32(2, 4)), {}, ValueError, "an entry for each of the 3 rows"),
    ("weights", dict(lens=_i32(2)), {}, ValueError, "an entry for each of the 3 rows"),
    ("evict", dict(v=torch.zeros(4, 16, 2, 128, dtype=torch.float16)), {}, TypeError, "v_cache"),
    ("evict", dict(v=torch.zeros(4, 8, 2, 128, dtype=torch.bfloat16)), {}, ValueError, "shape mismatch"),
    ("evict", dict(k=torch.zeros(4, 16, 2, 128)), {}, TypeError, "k_cache"),
] + [(c, {}, {}, ValueError, "CUDA") for c in ("bounds", "select", "blocks", "weights", "evict")]


@pytest.mark.parametrize("call,tensors,kw,error,text", BAD)
def test_binding_refuses(lib, call, tensors, kw, error, text):
    with pytest.raises(error, match=text):
        _calls(_tensors(**tensors))[call](**kw)


def test_binding_needs_the_scales():
    x = _tensors()
    with pytest.raises(TypeError, match="k_scale"):
        da.gqa_decode_fp8kv_blocks(x["q"], x["k"], x["v"], None, None, x["table"], x["lens"], x["some"],
                                   scale=0.1, max_seq_len=64)
    with pytest.raises(TypeError, match="k_scale"):
        da.gqa_decode_fp8kv_weights(x["q"], x["k"], x["v"], None, None, x["w"], x["table"], x["lens"],
                                    scale=0.1, max_seq_len=64)


# ------------------------------------------------------------------ the plain forms


def _cache(seed, nb=6, bs=8, h_kv=2, d=16):
    return np.random.default_rng(seed).normal(size=(nb, bs, h_kv, d))


def test_plain_bounds_hold_every_key_and_no_more():
    k = _cache(0)
    table = np.array([[3, 1, 5], [0, 2, -1]])
    got = long_cache.block_bounds(k, table, None, [20, 9], np.full((6, 2, 2, 16), 9.0))
    for b, c, rows in [(0, 0, 8), (0, 1, 8), (0, 2, 4), (1, 0, 8), (1, 1, 1)]:
        x = k[table[b, c], :rows]
        assert (x >= got[table[b, c], 0]).all() and (x <= got[table[b, c], 1]).all()
        assert (x == got[table[b, c], 0]).any(0).all() and (x == got[table[b, c], 1]).any(0).all()
    assert (got[4] == 9.0).all()
    again = long_cache.block_bounds(k, table, [20, 8], [20, 9], np.full((6, 2, 2, 16), 9.0))
    assert (again[[0, 1, 3]] == 9.0).all() and (again[[2, 5]] == got[[2, 5]]).all()


def test_plain_score_bounds_every_product():
    rng = np.random.default_rng(1)
    k, q = _cache(1, bs=30), rng.normal(size=(4, 16))
    for i in range(6):
        s = long_cache.block_score(q, k[i].min((0, 1)), k[i].max((0, 1)))
        assert s >= (k[i].reshape(-1, 16) @ q.T).max()
    assert long_cache.block_score(q, np.full(16, np.nan), np.zeros(16)) == math.inf
    one = k[0, 0, 0]
    assert long_cache.block_score(q, one, one) == pytest.approx((q @ one).max())


def test_plain_choice():
    bounds = np.zeros((9, 2, 1, 4))
    bounds[:, 1, 0, 0] = [5, 1, 7, 7, 2, 7, 0, 3, 4]  # scores of blocks 0 .. 8 for q = e_0
    q = np.zeros((1, 2, 4))
    q[0, 0, 0] = 1
    table = np.arange(9)[None]

    def choose(n, count, first, last):
        return long_cache.select_blocks(q, bounds, table, [n], block_size=8, count=count, first=first,
                                        last=last)[0, 0].tolist()

    assert choose(72, 3, 0, 0) == [2, 3, 5] and choose(72, 2, 0, 0) == [2, 3]
    assert choose(65, 4, 1, 1) == [0, 2, 3, 8] and choose(72, 2, 1, 1) == [0, 8]
    assert choose(20, 5, 1, 1) == [0, 1, 2, -1, -1] and choose(0, 2, 0, 0) == [-1, -1]


def test_plain_attention_weights_and_eviction_agree():
    """Attention over every block is attention; weights of each row sum to one; what is
    evicted is what weighs least."""
    rng = np.random.default_rng(2)
    k, v, q = _cache(3), _cache(4), rng.normal(size=(2, 4, 16))
    table, lens = np.array([[4, 0, 2], [5, 1, -1]]), [21, 16]
    every = np.array([[[0, 1, 2]] * 2, [[0, 1, -1]] * 2])
    a = long_cache.attend(q, k, v, table, lens, scale=0.3)
    b = long_cache.attend(q, k, v, table, lens, scale=0.3, selected=every)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[4][0], b[4][0])
    assert all(np.allclose(w.sum(1), 1) for w in a[4])
    w = long_cache.add_weights(np.full((6, 2, 8), np.nan), a[4], table, lens, [0, 0])
    assert np.isnan(w[3]).all() and np.isnan(w[2, :, 5:]).all()
    assert sum(w[i, :, s].sum() for i, s in [(4, 0)]) == pytest.approx(a[4][0][:, 0].sum())
    twice = long_cache.add_weights(w, a[4], table, lens, [21, 3], decay=0.5)
    assert np.allclose(twice[4], 1.5 * w[4]) and np.allclose(twice[1], w[1])
    k1, v1, w1, new, kept = long_cache.evict(k, v, w, table, lens, keep=10, recent=3, limit=16)
    assert new.tolist() == [-11, 0] and (kept[1] == -1).all()
    for j in range(2):
        assert kept[0, j, -3:].tolist() == [18, 19, 20] and (np.diff(kept[0, j]) > 0).all()
        weight = [w[table[0, t // 8], j, t % 8] for t in range(18)]
        assert min(weight[t] for t in kept[0, j, :-3]) >= max(
            x for t, x in enumerate(weight) if t not in kept[0, j])
        for r, t in enumerate(kept[0, j]):
            assert np.array_equal(k1[table[0, r // 8], r % 8, j], k[table[0, t // 8], t % 8, j])
            assert np.array_equal(v1[table[0, r // 8], r % 8, j], v[table[0, t // 8], t % 8, j])
    assert np.array_equal(k1[[5, 1, 3]], k[[5, 1, 3]])
