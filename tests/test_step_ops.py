"""The serving step's operators without a GPU: refusals of the C ABI and of the
binding, the split planners, the rotary table, and the plain forms themselves."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gqa_mqa_mla_gb300 as da
from gqa_mqa_mla_gb300 import binding, build
from oracle import step

FAKE = 0x100000
INVALID, UNSUPPORTED, WORKSPACE = (binding.DECATTN_ERR_INVALID_ARG,
                                   binding.DECATTN_ERR_UNSUPPORTED,
                                   binding.DECATTN_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def _launch(**kw):
    d = dict(batch=2, num_blocks=64, block_size=16, max_blocks_per_seq=16, max_seq_len=256,
             num_splits=1, dtype=binding.DECATTN_BF16, workspace=None, workspace_bytes=0,
             err_flag=None, stream=None)
    d.update(kw)
    return binding.Launch(**d)


# ------------------------------------------------------------------ refusals


@pytest.mark.parametrize("case,expect", [
    (dict(L=None), INVALID),
    (dict(cached=None), INVALID),
    (dict(new=None), INVALID),
    (dict(table=FAKE + 2), INVALID),
    (dict(free=None), INVALID),
    (dict(count_out=FAKE + 1), INVALID),
    (dict(start=None), INVALID),
    (dict(slots=None), INVALID),
    (dict(positions=None), INVALID),
    (dict(tokens=-1), INVALID),
    (dict(L=dict(batch=0)), INVALID),
    (dict(L=dict(batch=8193)), UNSUPPORTED),
    (dict(L=dict(block_size=12)), INVALID),
    (dict(L=dict(block_size=4)), UNSUPPORTED),
    (dict(L=dict(block_size=512)), UNSUPPORTED),
    (dict(L=dict(num_blocks=1 << 28)), UNSUPPORTED),
    (dict(L=dict(max_blocks_per_seq=1 << 27)), UNSUPPORTED),
    (dict(L=dict(err_flag=FAKE + 2)), INVALID),
])
def test_plan_host_checks(lib, case, expect):
    a = dict(cached=FAKE, new=FAKE, table=FAKE, free=FAKE, count=FAKE, count_out=FAKE, lens=FAKE,
             start=FAKE, slots=FAKE, positions=FAKE, tokens=8, L={})
    a.update(case)
    L = None if a["L"] is None else ctypes.byref(_launch(**a["L"]))
    assert lib.paged_plan(a["cached"], a["new"], a["table"], a["free"], a["count"],
                          a["count_out"], a["lens"], a["start"], a["slots"], a["positions"],
                          a["tokens"], L) == expect


def _rope(lib, fp8, **case):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=1024, ks=256, vs=256, k_scale=FAKE, v_scale=FAKE,
             pos=FAKE, rope=da.rope_table([0.1] * 64), slots=FAKE, out=2 * FAKE, kc=FAKE, vc=FAKE,
             tokens=4, h_q=8, h_kv=2, d=128, L={})
    a.update(case)
    L = None if a["L"] is None else ctypes.byref(_launch(**a["L"]))
    rope = None if a["rope"] is None else ctypes.byref(a["rope"])
    scales = [a["k_scale"], a["v_scale"]] if fp8 else []
    fn = lib.gqa_rope_append_fp8kv if fp8 else lib.gqa_rope_append
    return fn(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], *scales, a["pos"], rope,
              a["slots"], a["out"], a["kc"], a["vc"], a["tokens"], a["h_q"], a["h_kv"], a["d"], L)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case,expect", [
    (dict(L=None), INVALID),
    (dict(rope=None), INVALID),
    (dict(q=None), INVALID),
    (dict(k=FAKE + 8), INVALID),
    (dict(v=None), INVALID),
    (dict(pos=None), INVALID),
    (dict(slots=FAKE + 2), INVALID),
    (dict(out=None), INVALID),
    (dict(kc=None), INVALID),
    (dict(tokens=-1), INVALID),
    (dict(tokens=0, q=None), binding.DECATTN_OK),
    (dict(qs=1016), INVALID),   # shorter than a token's row
    (dict(ks=260), INVALID),    # not a multiple of 8
    (dict(out=FAKE, qs=2048), INVALID),  # in place over strided rows
    (dict(h_kv=0), INVALID),
    (dict(d=64), UNSUPPORTED),
    (dict(L=dict(dtype=7)), INVALID),
    (dict(L=dict(block_size=12)), INVALID),
    (dict(L=dict(block_size=512)), UNSUPPORTED),
    (dict(L=dict(num_blocks=0)), INVALID),
])
def test_rope_host_checks(lib, fp8, case, expect):
    assert _rope(lib, fp8, **case) == expect


def test_rope_table_contents_are_checked(lib):
    for field, value, expect in [("rot_dim", 24, UNSUPPORTED), ("rot_dim", 144, UNSUPPORTED),
                                 ("n_axes", 0, INVALID), ("n_axes", 9, INVALID),
                                 ("interleaved", 2, INVALID)]:
        r = da.rope_table([0.1] * 64)
        setattr(r, field, value)
        assert _rope(lib, False, rope=r) == expect
    r = da.rope_table([0.1] * 64)
    r.axis[63] = 1  # an axis that has no positions
    assert _rope(lib, False, rope=r) == INVALID
    assert _rope(lib, True, k_scale=None) == INVALID


def _prefill(lib, fp8, **case):
    a = dict(q=FAKE, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, bt=FAKE, start=FAKE, lens=FAKE,
             out=FAKE, tokens=4, max_q=2, h_q=8, h_kv=2, d=128, scale=0.09, window=0, sinks=0, L={})
    a.update(case)
    L = None if a["L"] is None else ctypes.byref(_launch(**a["L"]))
    scales = [a["k_scale"], a["v_scale"]] if fp8 else []
    fn = lib.gqa_prefill_fp8kv if fp8 else lib.gqa_prefill
    return fn(a["q"], a["k"], a["v"], *scales, a["bt"], a["start"], a["lens"], a["out"],
              a["tokens"], a["max_q"], a["h_q"], a["h_kv"], a["d"], a["scale"], a["window"],
              a["sinks"], L)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case,expect", [
    (dict(L=None), INVALID),
    (dict(q=None), INVALID),
    (dict(k=FAKE + 8), INVALID),
    (dict(bt=None), INVALID),
    (dict(start=None), INVALID),
    (dict(start=FAKE + 2), INVALID),
    (dict(lens=None), INVALID),
    (dict(out=None), INVALID),
    (dict(tokens=-1), INVALID),
    (dict(tokens=0, q=None, out=None), binding.DECATTN_OK),
    (dict(max_q=0), INVALID),
    (dict(h_q=9), INVALID),
    (dict(h_q=130, h_kv=2), UNSUPPORTED),
    (dict(d=64), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID),
    (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID),
    (dict(L=dict(max_seq_len=257)), INVALID),
    (dict(L=dict(num_splits=257)), INVALID),
    (dict(L=dict(num_splits=2)), WORKSPACE),
    (dict(L=dict(num_splits=2, workspace=FAKE, workspace_bytes=64)), WORKSPACE),
    (dict(tokens=1 << 30, L=dict(num_splits=1)), UNSUPPORTED),
])
def test_prefill_host_checks(lib, fp8, case, expect):
    assert _prefill(lib, fp8, **case) == expect


@pytest.mark.parametrize("fp8", [False, True])
def test_sinks_host_checks(lib, fp8):
    def call(window, sinks, **kw):
        scales = [FAKE, FAKE] if fp8 else []
        fn = lib.gqa_decode_fp8kv_sinks if fp8 else lib.gqa_decode_sinks
        return fn(FAKE, FAKE, FAKE, *scales, FAKE, FAKE, FAKE, 8, 2, 128, 0.09, window, sinks,
                  ctypes.byref(_launch(**kw)))

    assert call(0, 4) == INVALID
    assert call(16, -1) == INVALID
    assert call(16, 4, dtype=9) == INVALID
    assert call(100, 100, num_splits=4) == WORKSPACE


def test_binding_refuses_what_the_library_cannot_see():
    cpu = torch.zeros
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):  # tensors of the host
        da.paged_plan(cpu(2, **i32), cpu(2, **i32), cpu(2, 4, **i32), cpu(8, **i32),
                      cpu(1, **i32), block_size=16, max_tokens=4)
    with pytest.raises(TypeError):
        da.paged_plan(cpu(2), cpu(2, **i32), cpu(2, 4, **i32), cpu(8, **i32), cpu(1, **i32),
                      block_size=16, max_tokens=4)
    q = cpu(3, 8, 128, dtype=torch.bfloat16)
    kv = cpu(3, 2, 128, dtype=torch.bfloat16)
    cache = cpu(4, 16, 2, 128, dtype=torch.bfloat16)
    rope = da.rope_table([0.1] * 64)
    good = dict(q=q, k=kv, v=kv, pos=cpu(1, 3, **i32), rope=rope, slots=cpu(3, **i32), kc=cache,
                vc=cache.clone())
    for bad in [dict(pos=cpu(2, 3, **i32)), dict(slots=cpu(2, **i32)), dict(k=kv[:2]),
                dict(q=q.transpose(1, 2)), dict(kc=cache[:, :, :1].contiguous())]:
        a = dict(good, **bad)
        with pytest.raises((ValueError, TypeError)):
            da.gqa_rope_append(a["q"], a["k"], a["v"], a["pos"], a["rope"], a["slots"], a["kc"],
                               a["vc"])
    start, lens, bt = cpu(3, **i32), cpu(2, **i32), cpu(2, 4, **i32)
    for kw in [dict(sinks=4), dict(sinks=-1), dict(window=0)]:
        with pytest.raises(ValueError):
            da.gqa_prefill(q, cache, cache, bt, start, lens, scale=0.1, max_q_len=3,
                           max_seq_len=64, **kw)
    with pytest.raises(ValueError):
        da.gqa_prefill(q, cache, cache, bt, start[:2], lens, scale=0.1, max_q_len=3,
                       max_seq_len=64)
    with pytest.raises(ValueError):
        da.gqa_decode(q, cache, cache, bt, lens, scale=0.1, max_seq_len=64, sinks=4)


# ------------------------------------------------------------------ planners


def test_sinks_planner_plans_for_the_window_and_the_sinks(lib):
    for B, h_q, h_kv, S, W, N, bs in [(1, 64, 8, 131072, 4096, 4, 16), (4, 32, 8, 65536, 1024, 200, 128),
                                      (64, 64, 8, 8192, 4096, 4096, 16), (3, 16, 2, 100, 50, 49, 16)]:
        span = S if W + N >= S else min(S, W + min(bs, 64) - 1) + -(-N // 64) * 64
        for kv_bytes, plan in ((2, binding.gqa_plan_splits), (1, binding.gqa_fp8_plan_splits)):
            got = da.gqa_sinks_plan_splits(B, h_q, h_kv, S, W, N, bs, kv_bytes, num_sms=152)
            base = plan(B, h_q, h_kv, span, num_sms=152)
            assert base <= got <= max(base, 8)
            if W + N >= S or span < 6 * 64:
                assert got == base
    # few sequences in a window: up to eight splits of two tiles or more, one wave
    for kv_bytes in (1, 2):
        assert da.gqa_sinks_plan_splits(18, 5, 1, 20000, 1335, 1, 8, kv_bytes, num_sms=152) == 8
        assert da.gqa_sinks_plan_splits(1, 8, 1, 8192, 448, 4, 16, kv_bytes, num_sms=152) == 4
        assert da.gqa_sinks_plan_splits(64, 32, 8, 8192, 1000, 4, 16, kv_bytes, num_sms=152) == 1
    # no sinks: the windowed planner; lengths near the integers' limit stay in range
    assert da.gqa_sinks_plan_splits(2, 8, 2, 4096, 100, 0, 16, num_sms=152) == \
        binding.gqa_window_plan_splits(2, 8, 2, 4096, 100, 16, num_sms=152)
    assert da.gqa_sinks_plan_splits(1, 8, 2, 2**31 - 1, 2**30, 2**30 - 8, 16, num_sms=152) >= 1
    with pytest.raises(da.DecAttnError):
        da.gqa_sinks_plan_splits(2, 8, 2, 4096, 100, -1, 16, num_sms=152)


def test_prefill_planner_splits_few_rows_and_leaves_many_alone(lib):
    assert da.gqa_prefill_plan_splits(1, 8192, 8192, 64, 8, 8192, num_sms=152) == 1
    assert da.gqa_prefill_plan_splits(1, 4, 4, 64, 8, 131072, num_sms=152) > 4
    for args in [(1, 1, 1, 8, 8, 0), (32, 200, 8, 64, 8, 8192), (5, 70, 33, 5, 1, 129)]:
        ns = da.gqa_prefill_plan_splits(*args, num_sms=152)
        assert 1 <= ns <= binding.MAX_SPLITS
    # a window bounds what there is to split
    assert da.gqa_prefill_plan_splits(1, 4, 4, 64, 8, 131072, 100, 4, num_sms=152) <= 3
    assert da.gqa_prefill_workspace_size(10, 8, 1) == 0
    assert da.gqa_prefill_workspace_size(10, 8, 3) >= 10 * 8 * 3 * 129 * 4


# ------------------------------------------------------------------ rotary table


def test_rope_table_reduces_far_positions_exactly(lib):
    """turns[i] * position modulo 2^64 is the phase: compared, at positions up
    to 2^31, with exact rational arithmetic on the double frequency over the
    double 2 pi (the quotient's rounding is 2^-53 of the frequency)."""
    freq = [1e6 ** (-i / 64) for i in range(64)]
    r = da.rope_table(freq, sections=(16, 24, 24))
    assert [list(r.axis).count(a) for a in range(3)] == [16, 24, 24]
    assert list(r.axis[:16]) == [0] * 16 and r.n_axes == 3 and r.rot_dim == 128
    for i in (0, 1, 31, 63):
        for pos in (1, 2, 8191, 131071, 10**7, 2**31 - 1, -1, -(2**31)):
            phase = (pos * r.turns[i]) % 2**64 / 2**64
            want = math.fmod(pos * (freq[i] / (2 * math.pi)), 1.0) % 1.0
            d = abs(phase - want)
            # the table and the product each round by 2^-53 of |pos| f / 2 pi
            assert min(d, 1 - d) <= 4 * 2.0**-53 * max(1.0, abs(pos) * freq[i]), (i, pos)


def test_rope_table_refusals(lib):
    for kw in [dict(inv_freq=[0.1] * 7), dict(inv_freq=[]), dict(inv_freq=[0.1] * 72),
               dict(inv_freq=[float("inf")] * 64), dict(inv_freq=[0.1] * 64, sections=(32, 31)),
               dict(inv_freq=[0.1] * 64, sections=(65, -1)),
               dict(inv_freq=[0.1] * 64, sections=(8,) * 9)]:
        with pytest.raises(da.DecAttnError):
            da.rope_table(**kw)
    r = da.rope_table(torch.tensor([0.5] * 16), sections=(0, 16, 0), interleaved=True)
    assert list(r.axis[:16]) == [1] * 16 and r.interleaved == 1
    # a whole number of turns per position does not turn at all
    assert da.rope_table([2 * math.pi] * 8).turns[0] == 0


# ------------------------------------------------------------------ the plain forms


def test_plain_plan_keeps_the_pool_whole():
    """Every block is in exactly one place before and after a step."""
    rng = np.random.default_rng(0)
    for trial in range(30):
        bs, M, B = int(rng.choice([8, 16, 64])), 9, int(rng.integers(1, 12))
        cached = rng.integers(0, M * bs + 1, B)
        new = [int(rng.integers(-c, M * bs - c + 1)) for c in cached]
        held = -(-cached // bs)
        nb = int(held.sum() + rng.integers(0, 40))
        ids = rng.permutation(nb)
        table = np.full((B, M), -1)
        at = 0
        for b in range(B):
            table[b, :held[b]] = ids[at:at + held[b]]
            at += held[b]
        free = np.full(nb, -1)
        free[:nb - at] = ids[at:]
        tokens = int(rng.integers(0, 300))
        r = step.paged_plan(cached, new, table, free, nb - at, block_size=bs, max_tokens=tokens)
        now = -(-r["seq_lens"] // bs)
        own = [int(r["table"][b, k]) for b in range(B) for k in range(now[b])]
        own += [int(i) for i in r["free"][:r["count"]]]
        assert sorted(own) == list(range(nb))
        live = r["slots"][r["slots"] >= 0]
        assert len(set(live.tolist())) == len(live) == r["q_start"][-1]


def test_plain_attention_is_softmax_attention():
    """One sequence, identity table: torch's own softmax in 64 bits; and a
    window that covers everything, sinks that cover everything, change nothing."""
    g = torch.Generator().manual_seed(3)
    n, L, h_q, h_kv = 5, 21, 4, 2
    q = torch.randn(n, h_q, 128, generator=g, dtype=torch.float64)
    k, v = (torch.randn(3, 8, h_kv, 128, generator=g, dtype=torch.float64) for _ in range(2))
    args = (q.numpy(), k.numpy(), v.numpy(), [[0, 1, 2]], [0, n], [L])
    out, spread, _, _ = step.attend(*args, scale=0.1)
    K = k.reshape(-1, h_kv, 128)[:L].repeat_interleave(2, 1)
    V = v.reshape(-1, h_kv, 128)[:L].repeat_interleave(2, 1)
    s = torch.einsum("ihd,thd->hit", q, K) * 0.1
    hidden = torch.arange(L)[None] > torch.arange(L - n, L)[:, None]
    ref = torch.einsum("hit,thd->ihd", s.masked_fill(hidden, -math.inf).softmax(-1), V)
    assert np.abs(out - ref.numpy()).max() < 1e-12
    assert (np.abs(out) <= spread + 1e-12).all()
    for kw in [dict(window=L), dict(window=1, sinks=L), dict(window=10, sinks=L - 10)]:
        assert np.abs(step.attend(*args, scale=0.1, **kw)[0] - out).max() < 1e-12
    assert np.abs(step.attend(*args, scale=0.1, window=4, sinks=2)[0] - out).max() > 1e-3


def test_plain_rotation_preserves_lengths_and_relative_positions():
    g = np.random.default_rng(4)
    x = g.standard_normal((1, 1, 32))
    y = g.standard_normal((1, 1, 32))
    f, a = [10.0 ** -i for i in range(8)], [0] * 4 + [1] * 4
    for inter in (False, True):
        def turn(z, p):
            return step.rope(z, np.array([[p], [2 * p]]), f, a, inter)[0, 0]
        assert abs(np.linalg.norm(turn(x, 77)) - np.linalg.norm(x)) < 1e-12
        assert abs(turn(x, 105) @ turn(y, 100) - turn(x, 5) @ turn(y, 0)) < 1e-10
        assert np.array_equal(turn(x, 9)[16:], x[0, 0, 16:])


def test_prefill_refuses_lengths_whose_tiles_pass_31_bits(lib):
    for n, expect in [(2**31 - 1, UNSUPPORTED), (2**31 - 4096, UNSUPPORTED)]:
        assert _prefill(lib, False, L=dict(max_seq_len=n, max_blocks_per_seq=2**28)) == expect


def test_prefill_planner_is_the_same_for_windows_that_hide_nothing():
    """The library drops such a window before it plans: a workspace sized by the
    planner's answer fits either way."""
    for B, n, S, h_q, h_kv in [(1, 4, 8192, 64, 8), (3, 200, 1000, 32, 8), (2, 1, 64, 8, 8)]:
        plain = da.gqa_prefill_plan_splits(B, B * n, n, h_q, h_kv, S, num_sms=152)
        for window, sinks in [(S, 0), (S + 5, 7), (2**31 - 1, 2**31 - 1)]:
            assert da.gqa_prefill_plan_splits(B, B * n, n, h_q, h_kv, S, window, sinks,
                                              num_sms=152) == plain
            for kv in (1, 2):
                sink_plan = da.gqa_sinks_plan_splits(B, h_q, h_kv, S, window, sinks, 16, kv,
                                                     num_sms=152)
                plan = binding.gqa_plan_splits if kv == 2 else binding.gqa_fp8_plan_splits
                assert sink_plan == plan(B, h_q, h_kv, S, num_sms=152)
