"""How the serving step's operators are called, on the GPU."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import gqa_mqa_mla_gb300 as da
from gqa_mqa_mla_gb300 import binding
from oracle import step

from test_step_ops_gpu import (DEV, HALF, TYPES, _attn_case, _close, _fp16_probs, _gen, _i32,
                               _plain_prefill, _plan_case, _run_plan, _run_prefill, _same_plan)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ row offsets


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch,at,rows", [(64, 5, 1), (64, 0, 1), (64, 63, 1), (33, 0, 2),
                                           (1000, 7, 1), (1000, 998, 1), (200, 3, 40)])
def test_prefill_flags_bad_offsets_of_any_sequence(batch, at, rows, fp8):
    """One chunk that is longer than said, or an offset that decreases, and nothing
    else wrong, wherever in the batch it stands."""
    q_lens = [rows] * batch
    q_lens[at] = rows + 3
    x = _attn_case(q_lens, [n + 20 for n in q_lens], 8, 4, "bf16", 16, 800, fp8=fp8)
    assert _run_prefill(x)[1] == 0
    start = x["start"].cpu().numpy()
    for splits in (1, 0, 2):
        out = torch.full_like(x["q"], 7.0)
        _, flag = _run_prefill(dict(x, max_q=rows), out=out, num_splits=splits)
        assert flag == da.FLAG_BAD_SEQ_LEN
        assert bool((out[start[at]: start[at + 1]] == 7).all())
        bad = start.copy()
        bad[at + 1] = bad[at] - 1
        _, flag = _run_prefill(dict(x, start=_i32(bad)), num_splits=splits)
        assert flag == da.FLAG_BAD_SEQ_LEN


# ------------------------------------------------------------------ the plan


def _plan_once(B):
    rng = np.random.default_rng(B)
    case = _plan_case(rng, B, 16, 4, -20, 40, 4 * B)
    want = step.paged_plan(*case, block_size=16, max_tokens=20 * B)
    _same_plan(_run_plan(*case, 16, 20 * B), want)


@pytest.mark.parametrize("B", [2416, 2417, 2418, 2440, 2457, 2458, 8192])
def test_plan_batches_around_the_default_shared_memory(B):
    _plan_once(B)


@pytest.mark.parametrize("B", [2418, 2457, 8192])
def test_plan_as_the_first_call_of_a_process(B):
    here = os.path.dirname(os.path.abspath(__file__))
    code = (f"import sys; sys.path[:0] = [{here!r}, {os.path.dirname(here)!r}]\n"
            f"import test_step_ops_calls_gpu as t; t._plan_once({B})")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_plans_of_different_sizes_from_two_threads():
    """The launches' shared memory does not depend on what another thread plans."""
    failed = []

    def work(B, n):
        try:
            rng = np.random.default_rng(B)
            cached, new, table, free, count = _plan_case(rng, B, 16, 4, -20, 40, 4 * B)
            t, f, c = _i32(table), _i32(free), _i32([count])
            args = (_i32(cached), _i32(new))
            for _ in range(n):
                da.paged_plan(*args, t.clone(), f.clone(), c, block_size=16, max_tokens=16)
            torch.cuda.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append((B, e))

    threads = [threading.Thread(target=work, args=(B, 400)) for B in (2600, 8192, 3000, 100)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


# ------------------------------------------------------------------ streams


def test_results_on_a_given_stream_may_be_used_on_the_current_one():
    """A result that was allocated for a call on another stream, then read on the
    current one and dropped, is not handed to that stream's next work while the
    current one still reads it."""
    x = _attn_case([1, 1, 1], [900, 90, 700], 16, 4, "bf16", 16, 820)
    rope = da.rope_table([0.5] * 64)
    slots = _i32([-1, -1, -1])
    kv = torch.randn((3, 4, 128), generator=_gen(1), device=DEV).bfloat16()
    pos = _i32([[3, 4, 5]])
    table, new, free, top = x["table"].clone(), _i32([1, 1, 1]), _i32([0, 1, 2, 3]), _i32([4])
    calls = {
        "decode": lambda **kw: da.gqa_decode(x["q"], *x["caches"], x["table"], x["lens"], scale=0.1,
                                             max_seq_len=900, **kw),
        "prefill": lambda **kw: da.gqa_prefill(x["q"], *x["caches"], x["table"], x["start"],
                                               x["lens"], scale=0.1, max_q_len=1, max_seq_len=900,
                                               **kw),
        "rope": lambda **kw: da.gqa_rope_append(x["q"], kv, kv, pos, rope, slots, *x["caches"], **kw),
        "plan": lambda **kw: da.paged_plan(x["lens"], new, table, free, top, block_size=16,
                                           max_tokens=4, **kw).positions,
    }
    s = torch.cuda.Stream()
    for name, call in calls.items():
        want = call()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        got = call(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(20_000_000)  # what reads the result runs in some ms
        seen = got.clone()
        size = got.untyped_storage().nbytes()
        del got
        with torch.cuda.stream(s):
            spoil = [torch.full((size,), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(6)]
        torch.cuda.synchronize()
        assert torch.equal(seen, want) and len(spoil) == 6, name


def test_a_workspace_may_be_any_dense_tensor():
    """Strides in another order hold the same bytes."""
    x = _attn_case([1, 1, 1], [900, 90, 700], 16, 4, "bf16", 16, 821)
    ws = torch.empty(512, 512, dtype=torch.uint8, device=DEV).t()
    assert not ws.is_contiguous()
    kw = dict(scale=0.1, max_seq_len=900, num_splits=4)
    args = (x["q"], *x["caches"], x["table"])
    assert torch.equal(da.gqa_decode(*args, x["lens"], workspace=ws, **kw),
                       da.gqa_decode(*args, x["lens"], **kw))
    assert torch.equal(da.gqa_prefill(*args, x["start"], x["lens"], max_q_len=1, workspace=ws, **kw),
                       da.gqa_prefill(*args, x["start"], x["lens"], max_q_len=1, **kw))
    for bad in (ws[::2], torch.empty(1, dtype=torch.uint8, device=DEV).expand(2**18)):
        with pytest.raises(ValueError):
            da.gqa_decode(*args, x["lens"], workspace=bad, **kw)


# ------------------------------------------------------------------ without the native half


@pytest.mark.parametrize("native", [True, False])
def test_a_call_on_the_default_stream_from_another(monkeypatch, native):
    """Stream handle 0 is the default stream, not a new one: the call comes behind the
    work that makes its input there."""
    x = _attn_case([1, 1, 1], [900, 90, 700], 16, 4, "bf16", 16, 823)
    if not native:
        monkeypatch.setattr(binding, "_calls", None)
        monkeypatch.setattr(binding._build, "calls_match", lambda: False)
        monkeypatch.setattr(binding.warnings, "warn", lambda *a, **k: None)
    q, spoilt = x["q"].clone(), torch.full_like(x["q"], 3.0)
    call = lambda t, **kw: da.gqa_decode(t, *x["caches"], x["table"], x["lens"],  # noqa: E731
                                         scale=0.1, max_seq_len=900, **kw)
    want = call(q)
    torch.cuda.synchronize()
    for handle in (0, torch.cuda.default_stream()):
        t = spoilt.clone()
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        t.copy_(q)
        with torch.cuda.stream(torch.cuda.Stream()):
            out = call(t, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_through_ctypes_gives_the_same(monkeypatch, fp8):
    x = _attn_case([1, 1, 1], [900, 90, 700], 16, 4, "bf16", 16, 822, fp8=fp8)
    fn = da.gqa_decode_fp8kv if fp8 else da.gqa_decode
    args = (x["q"], *x["caches"], *(x["scales"] or []), x["table"], x["lens"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    forms = [{}, dict(num_splits=3), dict(window=300), dict(window=300, sinks=4),
             dict(num_splits=4, window=800, sinks=70), dict(stream=s), dict(stream=s.cuda_stream),
             dict(out=torch.zeros(4, 16 * 128, dtype=torch.bfloat16, device=DEV)),
             dict(num_splits=4, workspace=torch.empty(2**18, device=DEV))]
    kw = dict(scale=0.09, max_seq_len=900)
    want = [fn(*args, **kw, **f).clone() for f in forms if "stream" not in f]
    torch.cuda.synchronize()
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.setattr(binding._build, "calls_match", lambda: False)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        got = [fn(*args, **kw, **f) for f in forms]
        torch.cuda.synchronize()
        bad = [dict(max_seq_len=10**6), dict(num_splits=-1), dict(num_splits=4, workspace=x["q"][0])]
        for b in bad:
            with pytest.raises(da.DecAttnError):
                fn(*args, **{**kw, **b})
        ws = torch.empty(512, 512, dtype=torch.uint8, device=DEV)
        assert torch.equal(fn(*args, **kw, num_splits=3, workspace=ws.t()), want[1])
        for b in (dict(out=x["q"].float()), dict(out=x["q"].cpu()), dict(out=x["q"][:1]),
                  dict(workspace=ws[::2]), dict(workspace=ws[:1].expand(512, 512)),
                  dict(workspace=3), dict(workspace=ws.cpu()), dict(err_flag=3),
                  dict(err_flag=ws[0, :3])):
            with pytest.raises((TypeError, ValueError)):
                fn(*args, **{**kw, **b})
    same = [o for o, f in zip(got, forms) if "stream" not in f]
    assert all(torch.equal(a, b) for a, b in zip(same, want))
    assert all(torch.equal(o, want[0]) for o, f in zip(got, forms) if "stream" in f)


# ------------------------------------------------------------------ 8-bit cache


def test_pieces_of_two_tiles_and_of_one_in_turn_over_an_8_bit_cache():
    """CTAs that go from a piece with two Q tiles and a single K / V tile to one with
    one Q tile and several: each row keeps the exponent of its own query (the rows'
    sizes differ by up to 2^12)."""
    rng = np.random.default_rng(30)
    q_lens, lens = [], []
    for _ in range(160):
        q_lens += [32, int(rng.integers(1, 16))]
        lens += [int(rng.integers(32, 128)), int(rng.integers(260, 500))]
    for dtype in ("bf16", "fp16"):
        x = _attn_case(q_lens, lens, 16, 2, dtype, 16, 830, fp8=True)
        size = 2.0 ** torch.randint(-8, 5, (x["q"].shape[0], 16, 1), generator=_gen(3), device=DEV)
        x["q"] = (x["q"].float() * size / 4).to(x["q"].dtype)
        out, flag = _run_prefill(x, num_splits=1)
        assert flag == 0
        for _ in range(5):
            again, _ = _run_prefill(x, num_splits=1)
            assert torch.equal(again, out)
        start = np.concatenate([[0], np.cumsum(q_lens)])
        for b in range(0, 320, 41):
            rows = slice(int(start[b]), int(start[b + 1]))
            y = dict(x, q=x["q"][rows], table=x["table"][b: b + 1], start=_i32([0, q_lens[b]]),
                     lens=x["lens"][b: b + 1])
            _close(out[rows], _fp16_probs(_plain_prefill(y), dtype), dtype, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("wide", [False, True])
def test_what_the_terms_of_a_query_lose(wide, dtype):
    """A row whose largest value is just above 1.75 * 2^k and whose others lie on half
    of the terms' smallest step loses as much as a row can: each value is off by at
    most 2^-10 / 224 (2^-17.8) of the largest.  Two tokens, V = 1 and 0: the output is
    the first one's weight, 1 / (1 + e^-s), so its score s can be read off."""
    big = 1.7578125  # a value of both types; scaled by 2^7 to 225, the other values to 2^-10
    small = 2.0**-17
    h_q = 33 if wide else 2
    q = torch.full((1, h_q, 128), small, dtype=TYPES[dtype], device=DEV)
    q[:, :, 0] = big
    k = torch.zeros((1, 16, 1, 128), device=DEV)
    k[0, 0, 0, 1:] = 448.0
    v = torch.zeros((1, 16, 1, 128), device=DEV)
    v[0, 0] = 1.0
    codes = [c.to(torch.float8_e4m3fn).view(torch.uint8) for c in (k, v)]
    one = torch.ones(1, device=DEV)
    if wide:
        out = da.gqa_decode_fp8kv(q, *codes, one, one, _i32([[0]]), _i32([2]), scale=1.0,
                                  max_seq_len=2)
    else:
        out = da.gqa_prefill_fp8kv(q, *codes, one, one, _i32([[0]]), _i32([0, 1]), _i32([2]),
                                   scale=1.0, max_q_len=1, max_seq_len=2)
    got = out.double().cpu().numpy()
    score = 127 * small * 448
    bound = 2.0**-10 / 224 * big * 127 * 448
    lo, hi = (1 / (1 + np.exp(-(score + e))) for e in (-bound, bound))
    u = HALF[dtype]  # the output's rounding; the probabilities' (fp16), exp2 and the sums: 2^-10
    assert (got >= lo * (1 - u - 2.0**-10)).all() and (got <= hi * (1 + u + 2.0**-10)).all()


# ------------------------------------------------------------------ waits


@pytest.mark.parametrize("limit_us", [200, 2000])
def test_a_wait_that_runs_out_for_some_lanes_does_for_the_warp(limit_us):
    """Else the others would wait for them in the warp's next collective."""
    flag, lanes = binding.selftest_warp_wait(limit_us)
    assert flag == da.FLAG_TIMEOUT and lanes == [0, 0, 32, 32]
