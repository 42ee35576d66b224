"""How the GQA decode calls and the serving step's operators are called: what the
binding refuses, without a GPU."""
import pytest
import torch

import gqa_mqa_mla_gb300 as da
from gqa_mqa_mla_gb300 import binding, build

I32 = dict(dtype=torch.int32)


@pytest.mark.parametrize("rows,entries", [(2, 3), (3, 2), (0, 3), (3, 0)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [{}, dict(window=16), dict(window=16, sinks=4)])
def test_decode_refuses_lists_that_are_too_short(rows, entries, fp8, kw):
    """Three rows of q and a table or lengths of fewer: read past their end before."""
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    cache = torch.zeros(4, 16, 2, 128, dtype=torch.uint8 if fp8 else torch.bfloat16)
    scales = [torch.ones(2)] * 2 if fp8 else []
    fn = da.gqa_decode_fp8kv if fp8 else da.gqa_decode
    with pytest.raises(ValueError, match="an entry for each of the 3 rows"):
        fn(q, cache, cache, *scales, torch.zeros(rows, 4, **I32), torch.zeros(entries, **I32),
           scale=0.1, max_seq_len=64, **kw)
    # as many or more: the next check, of the device
    with pytest.raises(ValueError, match="CUDA"):
        fn(q, cache, cache, *scales, torch.zeros(3, 4, **I32), torch.zeros(5, **I32), scale=0.1,
           max_seq_len=64, **kw)


@pytest.mark.parametrize("rows,entries", [(2, 3), (3, 2)])
def test_mla_decode_refuses_lists_that_are_too_short(rows, entries):
    bf16 = dict(dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="an entry for each of the 3 rows"):
        da.mla_decode(torch.zeros(3, 128, 512, **bf16), torch.zeros(3, 128, 64, **bf16),
                      torch.zeros(4, 16, 576, **bf16), torch.zeros(rows, 4, **I32),
                      torch.zeros(entries, **I32), scale=0.1, max_seq_len=64)


@pytest.mark.parametrize("args", [(None, 16, 10), (16, None, 10), (18, 16, 10), (16, 17, 10),
                                  (16, 16, 0), (16, 16, 100001)])
def test_warp_wait_selftest_argument_checks(args):
    assert binding.lib().decattn_selftest_warp_wait(*args, None) == binding.DECATTN_ERR_INVALID_ARG


@pytest.fixture
def no_native_half(monkeypatch):
    """As after an update of PyTorch without a rebuild."""
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.setattr(build, "calls_match", lambda: False)


def test_decode_does_not_need_the_native_half(no_native_half):
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    cache = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 4, **I32), torch.zeros(3, **I32)
    kw = dict(scale=0.1, max_seq_len=64)
    with pytest.warns(RuntimeWarning, match="ctypes"):  # it gets as far as the device
        with pytest.raises(ValueError, match="CUDA"):
            da.gqa_decode(q, cache, cache, table, lens, **kw)
    bad = [dict(table=table[:2]), dict(lens=lens[:2]), dict(v=cache[:, :8].contiguous()),
           dict(q=q.float()), dict(k=cache.half()), dict(table=table.long()),
           dict(q=q[:, :7].contiguous()), dict(k=cache[..., ::2])]
    for b in bad:
        a = dict(dict(q=q, k=cache, v=cache, table=table, lens=lens), **b)
        with pytest.warns(RuntimeWarning), pytest.raises((TypeError, ValueError)) as e:
            da.gqa_decode(a["q"], a["k"], a["v"], a["table"], a["lens"], **kw)
        assert "CUDA" not in str(e.value)
    codes = cache.to(torch.uint8)
    for scales in ([torch.ones(3)] * 2, [torch.ones(2).double()] * 2):
        with pytest.warns(RuntimeWarning), pytest.raises((TypeError, ValueError)) as e:
            da.gqa_decode_fp8kv(q, codes, codes, *scales, table, lens, **kw)
        assert "CUDA" not in str(e.value)
    with pytest.raises(RuntimeError, match="another PyTorch"):  # the step operators do
        da.paged_plan(lens, lens, table, lens, lens[:1], block_size=16, max_tokens=1)
