"""Calls of the operators for long caches that their documentation allows, beside those of
test_long_cache_gpu.py, against the same plain forms in 64 bits with the same tolerances."""

import numpy as np
import pytest
import torch

import gqa_mqa_mla_gb300 as da
from gqa_mqa_mla_gb300 import binding

from test_long_cache_gpu import _attend, _case, _close, _decode, _flag, _i32, _lists, _weights_close

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


# ------------------------------------------------------------------ a call that gave up


@pytest.mark.parametrize("limit_us", [200, 2000])
def test_a_split_that_gave_up_is_marked_in_every_row(limit_us):
    """(What the second launch does with such a split is tested with bad block ids, whose
    mark is the same.)"""
    flag, rows = binding.selftest_gave_up(limit_us)
    want = torch.arange(40.0)[:, None].repeat(1, 3)
    want[:, 1] = float("inf")
    assert flag == da.FLAG_TIMEOUT and torch.equal(rows, want)
