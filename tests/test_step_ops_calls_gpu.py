"""How the serving step's operators are called, on the GPU."""
import pytest
import torch

import gqa_mqa_mla_gb300 as da

from test_step_ops_gpu import _attn_case, _i32, _run_prefill

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
