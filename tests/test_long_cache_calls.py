"""The self test of a split that gave up, without a GPU: its refusals."""
import pytest

from gqa_mqa_mla_gb300 import binding, build

FAKE = 0x100000


@pytest.mark.parametrize("args", [(None, FAKE, 1000), (FAKE, None, 1000), (FAKE + 2, FAKE, 1000),
                                  (FAKE, FAKE + 1, 1000), (FAKE, FAKE, 0), (FAKE, FAKE, 100001)])
def test_gave_up_selftest_argument_checks(args):
    build.build()
    assert binding.lib().decattn_selftest_gave_up(*args, None) == binding.DECATTN_ERR_INVALID_ARG
