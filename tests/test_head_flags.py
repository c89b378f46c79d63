"""What the head's calls accept and refuse beside test_head_ref's cases, without a GPU."""
import pytest

from bwd_ssm_conv_gb300 import binding, head
from bwd_ssm_conv_gb300.build import build
from test_block_ref import INV
from test_head_ref import _calls


@pytest.fixture(scope="module")
def H():
    build()
    return head.lib()


@pytest.mark.parametrize("flags,known", [(0, True), (head.SSM_HEAD_FINE_G, True),
                                         (head.SSM_HEAD_FINE_G | binding.SSM_DEBUG_NO_WAIT, True),
                                         (4, False), (head.SSM_HEAD_FINE_G | 1, False), (1 << 31, False)])
def test_flags(H, flags, known):
    for name, (call, _, _) in _calls(H, flags=flags).items():
        # the workspace refuses what the flags do not (its size cannot be known without a GPU)
        assert (call(ws=(None, 0)) == INV) == (not known), name
