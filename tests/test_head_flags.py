"""What the head's calls accept and refuse beside test_head_ref's cases, without a GPU."""
import pytest

from bwd_ssm_conv_gb300 import binding, head
from bwd_ssm_conv_gb300.build import build
from test_block_ref import INV, UNS
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


@pytest.mark.parametrize("io,size", [(0, 4), (1, 2)])
def test_rows_of_w_too_far_apart_are_refused_before_anything_runs(H, io, size):
    """A vocabulary of one has no second row, but its stride still goes into a descriptor of 40 bits."""
    for name, (call, _, _) in _calls(H, io=io, vocab=1).items():
        assert call(ld_w=(1 << 40) // size) == UNS and call(ld_w=(1 << 40) // size + 8) == UNS, name
        assert call(ld_w=(1 << 40) // size - 8, ws=(None, 0)) not in (INV, UNS), name
