"""CPU tests of what eviction refuses beside sizes and null pointers."""
import ctypes as C

import pytest

import lossless_depth_adaptive_gb300 as dexlib
from test_paged_host import kv, library   # noqa: F401  (library: the fixture that builds it)
from test_serving_host import evict_args


@pytest.mark.parametrize("at", [4, -4, 0])
def test_new_len_may_not_overlap_seq_len(at):
    """Heads of a sequence read its length while another one's may already be written."""
    c = kv(batch=3)
    assert dexlib.lib().dex_paged_evict(C.byref(c), C.byref(evict_args(new_len=(1 << 24) + at)), None, None) == dexlib.DEX_EINVAL
    assert dexlib.lib().dex_paged_evict(C.byref(c), C.byref(evict_args(new_len=(1 << 24) + 2 * at)), None, None) == dexlib.DEX_EINVAL
