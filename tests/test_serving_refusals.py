"""CPU tests of what eviction and sampling refuse beside sizes and null pointers."""
import ctypes as C

import pytest
import torch

import lossless_depth_adaptive_gb300 as dexlib
from test_paged_host import kv, library   # noqa: F401  (library: the fixture that builds it)
from test_serving_host import evict_args


@pytest.mark.parametrize("at", [4, -4, 0])
def test_new_len_may_not_overlap_seq_len(at):
    """Heads of a sequence read its length while another one's may already be written."""
    c = kv(batch=3)
    assert dexlib.lib().dex_paged_evict(C.byref(c), C.byref(evict_args(new_len=(1 << 24) + at)), None, None) == dexlib.DEX_EINVAL
    assert dexlib.lib().dex_paged_evict(C.byref(c), C.byref(evict_args(new_len=(1 << 24) + 2 * at)), None, None) == dexlib.DEX_EINVAL


@pytest.mark.parametrize("bad", [dict(top_k=50.0), dict(top_k="50"), dict(temperature="hot"), dict(temperature=None), dict(top_p=1j),
                                 dict(min_p=[0.1, 0.2, 0.3])])
def test_settings_that_are_no_numbers(bad):
    with pytest.raises(dexlib.DexError) as e:
        dexlib.sample(torch.zeros((3, 10)), torch.zeros(3), **bad)
    assert e.value.code == dexlib.DEX_EINVAL and next(iter(bad)) in str(e.value)
