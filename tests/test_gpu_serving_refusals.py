"""GPU test of what the paged cache's calls refuse before anything is launched."""
import pytest
import torch

from gpu_util import require_gpu
from test_gpu_paged import paged, queries

pytestmark = pytest.mark.gpu


def test_sizes_that_are_no_whole_numbers():
    dexlib = require_gpu()
    cache, _, _ = paged(dexlib, 2, 64, 16, [20, 9], torch.bfloat16)
    q, start = queries(4, 64, [1, 1], torch.bfloat16)
    seq, lse = torch.tensor([20, 9], dtype=torch.int32, device="cuda"), torch.zeros((2, 4), device="cuda")
    mass = torch.full((2, 2, cache.table.shape[1] * 16), 7.0, device="cuda")
    for bad in (dict(window=1.0), dict(window="1"), dict(window=None), dict(window=1, first=0.0), dict(window=1, scale="1")):
        with pytest.raises(dexlib.DexError) as e:
            cache.attention_mass(q, lse, start.cuda(), seq, mass=mass, **bad)
        assert e.value.code == dexlib.DEX_EINVAL
    for bad in (dict(keep=5.0), dict(keep=None), dict(keep=5, recent=1.5), dict(keep=5, first="0")):
        with pytest.raises(dexlib.DexError) as e:
            cache.evict(mass, seq, **bad)
        assert e.value.code == dexlib.DEX_EINVAL
    torch.cuda.synchronize()
    assert bool((mass == 7.0).all())
