"""GPU tests of attention mass over keys with infinite elements."""
import math

import pytest
import torch

import serving_ref as ref
from gpu_util import require_gpu
from test_gpu_paged import paged, queries
from test_gpu_serving import BF, FP

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,kvh,hd,new,window", [
    (8, 2, 64, [1, 1, 1], 1), (32, 8, 128, [1, 0, 1], 1), (3, 1, 128, [1, 1, 1], 1), (6, 2, 64, [9, 3, 2], 7), (5, 1, 128, [30, 1, 7], 20),
    (3, 3, 128, [200, 3, 33], 300), (16, 2, 64, [70, 90, 45], 1000), (71, 1, 64, [2, 2, 5], 3)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_mass_of_infinite_keys(H, kvh, hd, new, window, dtype):
    """A key whose scores are all -inf (an element beyond the type's range, which every query turns away from) receives nothing, in
    whichever tile it lies."""
    dexlib = require_gpu()
    lens = [1000, 300, 555]
    cache, pages, table = paged(dexlib, kvh, hd, 32, lens, dtype)
    q, start = queries(H, hd, new, dtype)
    q[:, :, 5] = q[:, :, 5].abs() + 0.01
    at = [(b, j) for b in range(3) for j in (3, 130, 255, lens[b] - new[b] - 3, lens[b] - new[b] - 150)]
    for b, j in at:
        pages[int(table[b, j // 32]), 0, :, j % 32, 5] = -math.inf
    cache.pages.copy_(pages)
    finite = pages.clone()
    for b, j in at:
        finite[int(table[b, j // 32]), 0, :, j % 32] = 0.0   # (the bound's products stay numbers)
    # lse without them: from the 64-bit scores, where they are -inf
    lse = torch.full((len(q), H), -math.inf)
    for b, n in enumerate(new):
        k = ref.gather(pages, table[b], lens[b])[0]
        for h in range(H):
            s = q[int(start[b]):int(start[b + 1]), h].cpu().double() @ k[:, h // (H // kvh)].T * hd ** -0.5
            seen = torch.arange(lens[b])[None] <= (lens[b] - n + torch.arange(n))[:, None]
            lse[int(start[b]):int(start[b + 1]), h] = s.masked_fill(~seen, -math.inf).logsumexp(1).float()
    want, bound = ref.attention_mass(finite, table, q.cpu(), lse, start, lens, window)
    for b, j in at:
        if new[b]:
            want[b, :, j], bound[b, :, j] = 0.0, 0.0
    mass = cache.attention_mass(q, lse.cuda(), start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), window).cpu()
    ok = ~torch.isnan(want)
    err = (mass.double() - want).abs()[ok]
    assert not torch.isnan(err).any()
    assert bool((err <= bound[ok]).all())
