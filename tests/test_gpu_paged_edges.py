"""GPU tests of the paged-cache operators at the edges of their masks, scores and angles."""
import math

import pytest
import torch

from gpu_util import require_gpu
from paged_ref import HALF
from test_gpu_paged import BF, FP, SHARED, run_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,kvh,hd,ps,new,prefix", SHARED)
def test_tree_bits_beyond_the_queries(H, kvh, hd, ps, new, prefix):
    """Bits of a word at and above the sequence's number of queries select nothing, whether the prefix is read once
    or by every sequence, behind it, in it and at length zero."""
    g = torch.Generator().manual_seed(prefix + 3)
    lens = [prefix + n + 40 * (b % 2) for b, n in enumerate(new)]
    lens[1] = prefix // 2
    lens[2] = 0
    lens[-1] = 30
    words = [-1 if i % 3 else (int(torch.randint(0, 1 << n, (1,), generator=g)) | -(1 << n)) for n in new for i in range(n)]
    tree = torch.tensor(words, dtype=torch.int64)
    run_case(H, kvh, hd, ps, FP, lens, new, prefix, tree)
    run_case(H, kvh, hd, ps, BF, [min(n, 90) for n in lens], new, 0, tree)


def test_tree_bits_of_full_words():
    """64 queries of a sequence: every bit of a word counts."""
    g = torch.Generator().manual_seed(6)
    words = torch.randint(-2 ** 63, 2 ** 63 - 1, (64 + 3,), generator=g)
    words[5], words[64], words[66] = -1, -1, -(1 << 62)
    run_case(8, 2, 64, 16, FP, [64, 10], [64, 3], tree=words)
    run_case(8, 2, 128, 32, BF, [264, 203], [64, 3], 200, tree=words)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("big", [2.0 ** 11, 2.0 ** 12, 2.0 ** 13, 2.0 ** 14, 2.0 ** 15])
@pytest.mark.parametrize("n", [1, 6, 20, 40])
def test_scores_of_any_size(n, big, dtype):
    """Scores whose fp32 neighbours lie far apart: two keys one step of the sum (8 at 2^26) from each other.  The larger
    one takes all the weight, and no probability overflows on the way."""
    dexlib = require_gpu()
    kvh, G, hd, ps, length, batch = 2, 4, 64, 64, 400, 120   # segments of four tiles, one or two per thread block
    gen = torch.Generator().manual_seed(7)
    step = max(8.0, big * big * 2.0 ** -23)
    for scale in (2.0, 2.0 + 2.0 ** -21, 2.0 + 2.0 ** -20, 2.0 + 3 * 2.0 ** -21, -2.0):
        pages = torch.zeros((7, 2, kvh, ps, hd), dtype=dtype)
        pages[:, 1] = torch.randn((7, kvh, ps, hd), generator=gen).to(dtype)
        sign = math.copysign(1.0, scale)
        pages[0, 0, :, 5, 0] = sign * big
        pages[4, 0, :, 10, 0] = sign * big      # position 266: the larger one, by its second dimension
        pages[4, 0, :, 10, 1] = sign * step
        table = torch.arange(7, dtype=torch.int32).expand(batch, 7).contiguous()
        cache = dexlib.PagedCache(pages.cuda(), table.cuda())
        q = torch.zeros((batch * n, kvh * G, hd), dtype=dtype)
        q[:, :, 0], q[:, :, 1] = big, 1.0
        start = (torch.arange(batch + 1) * n).int()
        lse = torch.zeros(q.shape[:2], device="cuda")
        out = cache.attention(q.cuda(), start.cuda(), torch.full((batch,), length, dtype=torch.int32, device="cuda"), n, lse=lse,
                              scale=scale).cpu()
        want = pages[4, 1, :, 10].repeat_interleave(G, 0)   # the other's weight is exp(-16) and less
        want = want.double()[None]
        # half a step of the result and one of the probability, 2 exp(-16) of values up to 5
        assert bool(((out.double() - want).abs() <= want.abs() * (2.01 * HALF[dtype]) + 10 * math.exp(-16.0)).all())
        top = (big * big + step) * abs(scale)
        assert bool(((lse.cpu().double() - top).abs() <= top * 2.0 ** -21).all())
