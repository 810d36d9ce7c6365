"""GPU tests of the paged-cache operators at the edges of their masks, scores and angles."""
import pytest
import torch

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
