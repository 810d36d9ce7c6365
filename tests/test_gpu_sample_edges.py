"""GPU tests of sampling at its edges, against 64-bit forms: temperatures from the smallest to the largest that a float
holds, log-probabilities of tokens far below the largest."""
import math

import pytest
import torch

from gpu_util import require_gpu
from test_gpu_serving import BF, F32, FP, sample_case, spread_logits

pytestmark = pytest.mark.gpu

# no limit, small and large top-k, top-p, min-p by itself and with others
LIMITS = [(0, 1.0, 0.0), (50, 1.0, 0.0), (300, 1.0, 0.0), (0, 0.9, 0.0), (50, 0.9, 0.0), (1000, 0.5, 0.01), (0, 1.0, 1e-3), (0, 0.7, 0.3)]


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("n,v", [(7, 37), (7, 5003), (9, 50257), (45, 32001)])
@pytest.mark.parametrize("T", [1e30, 2e30, 1e37, 3e37, 1e38, 3e38])
def test_sample_hot(T, n, v, dtype):
    """So hot that all weights are one: excluded tokens, logits of -inf and what lies behind the vocabulary still have none."""
    x, u = spread_logits(n, v, dtype, v)
    x[1] = -math.inf
    x[1, v // 3:v // 3 + 20] = 1.0          # fewer tokens than top-k leaves
    x[2, ::2] = -math.inf
    x[3, 9:] = -math.inf
    u[0], u[2], u[4] = 1.0 - 2.0 ** -24, 1.0 - 2.0 ** -24, 0.0
    exclude = torch.randint(v, (n, 40), generator=torch.Generator().manual_seed(2)).int()
    exclude[0] = torch.arange(v - 40, v) if v > 40 else exclude[0]   # the last ones
    exclude[4] = torch.arange(40)
    exclude[5] = -1
    if v < 100:
        exclude[:, 5:] = -1
    for k, p, m in LIMITS:
        sample_case(x, u, T, k, p, m)
        got = sample_case(x, u, T, k, p, m, exclude=exclude)
        assert not bool((got[:, None] == exclude)[got >= 0].any()) and bool((got < v).all())


@pytest.mark.parametrize("T", [1e30, 1e36, 1e37, 4e37, 1e38, 3.4e38])
@pytest.mark.parametrize("v", [301, 5003])
def test_sample_hot_and_wide(T, v):
    """Logits that span the range of a float, so that differences overflow and log2(e) / T is subnormal."""
    gen = torch.Generator().manual_seed(v)
    x = (torch.rand((12, v), generator=gen) * 2 - 1) * min(3.4e38, 12 * T)
    x[3, ::3] = -math.inf
    u = torch.rand(12, generator=gen)
    for k, p, m in LIMITS:
        sample_case(x, u, T, k, p, m)


@pytest.mark.parametrize("T", [1.5e-38, 1e-37, 1e-35, 1e-31])
@pytest.mark.parametrize("v", [301, 5003, 40000])
def test_sample_cold_and_narrow(T, v):
    """Logits that differ by some multiples of a temperature next to the smallest normal float."""
    x, u = spread_logits(12, v, F32, v)
    x = x * T                                # (subnormal in part)
    x[5] -= x[5].max()                       # the largest is zero
    for k, p, m in LIMITS:
        sample_case(x, u, T, k, p, m)


@pytest.mark.parametrize("v,below", [(1 << 17, 22.7), (1 << 17, 25.1), (1 << 17, 27.3), (1 << 18, 28.4), (400, 18.5), (3000, 20.0)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_sample_logprob_of_the_tail(v, below, dtype):
    """One peak and a tail of tokens far below it, drawn by a u next to one.  Which of the tail it is hangs on weights of a few units of
    2^-43; its log-probability does not: 2^-19 for the mass (rough weights are off by 2^-21 and 2^-24 ln 2 per octave, of which a
    row's tokens have at most log2 v in the mean, and units by 2^-24) and 2^-22 of its size for log, product and rounding."""
    dexlib = require_gpu()
    gen = torch.Generator().manual_seed(v)
    x = (torch.rand((6, v), generator=gen) * 0.5 - below - 0.25)
    x[:, 0] = 0.0
    x[2:4] += 7.0
    x = x.to(dtype)
    tail = (v - 1) * math.exp(-below)
    u = torch.tensor([1.0 - 2.0 ** -24, 1.0 - min(0.3 * tail, 2.0 ** -18), 1.0 - 2.0 ** -24, 1.0 - 2.0 ** -23, 1.0 - 2.0 ** -24, 0.5])
    tails = 0
    for k, p, m in [(0, 1.0, 0.0), (v - 1, 1.0, 0.0), (0, 1.0, 1e-13), (200, 1.0, 0.0), (0, 1.0 - 2.0 ** -24, 0.0)]:
        logprob = torch.empty(6, device="cuda")
        got = dexlib.sample(x.cuda(), u.cuda(), top_k=k, top_p=p, min_p=m, logprob=logprob).cpu().long()
        w = (x.double() - x.double().max(dim=1, keepdim=True).values).exp()
        down = w.sort(dim=1, descending=True).values[:, :k or v]
        ahead = down.cumsum(dim=1) - down
        left = (down * ((ahead < p * down.sum(dim=1, keepdim=True)) | (p == 1.0))).sum(dim=1)
        want = (w.gather(1, got[:, None])[:, 0] / left).log()
        err = (logprob.cpu().double() - want).abs()
        assert bool((err <= 2.0 ** -19 + 2.0 ** -22 * want.abs()).all()), (k, p, m, err.tolist())
        tails += int((got > 0).sum())
    assert tails >= 6


@pytest.mark.parametrize("T", [4e-39, 1e-41, 1.4e-45])
@pytest.mark.parametrize("v,ties", [(301, 1), (5003, 40), (40000, 700)])
def test_sample_coldest(T, v, ties):
    """Where log2(e) / temperature is no float only tokens of the largest logit have a chance, and share it."""
    x, u = spread_logits(12, v, F32, v)
    for r in range(0, 12, 2):
        x[r, torch.randperm(min(v, 2 * ties), generator=torch.Generator().manual_seed(r))[:ties]] = 30.0 if r < 6 else 0.0
    x[6:, :] -= x[6:].max(dim=1, keepdim=True).values
    for k, p, m in LIMITS:
        got = sample_case(x, u, T, k, p, m)
        assert bool((x.gather(1, got[:, None].long())[:, 0] == x.max(dim=1).values).all())
