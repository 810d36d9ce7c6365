"""GPU tests of sampling at its edges, against the 64-bit form: temperatures from the smallest to the largest that a float
holds."""
import math

import pytest
import torch

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
