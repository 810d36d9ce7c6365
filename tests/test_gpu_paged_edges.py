"""GPU tests of the paged-cache operators at the edges of their masks, scores and angles."""
import decimal
import math

import pytest
import torch

import test_gpu_paged
from gpu_util import require_gpu
from paged_ref import HALF, attention, gather
from test_gpu_paged import BF, FP, SHARED, compare, paged, queries, run_case

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


def below_a_peak(G, hd, dtype, n, batch, length, nats, at, prefix=0, sign=1.0):
    """A key at each position of `at` whose score lies `nats` above all the others' and whose value is zero: the result
    is what the others' weights, exp(-nats) and less each, add up to.  Sequences of the same pages and queries, so that
    a thread block takes many tiles of one; with a prefix they end at different positions behind it."""
    dexlib = require_gpu()
    kvh, ps = 2, 64
    gen = torch.Generator().manual_seed(int(nats) + n)
    _, pages, table = paged(dexlib, kvh, hd, ps, [length], dtype)
    pages[:, 0] *= 0.25
    pages[:, 0, :, :, 0] = 0.0
    pages[:, 1] = pages[:, 1].abs()
    for p in at:
        page, row = int(table[0, p // ps]), p % ps
        pages[page, 0, :, row] = 0.0
        pages[page, 0, :, row, 0] = sign * nats * hd ** 0.5 / 8.0
        pages[page, 1, :, row] = 0.0
    cache = dexlib.PagedCache(pages.cuda(), table.expand(batch, -1).contiguous().cuda())
    q = torch.randn((n, kvh * G, hd), generator=gen) * 0.25
    q[:, :, 0] = 8.0
    q = q.to(dtype)
    every = q.repeat(batch, 1, 1).cuda()
    start = (torch.arange(batch + 1) * n).int()
    lens = [length - (b % 3 if prefix else 0) for b in range(batch)]
    lse = torch.zeros(every.shape[:2], device="cuda")
    scale = sign * hd ** -0.5
    out = cache.attention(every, start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), n, prefix, lse=lse, scale=scale)
    for size in sorted(set(lens)):
        o, L, bo, bl = attention(pages, table, q, start[:2], [size], scale=scale)
        if dtype == FP:
            # A probability in fp16 is also off by half a step of its smallest numbers, 2^-25.  The kernels take them
            # relative to a tile's largest score so that this one comes to 2^-3 or more, and to 2^7 or more where it
            # raises the running maximum (the peak): a weight is off by 2^-22 of its tile's largest one, in the
            # peak's tile by 2^-32 of the peak's.
            k, v = gather(pages, table[0], size)
            for h in range(kvh * G):
                s = (q[:, h].double() @ k[:, h // G].T) * scale
                w = torch.exp(s - L[:, h][:, None])
                w[:, [p for p in at if p < size]] = 0.0
                # twice the sum of the largest weight of every 64 keys bounds that of any tiles of 64 or 128
                top = torch.stack([x.amax(-1) for x in w.split(64, dim=1)]).sum(0) * 2
                bo[:, h] += (128 * v.abs().max() * (2.0 ** -22 * top + 2.0 ** -32 * len(at)))[:, None]
        for b in [b for b in range(batch) if lens[b] == size]:
            compare(out[b * n:(b + 1) * n], lse[b * n:(b + 1) * n], (o, L, bo, bl), torch.ones(n, dtype=torch.bool))


@pytest.mark.parametrize("dtype,hd", [(FP, 128), (FP, 64), (BF, 128)])
@pytest.mark.parametrize("nats", [8.0, 13.0, 17.0, 21.0])
@pytest.mark.parametrize("n", [1, 6, 20, 70])
def test_weights_far_below_a_peak(n, nats, dtype, hd):
    """One key far above thousands of others: at the front, in the middle, near the end, several of them; single
    tokens and a few (rows_kernel), longer runs that share a row tile and that fill two (tile_kernel)."""
    for at in ([0], [1500], [2900], [0, 1000, 1501]):
        below_a_peak(4, hd, dtype, n, 40, 2930 + n, nats, at)


@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("nats", [13.0, 17.0])
def test_weights_below_a_peak_in_a_shared_prefix(G, nats):
    """The same behind a prefix that is read once, by either kernel, with the peak in it and behind it."""
    for at in ([0], [20000, 32775]):
        below_a_peak(G, 64, FP, 1, 16, 32790, nats, at, prefix=32768)


def test_weights_below_a_peak_negative_scale():
    below_a_peak(4, 128, FP, 20, 40, 2000, 17.0, [700], sign=-1.0)


def turn_of(theta, pos, hd):
    """The angles pos * theta^(-2j/hd), j < hd/2, in radians modulo a turn, from 60 digits."""
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        pi = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
        log = decimal.Decimal(theta).ln()
        turns = [((decimal.Decimal(-2 * j) / hd * log).exp() * pos / (2 * pi)) for j in range(hd // 2)]
        return [float((t - t.to_integral_value()) * 2 * pi) for t in turns]


@pytest.mark.parametrize("theta", [1.0, 1.0001, 1.01, 1.1, 2.0, 10.0, 1e4, 5e5, 1e6, 3e38])
@pytest.mark.parametrize("hd", [64, 128])
def test_far_rotations(hd, theta):
    """Angles at the farthest positions: the pair (sin a, cos a) turned by a is (0, 1), and what is left of the zero
    is the error of the angle."""
    dexlib = require_gpu()
    theta = torch.tensor(theta).item()   # as the call takes it, in 32 bits
    rope = [0, 1, 17, 131072, 10 ** 8 + 7, 2 ** 30, 2 ** 31 - 1, 2 ** 31 - 12345, -1, -(2 ** 31)]
    n = len(rope)
    angle = torch.tensor([turn_of(theta, r, hd) for r in rope], dtype=torch.float64)
    x = torch.cat((angle.sin(), angle.cos()), 1).float()[:, None].contiguous().cuda()
    cache = dexlib.PagedCache(torch.zeros((1, 2, 1, 16, hd), dtype=FP, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    seq, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    cache.append(x, x, seq, pos, theta=theta, rope_pos=torch.tensor(rope, dtype=torch.int32, device="cuda"))
    got = cache.pages[0, 0, 0, :n].cpu().double()
    # The angle in fp32 half-turns is off by pi 2^-25, sin and cos by two units in the last place (2^-23 of 1), the products and
    # inputs by half of one: 2^-21.4 together, and half a step of fp16 (2^-25 below 2^-14) for the result.
    assert got[:, :hd // 2].abs().max().item() <= 2.0 ** -21 + 2.0 ** -25
    assert (got[:, hd // 2:] - 1.0).abs().max().item() <= 2.0 ** -11 + 2.0 ** -21


def bad_page_case(H, kvh, hd, ps, dtype, lens, new, bad, prefix=0, tree=None):
    """Pages of `bad` (sequence or None for all, table entry) out of range: the rows that see a position on one of them
    are NaN, and all others as if nothing had happened."""
    dexlib = require_gpu()
    cache, pages, table = paged(dexlib, kvh, hd, ps, lens, dtype, prefix)
    q, start = queries(H, hd, new, dtype)
    ref = attention(pages, table, q.cpu(), start, lens, prefix, tree=tree)
    broken = table.clone()
    for b, entry in bad:
        broken[slice(None) if b is None else b, entry] = -3
    cache.table.copy_(broken)
    hit = torch.zeros(len(q), dtype=torch.bool)
    for b, (length, n) in enumerate(zip(lens, new)):
        for i in range(n):
            t = int(start[b]) + i
            for p in range(max(0, length)):
                first = length - n
                sees = p <= first + i if tree is None else p < first or bool(int(tree[t]) >> (p - first) & 1)
                if sees and int(broken[b, p // ps]) < 0:
                    hit[t] = True
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.zeros(q.shape[:2], device="cuda")
    out = cache.attention(q, start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), max(new), prefix, lse=lse,
                          status=status, tree_mask=None if tree is None else tree.cuda())
    assert int(status.item()) == dexlib.DEX_ATTN_BAD_PAGE
    assert bool(hit.any())
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
    compare(out, lse, ref, ~hit)


@pytest.mark.parametrize("H,kvh,hd,dtype", [(8, 2, 64, FP), (16, 4, 128, BF)])
@pytest.mark.parametrize("n", [6, 30, 90])
def test_bad_page_behind_the_first_queries(H, kvh, hd, dtype, n):
    """A run of queries, the later ones of which see a bad page: those before it do not."""
    for ps, past in ((16, 100), (32, 3), (64, 250)):
        lens, new = [past + n, 40, past + n + 7], [n, 1, n]
        entry = (past + n // 2) // ps
        bad_page_case(H, kvh, hd, ps, dtype, lens, new, [(0, entry)])
        bad_page_case(H, kvh, hd, ps, dtype, lens, new, [(0, entry), (2, (past + n + 6) // ps), (1, 0)])


@pytest.mark.parametrize("H,kvh,hd,ps,new,prefix", SHARED)
def test_bad_page_of_a_shared_prefix(H, kvh, hd, ps, new, prefix):
    """Sequences that end before the prefix's bad page keep their results."""
    lens = [prefix + n for n in new]
    entry = (prefix // 2) // ps
    for b in (1, 3, len(new) - 1):
        lens[b] = max(1, entry * ps - b % 3)
    bad_page_case(H, kvh, hd, ps, BF, lens, new, [(None, entry)], prefix)


@pytest.mark.parametrize("n", [7, 40])
def test_bad_page_that_tree_words_leave_out(n):
    """Nodes whose words select nothing on the bad page keep their results."""
    g = torch.Generator().manual_seed(n)
    past = [43, 0, 96]
    words = [w | (1 << i) if i % 2 else 1 << i for _ in past for i, w in enumerate(torch.randint(0, 1 << (n // 2), (n,), generator=g).tolist())]
    bad_page_case(8, 2, 64, 16, FP, [p + n for p in past], [n] * 3, [(0, (past[0] + n - 1) // 16), (2, (past[2] + 3) // 16)],
                  tree=torch.tensor(words, dtype=torch.int64))


def test_shared_steps_of_one_kernel_in_a_graph():
    """The captured steps over a shared prefix where one kernel reads the prefix and the sequences' own positions:
    few rows (32 of all sequences at most), and positions enough (912 tiles of 64 in all) that it is read once."""
    batch, kvh, prefix = 7, 32, 330
    assert batch * kvh * (prefix // 64) >= 912
    test_gpu_paged.test_shared_steps_in_a_graph(batch, kvh, 1, 128, prefix)


@pytest.mark.parametrize("batch,kvh,prefix,longest", [(32, 32, 450, 200), (16, 64, 260, 300), (31, 32, 1000, 130)])
@pytest.mark.parametrize("dtype,hd", [(BF, 64), (FP, 128)])
def test_two_ranges_per_block(batch, kvh, prefix, longest, dtype, hd):
    """Work enough that every thread block of the kernel for few rows takes two ranges in turn, prefix and own
    segments in one kernel: eight units (a segment's tiles of 64 and one more) for each of 304 blocks."""
    g = torch.Generator().manual_seed(prefix)
    tails = [int(t) for t in torch.randint(1, longest, (batch,), generator=g)]
    tails[0], tails[-1] = 1, longest
    tiles = lambda lo, hi: -(-hi // 64) - lo // 64
    units = kvh * (tiles(0, prefix) + 1 + sum(tiles(prefix, prefix + t) + 1 for t in tails))
    assert units >= 8 * 304 and batch * kvh * (prefix // 64) >= 912
    run_case(kvh, kvh, hd, 32, dtype, [prefix + t for t in tails], [1] * batch, prefix)
