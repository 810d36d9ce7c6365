"""GPU parity of the paged-cache operators (append with rotation, shared-prefix attention) against
plain 64-bit forms, element by element within bounds derived from the arithmetic."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

from gpu_util import require_gpu
from paged_ref import HALF, attention, rotate, rotate_bound

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def paged(dexlib, kvh, hd, ps, lens, dtype, prefix=0, width=0, spare=2, seed=0, layers=1, fill=math.nan):
    """A cache of the given lengths on shuffled pages; every row no sequence uses holds `fill`.

    Returns the PagedCache and CPU copies of its pages and table."""
    gen = torch.Generator().manual_seed(seed)
    shared = prefix // ps
    need = [max(0, -(-n // ps) - shared) for n in lens]
    n_pages = shared + sum(need) + spare
    ids = torch.randperm(n_pages, generator=gen).int()
    width = width or max(1, max(-(-n // ps) for n in lens))
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    table[:, :shared] = ids[:shared]
    at = shared
    big = torch.full((n_pages, layers, 2, kvh, ps, hd), fill, dtype=dtype)
    pages = big[:, layers - 1]
    pages[ids[:shared].long()] = torch.randn((shared, 2, kvh, ps, hd), generator=gen).to(dtype)
    tail = torch.randn((2, kvh, prefix % ps, hd), generator=gen).to(dtype)
    for b, n in enumerate(lens):
        table[b, shared:shared + need[b]] = ids[at:at + need[b]]
        at += need[b]
        rows = torch.randn((2, kvh, max(0, n - shared * ps), hd), generator=gen).to(dtype)
        rows[:, :, :prefix % ps] = tail[:, :, :rows.shape[2]]
        for i in range(need[b]):
            part = rows[:, :, i * ps:(i + 1) * ps]
            pages[int(table[b, shared + i]), :, :, :part.shape[2]] = part
    cache = dexlib.PagedCache(big.cuda()[:, layers - 1], table.cuda())
    return cache, pages, table


def queries(H, hd, new, dtype, seed=1, pad=0, strided=False):
    gen = torch.Generator().manual_seed(seed)
    n = sum(new) + pad
    q = torch.randn((n, H + (2 if strided else 0), hd), generator=gen).to(dtype).cuda()[:, :H]
    start = torch.tensor([0] + new).cumsum(0).int()
    return q, start


def compare(out, lse, ref, owned):
    o, L, bo, bl = ref
    out, lse = out.cpu().double(), lse.cpu().double()
    err = (out - o).abs()[owned]
    assert not torch.isnan(out[owned]).any()
    worst = (err / bo[owned].clamp_min(1e-30)).max().item() if err.numel() else 0.0
    assert bool((err <= bo[owned]).all()), f"out is {worst} of its bound"
    inf = torch.isinf(L[owned])
    assert torch.equal(inf, torch.isinf(lse[owned]))
    d = (lse - L).abs()[owned][~inf]
    assert bool((d <= bl[owned][~inf]).all()), f"lse off by {d.max().item()}"
    return worst


def run_case(H, kvh, hd, ps, dtype, lens, new, prefix=0, tree=None, pad=0, strided=False, layers=1, seed=0, scale=None,
             prefix_table=False):
    dexlib = require_gpu()
    cache, pages, table = paged(dexlib, kvh, hd, ps, lens, dtype, prefix, seed=seed, layers=layers)
    q, start = queries(H, hd, new, dtype, seed + 1, pad, strided)
    seq_len = torch.tensor(lens, dtype=torch.int32)
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ptab = table[0, :-(-prefix // ps)].clone() if prefix_table else None
    kw = dict(max_q=max(1, max(new)), prefix_len=prefix, scale=scale,
              tree_mask=None if tree is None else tree.cuda(), prefix_table=None if ptab is None else ptab.cuda())
    got = cache.attention(q, start.cuda(), seq_len.cuda(), out=out, lse=lse, status=status, **kw)
    assert got is out
    again, lse2 = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    cache.attention(q, start.cuda(), seq_len.cuda(), out=again, lse=lse2, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(out, again) and torch.equal(lse, lse2)   # the same bits every time
    ref = attention(pages, table, q.cpu(), start, lens, prefix, ptab, tree, scale)
    owned = torch.zeros(len(q), dtype=torch.bool)
    owned[:int(start[-1])] = True
    compare(out, lse, ref, owned)
    assert bool((out[int(start[-1]):] == 7.0).all()) and bool((lse[int(start[-1]):] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("H,kvh,hd", [(32, 8, 128), (4, 4, 64), (6, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("ps", [16, 64, 256])
def test_attention_decode(H, kvh, hd, ps, dtype):
    """Single tokens, no sharing: lengths of one, around tile and page borders, an inactive slot."""
    run_case(H, kvh, hd, ps, dtype, [1, 2, 63, 64, 65, 127, 128, 129, 300, 40], [1, 1, 1, 1, 1, 1, 1, 1, 1, 0])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("H,kvh,hd,ps", [(32, 8, 128, 16), (8, 8, 128, 32), (16, 4, 64, 64), (6, 2, 128, 128)])
@pytest.mark.parametrize("prefix", [1, 128, 200, 511])
def test_attention_decode_prefix(H, kvh, hd, ps, prefix, dtype):
    """Single tokens behind a shared prefix that ends anywhere in a page or tile."""
    own = [1, 2, 17, 64, 130, 5, 1, 90, 33, 128, 1, 77, 3, 1, 1, 40, 22]
    run_case(H, kvh, hd, ps, dtype, [prefix + n for n in own], [1] * len(own), prefix, prefix_table=prefix == 200)


@pytest.mark.parametrize("G", [1, 3, 5, 8, 12, 16, 17, 32, 71, 128])
def test_attention_group_sizes(G):
    """Any number of query heads per K/V head, with and without sharing."""
    run_case(2 * G, 2, 64, 32, FP, [300 + 13 * i for i in range(5)], [1, 2, 0, 1, 3], 260)
    run_case(G, 1, 128, 16, BF, [1, 140, 77], [1, 1, 1])


@pytest.mark.parametrize("H,kvh,hd,dtype", [(32, 8, 128, BF), (4, 4, 64, FP), (3, 1, 128, FP)])
@pytest.mark.parametrize("prefix", [0, 130, 384])
def test_attention_prompts(H, kvh, hd, dtype, prefix):
    """Query runs of every length, causal among themselves, padding rows behind the last one."""
    new = [1, 16, 17, 33, 64, 65, 130, 257, 0, 300]
    past = [0, 5, 0, 100, 63, 1, 0, 7, 3, 129]
    run_case(H, kvh, hd, 64, dtype, [prefix + p + n for p, n in zip(past, new)], new, prefix, pad=3, strided=True)


@pytest.mark.parametrize("H,kvh,hd", [(32, 8, 128), (4, 4, 64), (8, 1, 128)])
@pytest.mark.parametrize("prefix", [0, 150])
@pytest.mark.parametrize("most", [4, 15, 64])
def test_attention_tree(H, kvh, hd, prefix, most):
    """Lattice nodes: ancestry masks over the last positions, some words empty."""
    g = torch.Generator().manual_seed(most)
    new = [1, most, most // 2 + 1, 0, 2, most]
    past = [0, 3, 64, 9, 140, 0]
    words = []
    for n in new:
        for i in range(n):
            w = 1 << i
            for k in range(i):
                w |= int(torch.randint(0, 2, (1,), generator=g)) << k
            words.append(0 if i % 7 == 3 else w - (1 << 64) if w >= 1 << 63 else w)
    tree = torch.tensor(words, dtype=torch.int64)
    run_case(H, kvh, hd, 32, FP, [prefix + p + n for p, n in zip(past, new)], new, prefix, tree)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_attention_nothing_visible(dtype):
    """Empty sequences, queries ahead of a sequence's start, sequences inside the prefix."""
    run_case(8, 2, 64, 16, dtype, [0, 3, 0, 1, 200], [1, 5, 2, 4, 1])                    # p < 0 rows: zeros, -inf
    run_case(8, 2, 64, 16, dtype, [100, 260, 300, 30], [40, 1, 40, 30], prefix=100)      # a query run across the border
    tree = torch.zeros(4, dtype=torch.int64)
    run_case(8, 2, 128, 16, dtype, [2, 2], [2, 2], tree=tree)                            # all words empty, nothing cached


@pytest.mark.parametrize("dtype,hd", [(BF, 128), (FP, 64)])
def test_attention_short_segments_in_turn(dtype, hd):
    """Many one-tile segments per thread block, of more than 128 rows and of fewer in turn (the two halves of a block
    take a row tile each, or share the rows), some of them with a bad page: results and poison stay with their own."""
    dexlib = require_gpu()
    kvh, G, ps = 4, 4, 32
    new = [n for _ in range(70) for n in (75, 10, 1, 40)]
    lens = [n + 13 * (b % 3) for b, n in enumerate(new)]
    cache, pages, table = paged(dexlib, kvh, hd, ps, lens, dtype)
    q, start = queries(kvh * G, hd, new, dtype)
    owner = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    at = torch.tensor(lens)[owner] - torch.tensor(new)[owner] + torch.arange(len(q)) - start[:-1].long()[owner]   # positions
    ref = attention(pages, table, q.cpu(), start, lens)
    seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    victims = torch.tensor([b % 5 == 2 and n > 40 for b, n in enumerate(lens)])
    for entry in (None, 0, 1):
        bad = table.clone()
        if entry is not None:
            bad[victims, entry] = -1
        cache.table.copy_(bad)
        for _ in range(5):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            lse = torch.zeros(q.shape[:2], device="cuda")
            out = cache.attention(q, start.cuda(), seq_len, max(new), lse=lse, status=status)
            assert int(status.item()) == (0 if entry is None else dexlib.DEX_ATTN_BAD_PAGE)
            hit = victims[owner] if entry is not None else torch.zeros(len(q), dtype=torch.bool)
            compare(out, lse, ref, ~hit)
            if entry is not None:
                assert bool(torch.isnan(out[hit & (at >= entry * ps)]).all())


def test_attention_long_and_layers():
    """A long context split over the whole GPU, pages strided over the layers of a model."""
    run_case(8, 2, 128, 16, BF, [20011], [1], layers=3)
    run_case(8, 2, 128, 128, FP, [9000, 9001, 9002, 8999], [1, 2, 1, 1], prefix=8990)


def test_attention_scale_and_extremes():
    """Large scores (one key dominates), a negative and a zero scale."""
    for scale in (3.0, -0.5, 0.0):
        run_case(4, 2, 64, 32, FP, [150, 400, 90], [1, 3, 20], prefix=64, scale=scale)


def test_attention_bad_pages_and_ranges():
    """Bad page ids and lengths poison the rows that need them and nothing else."""
    dexlib = require_gpu()
    H, kvh, hd, ps = 8, 2, 64, 16
    lens, new = [50, 60, 70, 80], [1, 1, 1, 1]
    cache, pages, table = paged(dexlib, kvh, hd, ps, lens, BF)
    q, start = queries(H, hd, new, BF)
    ref = attention(pages, table, q.cpu(), start, lens)
    for victim, value in ((1, 10 ** 9), (1, -1), (1, -2 ** 31)):
        bad = table.clone()
        bad[victim, 2] = value
        cache.table.copy_(bad)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lse = torch.zeros((4, H), device="cuda")
        out = cache.attention(q, start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), max_q=1, lse=lse,
                              status=status)
        assert int(status.item()) == dexlib.DEX_ATTN_BAD_PAGE
        assert bool(torch.isnan(out[victim]).all()) and bool(torch.isnan(lse[victim]).all())
        compare(out, lse, ref, torch.tensor([b != victim for b in range(4)]))
    cache.table.copy_(table)
    for value in (-1, cache.table.shape[1] * ps + 1, 2 ** 31 - 1):
        L = torch.tensor(lens, dtype=torch.int32)
        L[2] = value
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lse = torch.zeros((4, H), device="cuda")
        out = cache.attention(q, start.cuda(), L.cuda(), max_q=1, lse=lse, status=status)
        assert int(status.item()) == dexlib.DEX_ATTN_BAD_RANGE
        assert bool(torch.isnan(out[2]).all())
        compare(out, lse, ref, torch.tensor([True, True, False, True]))
    # more queries than max_q: that sequence is left out, its rows stay
    q, start = queries(H, hd, [1, 3, 1, 1], BF)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    cache.attention(q, start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), max_q=2, out=out,
                    status=status)
    assert int(status.item()) == dexlib.DEX_ATTN_BAD_RANGE
    assert bool((out[1:4] == 7.0).all()) and not bool((out[[0, 4, 5]] == 7.0).any())


def test_attention_inactive_first_slot():
    """Sequence 0 is an empty slot without pages: the shared prefix comes from prefix_table."""
    dexlib = require_gpu()
    H, kvh, hd, ps, prefix = 32, 8, 128, 32, 200
    lens, new = [0] + [prefix + n for n in (3, 90, 1, 64, 17)], [0, 1, 1, 1, 1, 1]
    for h in (H, kvh):   # the prefix on either kernel
        cache, pages, table = paged(dexlib, kvh, hd, ps, lens, BF, prefix)
        shared = table[1, :-(-prefix // ps)].clone()
        cache.table[0] = -1
        q, start = queries(h, hd, new, BF)
        seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lse = torch.zeros(q.shape[:2], device="cuda")
        out = cache.attention(q, start.cuda(), seq_len, 1, prefix, prefix_table=shared.cuda(), lse=lse, status=status)
        assert int(status.item()) == 0
        compare(out, lse, attention(pages, table, q.cpu(), start, lens, prefix, shared), torch.ones(5, dtype=torch.bool))


@pytest.mark.parametrize("H,new", [(32, [0, 1, 2, 1, 1, 2]), (8, [0, 1, 1, 1, 1, 1])])
def test_shared_prefix_without_row_zero(H, new):
    """A prefix long enough to be read once, by either kernel, whose pages row 0 of the table does not name."""
    dexlib = require_gpu()
    kvh, hd, ps, prefix = 8, 128, 32, 1600
    lens = [0] + [prefix + n for n in (3, 90, 2, 64, 17)]
    cache, pages, table = paged(dexlib, kvh, hd, ps, lens, BF, prefix)
    shared = table[1, :prefix // ps].clone()
    cache.table[0] = -1
    q, start = queries(H, hd, new, BF)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.zeros(q.shape[:2], device="cuda")
    out = cache.attention(q, start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), max(new), prefix,
                          prefix_table=shared.cuda(), lse=lse, status=status)
    assert int(status.item()) == 0
    compare(out, lse, attention(pages, table, q.cpu(), start, lens, prefix, shared), torch.ones(len(q), dtype=torch.bool))


@pytest.mark.parametrize("prefix", [0, 128])
def test_attention_large_batch(prefix):
    """The largest batch, most of it without queries or without positions."""
    g = torch.Generator().manual_seed(5)
    new = [int(x) for x in (torch.rand(1024, generator=g) < 0.06)]
    new[0] = 1
    lens = [prefix + int(x) if n else 0 for n, x in zip(new, torch.randint(1, 200, (1024,), generator=g))]
    run_case(8, 2, 64, 64, FP, lens, new, prefix)


@pytest.mark.parametrize("H,kvh,hd,dtype", [(32, 8, 128, BF), (8, 4, 64, FP)])
@pytest.mark.parametrize("batch,longest", [(20, 30), (60, 700), (200, 90), (77, 1)])
def test_attention_prefix_beside_tails(H, kvh, hd, dtype, batch, longest):
    """The prefix of many sequences next to their own ragged positions: few of them, some very long, none but the
    queries' own."""
    g = torch.Generator().manual_seed(batch)
    new = [int(x) for x in torch.randint(0, 3, (batch,), generator=g)]
    new[0] = 1
    tails = torch.randint(0, longest, (batch,), generator=g)
    run_case(H, kvh, hd, 32, dtype, [300 + int(t) + n for t, n in zip(tails, new)], new, prefix=300)


# (n_heads, kv_heads, head_dim, page, queries of each sequence, prefix): enough sequences and positions that the prefix
# is read once for all of them (912 tiles of 64 positions x sequences x K/V heads), by either kernel, next to own
# positions on either kernel
SHARED = [(32, 8, 128, 16, [1] * 8, 1000), (4, 4, 64, 64, [2, 1, 0, 1] * 3, 1300), (32, 32, 128, 32, [1] * 5, 450),
          (32, 8, 128, 64, [1, 3, 0, 2] * 4, 640), (6, 2, 64, 16, [1, 2] * 20, 777), (8, 1, 128, 256, [1, 5, 1] * 15, 1500),
          (16, 16, 64, 128, [7, 0, 30, 1] * 3, 500), (12, 4, 128, 32, [1] * 70, 260), (30, 2, 128, 16, [2] * 40, 800)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("H,kvh,hd,ps,new,prefix", SHARED)
def test_attention_shared(H, kvh, hd, ps, new, prefix, dtype):
    g = torch.Generator().manual_seed(prefix)
    past = torch.randint(0, 150, (len(new),), generator=g)
    past[1], past[-1] = 0, 400
    run_case(H, kvh, hd, ps, dtype, [prefix + int(p) + n for p, n in zip(past, new)], new, prefix, pad=2, strided=True)


@pytest.mark.parametrize("H,kvh,hd,ps,new,prefix", SHARED)
def test_attention_shared_tree(H, kvh, hd, ps, new, prefix):
    g = torch.Generator().manual_seed(prefix + 1)
    words = []
    for n in new:
        word = []
        for i in range(n):   # ancestors of a random tree; a root that does not see itself now and then
            parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            word.append((word[parent] if parent >= 0 else 0) | (1 << i if int(torch.randint(0, 9, (1,), generator=g)) else 0))
        words += word
    run_case(H, kvh, hd, ps, FP, [prefix + n + 40 * (n % 2) for n in new], new, prefix,
             torch.tensor(words, dtype=torch.int64))


@pytest.mark.parametrize("H,kvh,hd,ps,new,prefix", SHARED)
def test_attention_shared_edges(H, kvh, hd, ps, new, prefix):
    """Sequences that end inside the prefix or before their queries, empty ones, a scale below zero, the prefix by a
    table of its own."""
    lens = [prefix + n for n in new]
    lens[1] = prefix // 2
    lens[2] = 0
    lens[-1] = 1
    run_case(H, kvh, hd, ps, BF, lens, new, prefix, scale=-0.25, prefix_table=True)


@pytest.mark.parametrize("H,kvh,hd,ps,new,prefix", SHARED)
def test_attention_shared_bad_pages(H, kvh, hd, ps, new, prefix):
    """A bad page of a sequence's own poisons it, one of the prefix everyone, a bad length its sequence."""
    dexlib = require_gpu()
    lens = [prefix + 30 * (b % 3) + n for b, n in enumerate(new)]
    cache, pages, table = paged(dexlib, kvh, hd, ps, lens, BF, prefix)
    q, start = queries(H, hd, new, BF)
    ref = attention(pages, table, q.cpu(), start, lens, prefix)
    seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    owner = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    victim = max(b for b, n in enumerate(new) if n and (lens[b] - 1) // ps >= -(-prefix // ps))

    def call(length=seq_len):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lse = torch.zeros(q.shape[:2], device="cuda")
        out = cache.attention(q, start.cuda(), length, max(new), prefix, lse=lse, status=status)
        return out, lse, int(status.item())

    bad = table.clone()
    bad[victim, (lens[victim] - 1) // ps] = len(pages)
    cache.table.copy_(bad)
    out, lse, status = call()
    assert status == dexlib.DEX_ATTN_BAD_PAGE
    assert bool(torch.isnan(out[owner == victim]).all()) and bool(torch.isnan(lse[owner == victim]).all())
    compare(out, lse, ref, owner != victim)
    bad = table.clone()
    bad[:, prefix // ps // 2] = -5
    cache.table.copy_(bad)
    out, lse, status = call()
    assert status == dexlib.DEX_ATTN_BAD_PAGE and bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
    cache.table.copy_(table)
    length = seq_len.clone()
    length[victim] = -1
    out, lse, status = call(length)
    assert status == dexlib.DEX_ATTN_BAD_RANGE and bool(torch.isnan(out[owner == victim]).all())
    compare(out, lse, ref, owner != victim)


def test_attention_strides():
    """Queries that are one expanded row, an output inside a larger tensor, a table inside a wider one, tokens
    before the first sequence's."""
    dexlib = require_gpu()
    H, kvh, hd, ps, prefix = 8, 2, 64, 32, 96
    lens, new = [prefix + n for n in (5, 70, 33)], [1, 2, 1]
    for prefix_len in (0, prefix):
        cache, pages, table = paged(dexlib, kvh, hd, ps, lens, FP, prefix)
        wide = torch.full((3, table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
        wide[:, 2:2 + table.shape[1]] = table.cuda()
        cache = dexlib.PagedCache(cache.pages, wide[:, 2:2 + table.shape[1]])
        one = torch.randn((1, H, hd), device="cuda").to(FP)
        q = one.expand(6, H, hd)
        big = torch.full((6, H + 3, hd), 7.0, dtype=FP, device="cuda")
        lse = torch.full((6, H), 7.0, device="cuda")
        start = torch.tensor([2, 3, 5, 6], dtype=torch.int32)
        cache.attention(q, start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 2, prefix_len,
                        out=big[:, 1:H + 1], lse=lse)
        own = torch.tensor([False, False, True, True, True, True])
        compare(big[:, 1:H + 1], lse, attention(pages, table, q.cpu(), start, lens, prefix_len), own)
        assert bool((big[:2] == 7.0).all()) and bool((big[:, 0] == 7.0).all()) and bool((big[:, H + 1:] == 7.0).all())
        assert bool((lse[:2] == 7.0).all())


def test_offsets_beyond_32_bits():
    """Pages whose elements and bytes lie beyond 2^31 and 2^32: append and attention reach them."""
    dexlib = require_gpu()
    kvh, hd, ps, H = 8, 128, 64, 32
    n_pages = (1 << 32) // (2 * kvh * ps * hd) + 40   # 2^32 elements and some
    pages = torch.empty((n_pages, 2, kvh, ps, hd), dtype=BF, device="cuda")
    ids = torch.tensor([[n_pages - 1, 3], [n_pages - 30, n_pages - 2]], dtype=torch.int32)
    cache = dexlib.PagedCache(pages, ids.cuda())
    gen = torch.Generator().manual_seed(4)
    lens = [100, 128]
    n = sum(lens)
    k, v = (torch.randn((n, kvh, hd), generator=gen).to(BF) for _ in range(2))
    seq = torch.tensor([0] * 100 + [1] * 128, dtype=torch.int32, device="cuda")
    pos = torch.cat((torch.arange(100), torch.arange(128))).int().cuda()
    cache.append(k.cuda(), v.cuda(), seq, pos, theta=0.0)
    small = torch.zeros((4, 2, kvh, ps, hd), dtype=BF)
    small_ids = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    for i in range(4):
        small[i] = pages[int(ids.view(-1)[i])].cpu()
    for t in range(n):
        b, p = int(seq[t]), int(pos[t])
        assert t % 37 or (torch.equal(small[2 * b + p // ps, 0, :, p % ps], k[t]) and
                          torch.equal(small[2 * b + p // ps, 1, :, p % ps], v[t]))
    for new in ([1, 1], [20, 60]):
        q, start = queries(H, hd, new, BF)
        lse = torch.zeros(q.shape[:2], device="cuda")
        out = cache.attention(q, start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), max(new), lse=lse)
        compare(out, lse, attention(small, small_ids, q.cpu(), start, lens), torch.ones(len(q), dtype=torch.bool))


def test_calls_from_a_new_thread():
    """A thread whose first CUDA work is an attention call (or an append): it has no context of its own yet."""
    dexlib = require_gpu()
    H, kvh, hd, ps = 8, 2, 64, 16
    lens, new = [50, 20], [1, 2]
    cache, pages, table = paged(dexlib, kvh, hd, ps, lens, BF)
    q, start = queries(H, hd, new, BF)
    start, seq_len = start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = cache.attention_workspace(q, 2)
    want = cache.attention(q, start, seq_len, 2, workspace=ws)
    k, idx = pages[:2, 0, :, 0].cuda(), torch.full((2,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for calls in (lambda out: cache.attention(q, start, seq_len, 2, out=out, workspace=ws),
                  lambda out: (cache.append(k, k, idx, idx), cache.attention(q, start, seq_len, 2, out=out, workspace=ws))):
        out, errors = torch.zeros_like(q), []

        def run():
            try:
                calls(out)
            except Exception as e:
                errors.append(e)

        t = threading.Thread(target=run)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not errors and torch.equal(out, want), errors


FIRST_CALLS = """
import threading, torch
import lossless_depth_adaptive_gb300 as dexlib
pages = torch.randn((40, 2, 2, 16, 64), device="cuda").half()
table = torch.randperm(40, device="cuda")[:32].int().view(4, 8)
cache = dexlib.PagedCache(pages, table)
q = torch.randn((8, 8, 64), device="cuda").half()
start = torch.arange(0, 10, 2, dtype=torch.int32, device="cuda")
lens = torch.tensor([100, 17, 64, 128], dtype=torch.int32, device="cuda")
outs = [torch.zeros_like(q) for _ in range(8)]
spaces = [cache.attention_workspace(q, 2) for _ in outs]
streams = [torch.cuda.Stream() for _ in outs]
torch.cuda.synchronize()
gate, errors = threading.Barrier(len(outs)), []
def first(i):
    try:
        gate.wait()
        with torch.cuda.stream(streams[i]):
            cache.attention(q, start, lens, 2, out=outs[i], workspace=spaces[i])
    except Exception as e:
        errors.append(e)
threads = [threading.Thread(target=first, args=(i,)) for i in range(len(outs))]
[t.start() for t in threads], [t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
assert all(torch.equal(o, outs[0]) for o in outs) and bool(outs[0].any())
"""


def test_first_calls_on_several_threads():
    """A process whose first attention calls are made by several threads at once, a stream and a workspace each."""
    require_gpu()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]


def test_attention_two_at_once():
    """Calls on two streams, a workspace each, give what they give alone."""
    dexlib = require_gpu()
    H, kvh, hd, ps, prefix = 32, 8, 128, 64, 512
    lens, new = [prefix + 40 * i + 1 for i in range(20)], [1] * 20
    cache, pages, table = paged(dexlib, kvh, hd, ps, lens, BF, prefix)
    seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = [queries(H, hd, new, BF, seed=s)[0] for s in (1, 2)]
    start = queries(H, hd, new, BF)[1].cuda()
    alone = [cache.attention(q, start, seq_len, 1, prefix) for q in qs]
    outs = [torch.zeros_like(q) for q in qs]
    spaces = [cache.attention_workspace(q, 1, prefix) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(10):
        for q, o, w, st in zip(qs, outs, spaces, streams):
            with torch.cuda.stream(st):
                cache.attention(q, start, seq_len, 1, prefix, out=o, workspace=w)
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for a, o in zip(alone, outs))


def test_workspace_in_any_state():
    """A workspace holds anything before a call: the same bits from a fresh one, from one filled with any byte, and
    from one that calls of other plans (either kernel alone, both side by side) have used in between."""
    dexlib = require_gpu()
    H, kvh, hd, ps, prefix = 32, 8, 128, 32, 400
    lens, new = [prefix + 37 * i + 1 for i in range(24)], [1] * 24
    cache, pages, table = paged(dexlib, kvh, hd, ps, lens, BF, prefix)
    seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, start = queries(H, hd, new, BF)
    start = start.cuda()
    runs = torch.tensor([0] + [24] * 24, dtype=torch.int32, device="cuda")   # all tokens of sequence 0
    # both kernels, rows_kernel, tile_kernel, rows_kernel with the prefix
    calls = [(q, start, 1, prefix), (q, start, 1, 0), (q, runs, 24, 0), (q[:, :kvh], start, 1, prefix)]
    calls = [(x.contiguous(), *rest) for x, *rest in calls]
    size = max(cache.attention_workspace(x, m, p).numel() for x, _, m, p in calls)
    want = [cache.attention(x, st, seq_len, m, p) for x, st, m, p in calls]
    out, _, bound, _ = attention(pages, table, q.cpu(), start.cpu(), lens, prefix)
    assert bool(((want[0].cpu().double() - out).abs() <= bound).all())
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for fill in (0, 1, 0x7f, 0xff, None):
        if fill is not None:
            ws.fill_(fill)
        for _ in range(3):
            for (x, st, m, p), w in zip(calls, want):
                status = torch.zeros(1, dtype=torch.int32, device="cuda")
                assert torch.equal(cache.attention(x, st, seq_len, m, p, workspace=ws, status=status), w)
                assert int(status.item()) == 0


@pytest.mark.parametrize("batch,kvh,G,hd,prefix", [(24, 8, 4, 128, 400), (14, 8, 2, 64, 600), (7, 32, 1, 128, 300)])
def test_shared_steps_in_a_graph(batch, kvh, G, hd, prefix):
    """A captured step (append, then attention) replayed while the sequences grow, one of them runs ahead and some
    have no token: the prefix is read once, by either kernel, with the rest beside it or in the same one."""
    dexlib = require_gpu()
    H, ps, steps = kvh * G, 32, 12
    gen = torch.Generator().manual_seed(batch)
    lens = [prefix + int(x) for x in torch.randint(0, 60, (batch,), generator=gen)]
    lens[1] = prefix + 900
    cache, pages, table = paged(dexlib, kvh, hd, ps, [n + steps for n in lens], BF, prefix, fill=0.0)
    pages = pages.clone()
    rows = torch.randn((steps, batch, H + 2 * kvh, hd), generator=gen).to(BF)
    live = torch.rand((steps, batch), generator=gen) < 0.8
    live[0], live[:, 0], live[5] = True, True, False
    step = torch.zeros((batch, H + 2 * kvh, hd), dtype=BF, device="cuda")
    seq, pos, seq_len = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(3))
    start = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    out = torch.zeros((batch, H, hd), dtype=BF, device="cuda")
    lse = torch.zeros((batch, H), device="cuda")
    q = torch.zeros((batch, H, hd), dtype=BF, device="cuda")
    ws = cache.attention_workspace(q, 1, prefix)

    def call():
        cache.append(step[:, H:H + kvh], step[:, H + kvh:], seq, pos, q=step[:, :H], q_out=q, theta=0.0)
        cache.attention(q, start, seq_len, 1, prefix, out=out, lse=lse, workspace=ws)

    seq.fill_(-1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    now = list(lens)
    for i in range(steps):
        who = [b for b in range(batch) if live[i, b]]
        n = len(who)
        step[:n] = rows[i, who].cuda()
        seq.copy_(torch.tensor(who + [-1] * (batch - n), dtype=torch.int32))
        pos.copy_(torch.tensor([now[b] for b in who] + [0] * (batch - n), dtype=torch.int32))
        for t, b in enumerate(who):
            page, row = int(table[b, now[b] // ps]), now[b] % ps
            pages[page, 0, :, row], pages[page, 1, :, row] = rows[i, b, H:H + kvh], rows[i, b, H + kvh:]
            now[b] += 1
        first = torch.tensor([0] + [int(x) for x in live[i]]).cumsum(0).int()
        start.copy_(first)
        seq_len.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        own = torch.arange(batch) < n
        compare(out, lse, attention(pages, table, rows[i, who + [0] * (batch - n), :H], first, now, prefix), own)
        assert bool((out[n:] == 7.0).all()) and bool((lse[n:] == 7.0).all())


def test_calls_follow_each_other_closely():
    """Steps back to back on one stream, each changing the lengths and the cache the next one reads: what
    a step sees does not depend on how early its kernels become resident."""
    dexlib = require_gpu()
    H, kvh, hd, ps = 8, 2, 128, 16
    lens = [30, 61, 7]
    gen = torch.Generator().manual_seed(8)
    steps = 40
    cache, pages, table = paged(dexlib, kvh, hd, ps, [n + steps for n in lens], FP, fill=0.0)
    pages = pages.clone()
    qkv = torch.randn((steps, 3, H + 2 * kvh, hd), generator=gen).to(FP)
    dev, seq = qkv.cuda(), torch.arange(3, dtype=torch.int32, device="cuda")
    pos = torch.tensor(lens, dtype=torch.int32, device="cuda")
    start = torch.arange(4, dtype=torch.int32, device="cuda")
    outs, ws = [], cache.attention_workspace(dev[0, :, :H], 1)
    torch.cuda.synchronize()
    for i in range(steps):
        cache.append(dev[i, :, H:H + kvh], dev[i, :, H + kvh:], seq, pos, theta=0.0)
        pos += 1
        outs.append(cache.attention(dev[i, :, :H], start, pos, 1, workspace=ws))
    torch.cuda.synchronize()
    for i in range(steps):
        for b in range(3):
            p = lens[b] + i
            pages[int(table[b, p // ps]), 0, :, p % ps] = qkv[i, b, H:H + kvh]
            pages[int(table[b, p // ps]), 1, :, p % ps] = qkv[i, b, H + kvh:]
        o, _, bo, _ = attention(pages, table, qkv[i, :, :H], start.cpu(), [n + i + 1 for n in lens])
        assert bool(((outs[i].cpu().double() - o).abs() <= bo).all()), i


def test_attention_graph_and_streams():
    """A captured call replayed on other lengths and tables; a call on a side stream."""
    dexlib = require_gpu()
    H, kvh, hd, ps, prefix = 8, 2, 128, 32, 96
    lens, new = [prefix + 900, prefix + 5, prefix + 40], [1, 1, 1]
    cache, pages, table = paged(dexlib, kvh, hd, ps, lens, FP, prefix)
    q, start = queries(H, hd, new, FP)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st = start.cuda()
    ws = cache.attention_workspace(q, 1, prefix)
    out = torch.zeros(q.shape, dtype=FP, device="cuda")
    lse = torch.zeros(q.shape[:2], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.attention(q, st, seq, 1, prefix, out=out, lse=lse, workspace=ws)
    side.synchronize()
    own = torch.ones(3, dtype=torch.bool)
    compare(out, lse, attention(pages, table, q.cpu(), start, lens, prefix), own)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attention(q, st, seq, 1, prefix, out=out, lse=lse, workspace=ws)
    for now in (lens, [prefix + 1, prefix + 2, prefix + 3], [prefix + 300, prefix, prefix + 40]):
        seq.copy_(torch.tensor(now, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        compare(out, lse, attention(pages, table, q.cpu(), start, now, prefix), own)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("in32", [False, True])
@pytest.mark.parametrize("H,kvh,hd,ps", [(32, 8, 128, 16), (4, 4, 64, 64), (70, 70, 64, 32), (3, 1, 128, 256)])
def test_append(H, kvh, hd, ps, in32, dtype):
    """Rotation, destination rows, strided inputs, far positions, padding and rejected tokens."""
    dexlib = require_gpu()
    lens, width = [3 * ps, 2 * ps + 5, ps], 4
    cache, pages, table = paged(dexlib, kvh, hd, ps, lens, dtype, width=width, fill=0.5)
    gen = torch.Generator().manual_seed(3)
    it = torch.float32 if in32 else dtype
    toks = [(0, 0), (0, 1), (0, 3 * ps - 1), (1, 2 * ps), (1, ps - 1), (2, 5), (-1, 3), (2, -1), (3, 0), (0, 4 * ps),
            (2, 2 * ps), (-5, 0), (0, 2 ** 31 - 1)]   # the last six out of range, (2, 2 ps) on a page id of -1
    n = len(toks)
    rope = torch.tensor([0, 1, 131071, 2 ** 31 - 1, 77, 1000003, 5, 5, 5, 5, 5, 5, 5], dtype=torch.int32)
    qkv = torch.randn((n, (H + 2 * kvh) * hd + 8), generator=gen).to(it)
    dev = qkv.cuda()
    parts = [x.unflatten(1, (-1, hd)) for x in dev[:, :(H + 2 * kvh) * hd].split((H * hd, kvh * hd, kvh * hd), dim=1)]
    host = [x.unflatten(1, (-1, hd)) for x in qkv[:, :(H + 2 * kvh) * hd].split((H * hd, kvh * hd, kvh * hd), dim=1)]
    seq = torch.tensor([t[0] for t in toks], dtype=torch.int32)
    pos = torch.tensor([t[1] for t in toks], dtype=torch.int32)
    q_out = torch.full((n, H, hd), 7.0, dtype=dtype, device="cuda")
    rejected = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    for theta, use_rope in ((10000.0, True), (1e6, False), (0.0, True)):
        q_out.fill_(7.0)
        cache.pages.copy_(pages)
        r = rope if use_rope else pos
        got = cache.append(parts[1], parts[2], seq.cuda(), pos.cuda(), q=parts[0], q_out=q_out, theta=theta,
                           rope_pos=rope.cuda() if use_rope else None, rejected=rejected)
        assert got is q_out and int(rejected.item()) == 6
        want = pages.double()
        tol = torch.zeros_like(want)
        k, kb = rotate(host[1], r, theta), rotate_bound(host[1], dtype)
        for t in range(6):
            pg, row = int(table[toks[t][0], toks[t][1] // ps]), toks[t][1] % ps
            want[pg, 0, :, row], tol[pg, 0, :, row] = k[t], kb[t]
            want[pg, 1, :, row] = host[2][t].to(dtype).double()
        assert bool(((cache.pages.cpu().double() - want).abs() <= tol).all())
        qq = q_out.cpu().double()
        assert bool(((qq[:6] - rotate(host[0], r, theta)[:6]).abs() <= rotate_bound(host[0], dtype)[:6]).all())
        assert bool((qq[6:] == 7.0).all())
    # q rotated in place equals q rotated aside; without q the cache gets the same rows
    if not in32:
        before = cache.pages.clone()
        cache.append(parts[1], parts[2], seq.cuda(), pos.cuda(), q=parts[0], q_out=parts[0], theta=0.0, rope_pos=rope.cuda())
        assert torch.equal(dev, qkv.cuda())
        a = cache.append(parts[1], parts[2], seq.cuda(), pos.cuda(), q=parts[0], rope_pos=rope.cuda())
        first = cache.pages.clone()
        cache.pages.copy_(before)
        cache.append(parts[1], parts[2], seq.cuda(), pos.cuda(), q=parts[0], q_out=parts[0], rope_pos=rope.cuda())
        assert torch.equal(parts[0][:6], a[:6]) and torch.equal(first, cache.pages)
        cache.pages.copy_(before)
        assert cache.append(parts[1], parts[2], seq.cuda(), pos.cuda(), rope_pos=rope.cuda()) is None
        assert torch.equal(first, cache.pages)


def test_append_empty_and_graph():
    dexlib = require_gpu()
    cache, _, table = paged(dexlib, 2, 64, 16, [32, 32], FP, fill=0.0)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    rejected = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    cache.append(torch.zeros((0, 2, 64), dtype=FP, device="cuda"), torch.zeros((0, 2, 64), dtype=FP, device="cuda"), none,
                 none, rejected=rejected)
    assert int(rejected.item()) == 0
    k = torch.randn((2, 2, 64), dtype=FP, device="cuda")
    seq = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    cache.append(k, k, seq, pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(k, k, seq, pos, theta=0.0)
    for p in ([5, 6], [31, 0]):
        pos.copy_(torch.tensor(p, dtype=torch.int32))
        cache.pages.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            pg = int(table[b, p[b] // 16])
            assert torch.equal(cache.pages[pg, 0, :, p[b] % 16], k[b]) and torch.equal(cache.pages[pg, 1, :, p[b] % 16], k[b])
        assert int((cache.pages != 0).any(-1).sum()) == 2 * 2 * 2


@pytest.mark.parametrize("H,kvh,hd,dtype", [(32, 8, 128, BF), (4, 4, 64, FP)])
def test_append_then_attend_as_a_server_would(H, kvh, hd, dtype):
    """A common prompt appended once, private continuations, then decode steps and a round of lattice
    nodes: every step's output against attention over the tokens' own q, k, v in 64 bits."""
    dexlib = require_gpu()
    ps, theta, B, common = 32, 1e4, 5, 130
    gen = torch.Generator().manual_seed(9)
    private = [1, 60, 17, 128, 33]
    width = 12
    shared = common // ps
    n_pages = shared + B * (width - shared)
    ids = torch.randperm(n_pages, generator=gen).int()
    table = torch.empty((B, width), dtype=torch.int32)
    table[:, :shared] = ids[:shared]
    table[:, shared:] = ids[shared:].view(B, -1)
    cache = dexlib.PagedCache(torch.full((n_pages, 2, kvh, ps, hd), math.nan, dtype=dtype, device="cuda"), table.cuda())
    hist_k = [torch.zeros((0, kvh, hd), dtype=torch.float64) for _ in range(B)]
    hist_v = [torch.zeros((0, kvh, hd), dtype=torch.float64) for _ in range(B)]

    def step(new, rope=None, tree=None, prefix=common, shared_rows=False):
        """Append new[b] tokens to every sequence and attend; returns the worst share of the bound."""
        n = sum(new)
        qkv = torch.randn((n, H + 2 * kvh, hd), generator=gen).to(dtype)
        seq = torch.tensor([b for b in range(B) for _ in range(new[b])], dtype=torch.int32)
        pos = torch.tensor([len(hist_k[b]) + i for b in range(B) for i in range(new[b])], dtype=torch.int32)
        r = pos if rope is None else rope
        dev = qkv.cuda()
        q = cache.append(dev[:, H:H + kvh], dev[:, H + kvh:], seq.cuda(), pos.cuda(), q=dev[:, :H], theta=theta,
                         rope_pos=None if rope is None else rope.cuda())
        start = torch.tensor([0] + list(new)).cumsum(0).int()
        k, v = rotate(qkv[:, H:H + kvh], r, theta), qkv[:, H + kvh:].double()
        qr = rotate(qkv[:, :H], r, theta)
        for b in range(B):
            s = slice(int(start[b]), int(start[b + 1]))
            hist_k[b], hist_v[b] = torch.cat((hist_k[b], k[s])), torch.cat((hist_v[b], v[s]))
        lens = [len(x) for x in hist_k]
        out = cache.attention(q, start.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), max_q=max(new),
                              prefix_len=prefix, tree_mask=None if tree is None else tree.cuda()).cpu().double()
        u = HALF[dtype]
        for b in range(B):
            for i in range(new[b]):
                t, L = int(start[b]) + i, lens[b]
                seen = torch.arange(L) <= L - new[b] + i
                if tree is not None:
                    seen = torch.tensor([j < L - new[b] or bool(int(tree[t]) >> (j - L + new[b]) & 1) for j in range(L)])
                kk = hist_k[b][seen].repeat_interleave(H // kvh, 1)
                vv = hist_v[b][seen].repeat_interleave(H // kvh, 1)
                sc = torch.einsum("hd,jhd->hj", qr[t], kk) * hd ** -0.5
                w = torch.softmax(sc, -1)
                want = torch.einsum("hj,jhd->hd", w, vv)
                # q and k rounded to the cache's type move a score by up to 2u sum|q k| / sqrt(hd), a weight
                # by twice that relatively, and the weights' sum again
                ds = (torch.einsum("hd,jhd->hj", qr[t].abs(), kk.abs()) * hd ** -0.5).amax(-1) * 2.1 * u
                bound = u * want.abs() + (2.0 * torch.expm1(2 * ds) + 2 * u)[:, None] * torch.einsum("hj,jhd->hd", w, vv.abs())
                assert bool(((out[t] - want).abs() <= bound + 1e-6).all())

    # the prompt goes in through sequence 0; the others share its whole pages and copy the last one
    hist = [common, 0, 0, 0, 0]
    step(hist, prefix=0)
    for b in range(1, B):
        hist_k[b], hist_v[b] = hist_k[0].clone(), hist_v[0].clone()
        cache.pages[int(table[b, shared]), :, :, :common % ps] = cache.pages[int(table[0, shared]), :, :, :common % ps]
    step(private)
    for _ in range(3):
        step([1] * B)
    # lattice nodes: a chain of three and two siblings, cache rows apart from rotation positions
    words, rope = [], []
    for b in range(B):
        words += [0b00001, 0b00011, 0b00111, 0b01001, 0b10001]
        rope += [len(hist_k[b]) + d for d in (0, 1, 2, 1, 1)]
    step([5] * B, torch.tensor(rope, dtype=torch.int32), torch.tensor(words, dtype=torch.int64))
