"""Plain 64-bit forms of the paged-cache operators and the bounds their kernels are held to
(not collected: no test_ prefix)."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # finfo.eps / 2


def rotate(x, rope, theta):
    """x [tokens, heads, hd] turned by rope[t] * theta^(-2j/hd), in fp64 (theta 0: unchanged)."""
    x = x.double()
    if theta == 0:
        return x
    hd = x.shape[-1]
    ang = rope.double()[:, None] * torch.tensor([theta ** (-2.0 * j / hd) for j in range(hd // 2)], dtype=torch.float64)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x[..., :hd // 2], x[..., hd // 2:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def rotate_bound(x, dtype):
    """Largest error of a rotated, rounded row: half a step of the result, the products and sum in
    fp32 and an angle known to 2^-22 (fixed point to 32 bits, sin and cos to 2 ulp)."""
    x = x.double().abs()
    hd = x.shape[-1]
    both = x[..., :hd // 2] + x[..., hd // 2:]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0   # half a subnormal step
    return (HALF[dtype] + 2.0 ** -21) * torch.cat((both, both), -1) + tiny


def gather(pages, table_row, length, prefix_len=0, prefix_row=None):
    """K, V of one sequence as fp64 [length, kvh, hd]."""
    ps = pages.shape[3]
    j = torch.arange(length)
    ids = table_row[j // ps].long() if length else torch.zeros(0, dtype=torch.long)
    if prefix_len and length:
        m = min(prefix_len, length)
        ids[:m] = prefix_row[j[:m] // ps].long()
    return pages[ids, 0, :, j % ps].double(), pages[ids, 1, :, j % ps].double()


def attention(pages, table, q, q_start, seq_len, prefix_len=0, prefix_table=None, tree=None, scale=None):
    """fp64 attention and, per element, the error allowed to a kernel of this arithmetic.

    Returns out, lse, bound_out, bound_lse (NaN rows where no sequence owns the token).  All on the CPU."""
    n_tok, H, hd = q.shape
    kvh = pages.shape[2]
    G = H // kvh
    scale = hd ** -0.5 if scale is None else scale
    out = torch.full((n_tok, H, hd), math.nan, dtype=torch.float64)
    lse = torch.full((n_tok, H), math.nan, dtype=torch.float64)
    b_out, b_lse = out.clone(), lse.clone()
    u = HALF[q.dtype]
    tiny = 2.0 ** -24 if q.dtype == torch.float16 else 0.0
    prow = table[0] if prefix_table is None else prefix_table
    for b in range(len(seq_len)):
        q0, q1, length = int(q_start[b]), int(q_start[b + 1]), int(seq_len[b])
        n = q1 - q0
        if n <= 0:
            continue
        K, V = gather(pages, table[b], length, prefix_len, prow)
        j = torch.arange(length)
        first = length - n
        for h in range(H):
            qq = q[q0:q1, h].double()
            k, v = K[:, h // G], V[:, h // G]
            s = qq @ k.T * scale
            mag = qq.abs() @ k.abs().T * abs(scale)     # sum |q k|: the scores' rounding is relative to it
            if tree is None:
                seen = j[None] <= first + torch.arange(n)[:, None]
            else:
                seen = torch.stack([torch.tensor([jj < first or bool((int(tree[q0 + i]) >> (jj - first)) & 1)
                                                  for jj in range(length)], dtype=torch.bool) for i in range(n)]) \
                    if length else torch.zeros((n, 0), dtype=torch.bool)
            s = s.masked_fill(~seen, -math.inf)
            L = torch.logsumexp(s, -1) if length else torch.full((n,), -math.inf, dtype=torch.float64)
            w = torch.exp(s - torch.where(torch.isinf(L), torch.zeros_like(L), L)[:, None])
            o = w @ v
            out[q0:q1, h], lse[q0:q1, h] = o, L
            # scores: hd products summed in fp32 (and the tensor cores' sum, which may truncate:
            # four times the rounding error); an exponential is off by that much relatively, plus
            # 2^-21 of its own; sums run over tiles of at most 128 keys and then over the tiles
            ds = torch.where(seen, mag, torch.zeros_like(mag)).amax(-1) * 4 * (hd / 16 + 4) * 2.0 ** -24 \
                + torch.where(seen, s.abs(), torch.zeros_like(s)).amax(-1) * 2.0 ** -22 if length \
                else torch.zeros(n, dtype=torch.float64)
            sums = (128 + length / 64) * 4 * 2.0 ** -24
            A = w @ v.abs()
            # probabilities rounded to the cache's type in the numerator (u); both sums in fp32
            b_out[q0:q1, h] = u * (1 + u) * o.abs() + (u + 4 * ds + 2 * sums + 2.0 ** -19)[:, None] * A + tiny
            b_lse[q0:q1, h] = 2 * ds + sums + 2.0 ** -19 + 2.0 ** -21 * torch.where(torch.isinf(L), torch.zeros_like(L),
                                                                                 L).abs()
    return out, lse, b_out, b_lse
