"""Operators of the paged K/V cache, as measured work: appending keys and values with the
position rotation applied on the way, and attention over a cache whose sequences share a
prefix.

``run`` computes them in their plain form (elementary torch operations in 32 bits) or, where
``own`` is true, by the calls a user makes of ``lossless_depth_adaptive_gb300.PagedCache``.
``exact`` gives the same outputs from the definitions in 64 bits.

Definitions.  A page pool holds ``pages[n_pages, 2, kv_heads, page, head_dim]`` (keys, then
values); position p of sequence b is row ``p % page`` of page ``table[b, p // page]``.

* append: token t of sequence b with cache position p and rotation position r stores
  ``rot(k_t, r)`` and ``v_t`` at p, and ``rot(q_t, r)`` is returned.  ``rot`` turns the pair
  (x_j, x_{j + hd/2}) by the angle ``r * theta^(-2 j / hd)``.
* attend: sequence b has ``len_b`` positions, the last ``n_b`` of which are queries.  Query i
  stands at ``p = len_b - n_b + i`` and sees positions 0..p -- or, with a tree mask, every
  position before ``len_b - n_b`` and those of the last n_b whose bit is set in its word.
  Positions below ``prefix`` are the same for every sequence of the batch.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# query heads, K/V heads, head_dim: this repository's model shapes (32/32 and 32/8 x 128, 4 x 64)
# and two generic ones (a smaller grouped layout, one K/V head for all)
LAYOUTS = ((32, 8, 128), (32, 32, 128), (4, 4, 64), (16, 4, 64), (8, 1, 128))


def _append(name, layout, dtype, page, seqs, past, new, in_dtype="", tree=False, theta=1e4, shape_seed=1):
    h, kvh, hd = layout
    c = {"op": "append", "heads": h, "kv_heads": kvh, "head_dim": hd, "dtype": dtype, "page": page, "seqs": seqs,
         "past_lo": past[0], "past_hi": past[1], "new_lo": new[0], "new_hi": new[1], "in_dtype": in_dtype or dtype,
         "tree": tree, "theta": theta, "shape_seed": shape_seed}
    return dict(c, name=name) if name else c


def _attend(name, layout, dtype, page, seqs, prefix, past, new, tree=False, lse=False, shape_seed=1):
    h, kvh, hd = layout
    c = {"op": "attend", "heads": h, "kv_heads": kvh, "head_dim": hd, "dtype": dtype, "page": page, "seqs": seqs,
         "prefix": prefix, "past_lo": past[0], "past_hi": past[1], "new_lo": new[0], "new_hi": new[1], "tree": tree,
         "lse": lse, "shape_seed": shape_seed}
    return dict(c, name=name) if name else c


def listed():
    gqa, mha, tiny, small, _ = LAYOUTS
    return [
        # one decode step of the 8-sequence batch: the smallest call, all latency
        _append("append decode 8", gqa, "bf16", 16, 8, (2048, 2176), (1, 1), theta=1e6),
        # a serving batch of the 32-head model, one token each
        _append("append decode 64 mha", mha, "fp16", 64, 64, (1, 256), (1, 1)),
        # a prefill pass of several prompts at once, ragged
        _append("append prompts", gqa, "bf16", 64, 8, (0, 0), (1500, 2100), theta=1e6),
        # lattice nodes of a round from fp32 projections: cache rows apart from rotation positions
        _append("append lattice hd64", tiny, "fp16", 32, 13, (17, 500), (3, 15), in_dtype="fp32", tree=True),
        # decode of the 8-sequence batch after a common 2048-token prompt: the smallest call
        _attend("decode 8 prefix 2k", gqa, "bf16", 16, 8, 2048, (1, 128), (1, 1)),
        # a serving batch behind one system prompt
        _attend("decode 64 prefix 8k", gqa, "bf16", 64, 64, 8192, (1, 1024), (1, 1)),
        # the same without grouped heads: one query row per sequence and K/V head
        _attend("decode 32 mha prefix 4k", mha, "fp16", 128, 32, 4096, (1, 512), (1, 1)),
        # many short answers over one long document: bound by the tensor cores
        _attend("decode 256 prefix 32k", gqa, "bf16", 128, 256, 32768, (16, 512), (1, 1)),
        # a round of lattice nodes: several queries per sequence under a tree mask
        _attend("lattice 16 prefix 4k", gqa, "fp16", 64, 16, 4096, (1, 256), (8, 15), tree=True),
        # prompts continued behind the prefix: long query runs
        _attend("prompts 4 prefix 8k", gqa, "bf16", 64, 4, 8192, (0, 0), (300, 700)),
        # one sequence, long context, nothing to share
        _attend("decode 1 context 128k", gqa, "bf16", 64, 1, 0, (131072, 131072), (1, 1)),
        # odd everything: prefix that ends inside a page, ragged short runs, 64-wide heads
        _attend("odd 13 prefix 777 hd64", small, "fp16", 32, 13, 777, (0, 300), (1, 5), lse=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    top = [work(c) for c in listed()]
    top = (max(w["bytes"] for w in top), max(w["flops"] for w in top))
    while True:
        layout, page = rng.choice(LAYOUTS), rng.choice((16, 32, 64, 128, 256))
        dtype = rng.choice(("bf16", "fp16"))
        tree, seed = rng.random() < 0.25, rng.randrange(1 << 30)
        if rng.random() < 0.4:
            new = (1, 1) if rng.random() < 0.5 else (1, _log(rng, 2, 2048))
            tree = tree and new[1] <= 64
            past = _log(rng, 1, 1024)
            c = _append("", layout, dtype, page, _log(rng, 1, 256), (0, past), new,
                        in_dtype=rng.choice(("", "fp32")), tree=tree, theta=rng.choice((1e4, 1e6)), shape_seed=seed)
        else:
            kind = rng.random()
            new = (1, 1) if kind < 0.5 else (1, _log(rng, 2, 24)) if kind < 0.75 else (1, _log(rng, 32, 1500))
            tree = tree and new[1] <= 64
            prefix = 0 if rng.random() < 0.15 else _log(rng, 1, 32768)
            c = _attend("", layout, dtype, page, _log(rng, 1, 256), prefix, (0, _log(rng, 1, 4096)), new, tree=tree,
                        lse=rng.random() < 0.3, shape_seed=seed)
        w = work(c)
        if w["bytes"] <= top[0] and w["flops"] <= top[1] and _pool_rows(c) * 4 * c["kv_heads"] * c["head_dim"] < 6e8:
            return c


def _shape(case):
    """(cached, new) lengths of every sequence, apart from the prefix."""
    rng = random.Random(case["shape_seed"] * 7919 + case["seqs"])
    pick = lambda lo, hi: lo if lo == hi else _log(rng, max(lo, 1), hi) if rng.random() > 0.1 else rng.choice((lo, hi))
    return [(pick(case["past_lo"], case["past_hi"]), pick(case["new_lo"], case["new_hi"]))
            for _ in range(case["seqs"])]


def _parents(case):
    """Tree case: parent of every new token of every sequence (-1: the last cached one)."""
    rng = random.Random(case["shape_seed"] * 104729 + 5)
    return [[rng.randrange(-1, i) if i else -1 for i in range(n)] for _, n in _shape(case)]


def _pool_rows(case):
    return case.get("prefix", 0) + sum(p + n + case["page"] for p, n in _shape(case))


def work(case):
    h, kvh, hd = case["heads"], case["kv_heads"], case["head_dim"]
    lens = _shape(case)
    t = sum(n for _, n in lens)
    if case["op"] == "append":
        size = 4 if case["in_dtype"] == "fp32" else 2
        return {"bytes": t * ((h + 2 * kvh) * hd * (size + 2) + 12), "flops": t * (h + kvh) * hd * 3}
    rows = case["prefix"] + sum(p + n for p, n in lens)
    bytes_ = rows * 2 * kvh * hd * 2 + t * h * (hd * 4 + (4 if case["lse"] else 0)) + rows // case["page"] * 4
    if case["tree"]:
        pairs = 0
        for (p, n), par in zip(lens, _parents(case)):
            depth = []
            for i in range(n):
                depth.append(1 + (depth[par[i]] if par[i] >= 0 else 0))
            pairs += n * (case["prefix"] + p) + sum(depth)
    else:
        pairs = sum(n * (case["prefix"] + p) + n * (n + 1) // 2 for p, n in lens)
    return {"bytes": bytes_, "flops": 4 * hd * h * pairs}


def prepare(case, seed):
    h, kvh, hd, page, dt = (case[k] for k in ("heads", "kv_heads", "head_dim", "page", "dtype"))
    dt = DTYPES[dt]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = np.random.default_rng(seed)
    lens, prefix = _shape(case), case.get("prefix", 0)
    seq_len = np.array([prefix + p + n for p, n in lens], dtype=np.int64)
    n_new = np.array([n for _, n in lens], dtype=np.int64)
    start = np.concatenate(([0], np.cumsum(n_new)))
    t = int(start[-1])
    # pages in no order, those of the whole prefix pages shared by every row of the table
    shared = prefix // page
    width = int(-(-seq_len.max() // page)) + 1
    need = [int(-(-n // page)) - shared for n in seq_len]
    ids = rnd.permutation(shared + sum(need) + 3)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    table[:, :shared] = ids[:shared]
    at = shared
    for b, n in enumerate(need):
        table[b, shared:shared + n] = ids[at:at + n]
        at += n
    pages = torch.randn((len(ids), 2, kvh, page, hd), generator=gen, device="cuda", dtype=dt)
    if prefix % page:   # every sequence holds its own copy of the page in which the prefix ends
        src = pages[int(table[0, shared]), :, :, :prefix % page].clone()
        pages[torch.from_numpy(table[:, shared].astype(np.int64)).cuda(), :, :, :prefix % page] = src
    seq = np.repeat(np.arange(len(lens)), n_new)
    local = np.arange(t) - start[seq]
    s = {"case": case, "pages": pages, "table": torch.from_numpy(table).cuda(), "lens": seq_len.tolist(),
         "new": n_new.tolist(), "start": start.tolist()}
    bits = None
    if case["tree"]:
        bits, depth = np.zeros(t, dtype=np.uint64), np.zeros(t, dtype=np.int64)
        for b, par in enumerate(_parents(case)):
            for i, p in enumerate(par):
                k = start[b] + i
                bits[k] = (bits[start[b] + p] if p >= 0 else np.uint64(0)) | np.uint64(1 << i)
                depth[k] = depth[start[b] + p] + 1 if p >= 0 else 0
    if case["op"] == "append":
        pos = seq_len[seq] - n_new[seq] + local
        rope = seq_len[seq] - n_new[seq] + depth if case["tree"] else pos
        qkv = torch.randn((t, (h + 2 * kvh) * hd), generator=gen, device="cuda", dtype=DTYPES[case["in_dtype"]])
        s.update(qkv=qkv, seq=torch.from_numpy(seq.astype(np.int32)).cuda(),
                 pos=torch.from_numpy(pos.astype(np.int32)).cuda(), rope=torch.from_numpy(rope.astype(np.int32)).cuda(),
                 q_out=torch.zeros((t, h, hd), device="cuda", dtype=dt))
    else:
        s.update(q=torch.randn((t, h, hd), generator=gen, device="cuda", dtype=dt),
                 q_start=torch.from_numpy(start.astype(np.int32)).cuda(),
                 seq_len=torch.from_numpy(seq_len.astype(np.int32)).cuda(),
                 tree=None if bits is None else torch.from_numpy(bits.view(np.int64)).cuda(),
                 out=torch.zeros((t, h, hd), device="cuda", dtype=dt),
                 lse=torch.zeros((t, h), device="cuda", dtype=torch.float32) if case["lse"] else None)
    if own:
        import lossless_depth_adaptive_gb300 as dex
        s["cache"] = dex.PagedCache(s["pages"], s["table"])
        if case["op"] == "attend":
            s["workspace"] = s["cache"].attention_workspace(s["q"], max_q=int(n_new.max()), prefix_len=prefix)
    return s


def run(s):
    case = s["case"]
    h, kvh, hd = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        t = s["qkv"].shape[0]
        q, k, v = s["qkv"].split((h * hd, kvh * hd, kvh * hd), dim=1)
        q, k, v = q.view(t, h, hd), k.view(t, kvh, hd), v.view(t, kvh, hd)
        if own:
            s["cache"].append(k, v, s["seq"], s["pos"], q=q, q_out=s["q_out"], theta=case["theta"],
                              rope_pos=s["rope"] if case["tree"] else None)
        else:
            _plain_append(s, q, k, v)
        return [s["pages"], s["q_out"]]
    if own:
        s["cache"].attention(s["q"], s["q_start"], s["seq_len"], max_q=max(s["new"]), prefix_len=case["prefix"],
                             tree_mask=s["tree"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    else:
        _plain_attend(s)
    return [s["out"], s["lse"]] if case["lse"] else [s["out"]]


def _plain_append(s, q, k, v):
    case, page = s["case"], s["case"]["page"]
    hd = case["head_dim"]
    j = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    angle = s["rope"].double()[:, None] * torch.exp(j * (-2.0 / hd * math.log(case["theta"])))
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rot(x):
        a, b = x.float().chunk(2, dim=-1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)

    pos = s["pos"].long()
    page_id = s["table"][s["seq"].long(), pos // page].long()
    dt = s["pages"].dtype
    s["pages"][page_id, 0, :, pos % page] = rot(k).to(dt)
    s["pages"][page_id, 1, :, pos % page] = v.to(dt)
    s["q_out"].copy_(rot(q))


def _plain_attend(s):
    case, page = s["case"], s["case"]["page"]
    h, kvh, hd = case["heads"], case["kv_heads"], case["head_dim"]
    for b, (length, n) in enumerate(zip(s["lens"], s["new"])):
        j = torch.arange(length, device="cuda")
        page_id, row = s["table"][b].long()[j // page], j % page
        keys, values = (s["pages"][page_id, c, :, row].float().permute(1, 0, 2) for c in (0, 1))   # [kvh, length, hd]
        for i0 in range(0, n, 512):
            i1 = min(n, i0 + 512)
            rows = slice(s["start"][b] + i0, s["start"][b] + i1)
            q = s["q"][rows].float().view(i1 - i0, kvh, h // kvh, hd).permute(1, 2, 0, 3).reshape(kvh, -1, hd)
            score = torch.matmul(q, keys.transpose(1, 2)).view(kvh, h // kvh, i1 - i0, length) * (1.0 / math.sqrt(hd))
            behind = j[None, :] - (length - n)
            if case["tree"]:
                seen = (behind < 0) | ((s["tree"][rows][:, None] >> behind.clamp(0, 63)) & 1).bool() & (behind >= 0)
            else:
                seen = behind <= torch.arange(i0, i1, device="cuda")[:, None]
            score = torch.where(seen, score, -math.inf)
            top = score.amax(dim=-1, keepdim=True)
            weight = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
            total = weight.sum(dim=-1, keepdim=True)
            out = torch.matmul(weight.view(kvh, -1, length), values).view(kvh, h // kvh, i1 - i0, hd)
            out = torch.where(total > 0, out / total, 0.0)
            s["out"][rows] = out.permute(2, 0, 1, 3).reshape(i1 - i0, h, hd).to(s["out"].dtype)
            if s["lse"] is not None:
                s["lse"][rows] = (top + torch.log(total)).squeeze(-1).permute(2, 0, 1).reshape(i1 - i0, h)


def exact(case, seed):
    """The same outputs in 64 bits, key by key position rather than page by page."""
    global own
    kept, own = own, False
    s = prepare(case, seed)
    own = kept
    h, kvh, hd, page = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    g = h // kvh
    table = s["table"].cpu().numpy()
    if case["op"] == "append":
        pages, qkv = s["pages"].double(), s["qkv"].double()
        turn = torch.tensor([case["theta"] ** (-2.0 * k / hd) for k in range(hd // 2)], device="cuda",
                            dtype=torch.float64)
        phase = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), s["rope"].double()[:, None] * turn)
        x = qkv.view(qkv.shape[0], h + 2 * kvh, hd)
        z = torch.complex(x[:, :h + kvh, :hd // 2], x[:, :h + kvh, hd // 2:]) * phase[:, None]
        turned = torch.cat((z.real, z.imag), dim=-1)
        flat = pages.permute(0, 3, 1, 2, 4)   # [page, row, 2, kvh, hd], a view
        seq, pos = s["seq"].tolist(), s["pos"].tolist()
        where = torch.tensor([[int(table[b, p // page]), p % page] for b, p in zip(seq, pos)], device="cuda")
        flat[where[:, 0], where[:, 1]] = torch.stack((turned[:, h:], x[:, h + kvh:]), dim=1)
        return [pages, turned[:, :h].contiguous()]
    out = torch.zeros((len(s["q"]), h, hd), device="cuda", dtype=torch.float64)
    lse = torch.zeros((len(s["q"]), h), device="cuda", dtype=torch.float64)
    for b in range(case["seqs"]):
        length, n, r0 = s["lens"][b], s["new"][b], s["start"][b]
        ids = torch.from_numpy(table[b, :-(-length // page)].astype(np.int64)).cuda()
        for kv in range(kvh):
            dense = s["pages"][ids][:, :, kv].double().permute(1, 0, 2, 3).reshape(2, -1, hd)[:, :length]
            for i0 in range(0, n, 256):
                i1 = min(n, i0 + 256)
                q = s["q"][r0 + i0:r0 + i1, kv * g:(kv + 1) * g].double().reshape(-1, hd)
                logits = (q @ dense[0].T / math.sqrt(hd)).view(i1 - i0, g, length)
                hidden = torch.zeros((i1 - i0, length), dtype=torch.bool, device="cuda")
                for i in range(i0, i1):
                    if case["tree"]:
                        word = int(s["tree"][r0 + i]) & (2 ** 64 - 1)
                        hidden[i - i0, length - n:] = torch.tensor([not word >> k & 1 for k in range(n)])
                    else:
                        hidden[i - i0, length - n + i + 1:] = True
                logits.masked_fill_(hidden[:, None], -math.inf)
                norm = torch.logsumexp(logits, dim=-1, keepdim=True)
                prob = torch.exp(logits - torch.where(norm > -math.inf, norm, 0.0))
                out[r0 + i0:r0 + i1, kv * g:(kv + 1) * g] = (prob.view(-1, length) @ dense[1]).view(i1 - i0, g, hd)
                lse[r0 + i0:r0 + i1, kv * g:(kv + 1) * g] = norm.squeeze(-1)
    return [out, lse] if case["lse"] else [out]
