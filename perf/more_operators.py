"""Operators that choose key blocks and share prefixes: their measured cases and plain forms.

Two groups that a server uses next to the block-sparse prefill and decode:

  index     8-bit summaries of 64-token key blocks, kept beside a paged cache
  select    the key blocks of each decode query, by its score against those summaries
  mask      the block mask of a prompt, by the same score between query and key blocks
  shared    one query token per sequence over a prefix that sequences share, read once for all
            of them, and each sequence's own tokens

The plain forms are elementary torch operations in 32 bits, rounded once at the end.  With
`own` set, `run` makes the calls that a program makes of block_sparse_attention_gb300.
"""
import math

import numpy as np
import torch

own = False

F16, BF16 = "float16", "bfloat16"
BLOCK = 64

# ------------------------------------------------------------------------------ cases


def listed():
    return [
        # a decode step: one new token a sequence, so one block of each is summarised again
        dict(name="index_step_64", op="index", batch=64, hkv=8, d=128, dtype=BF16, page=64, lo=1, hi=4096, least=1,
             most=1),
        # prompts of up to 8191 tokens, written into the cache by one prefill
        dict(name="index_prompts_16", op="index", batch=16, hkv=8, d=128, dtype=BF16, page=128, lo=0, hi=0, least=512,
             most=8191),
        # one chat of 16k tokens
        dict(name="select_one_16385", op="select", batch=1, hq=32, hkv=8, d=128, dtype=BF16, page=64, lo=16385,
             hi=16385, chosen=64, sinks=1, recent=2),
        # a server's batch of ragged contexts, 64 blocks for each kv head
        dict(name="select_batch_64", op="select", batch=64, hq=32, hkv=8, d=128, dtype=BF16, page=64, lo=8192,
             hi=65536, chosen=64, sinks=1, recent=2),
        # a few whole books, head dimension 64
        dict(name="select_long_8", op="select", batch=8, hq=24, hkv=8, d=64, dtype=F16, page=256, lo=262144,
             hi=524288, chosen=128, sinks=1, recent=4),
        # a chunk of a prompt after 8192 cached tokens, ragged at both ends, kv heads shared by four
        dict(name="mask_chunk_257", op="mask", batch=1, hq=8, hkv=2, sq=257, sk=8449, d=128, dtype=BF16, causal=True,
             topk=32, sinks=1, recent=2, dense=False),
        # two prompts of 4096 tokens, 16 blocks a row and dense last rows
        dict(name="mask_prompt_4096", op="mask", batch=2, hq=8, hkv=8, sq=4096, sk=4096, d=128, dtype=BF16,
             causal=True, topk=16, sinks=1, recent=1, dense=True),
        # one long prompt of a 32-head model
        dict(name="mask_long_16384", op="mask", batch=1, hq=32, hkv=32, sq=16384, sk=16384, d=128, dtype=BF16,
             causal=True, topk=26, sinks=1, recent=1, dense=True),
        # four users who have just sent their first words after a system prompt
        dict(name="shared_few_4", op="shared", batch=4, groups=1, hq=32, hkv=8, d=128, dtype=BF16, page=64, plo=1999,
             phi=1999, lo=1, hi=200),
        # one long document, 64 questions about it
        dict(name="shared_document_64", op="shared", batch=64, groups=1, hq=32, hkv=8, d=128, dtype=BF16, page=64,
             plo=32768, phi=32768, lo=0, hi=1024),
        # six system prompts in one batch, head dimension 64
        dict(name="shared_prompts_192", op="shared", batch=192, groups=6, hq=16, hkv=8, d=64, dtype=F16, page=128,
             plo=3000, phi=16384, lo=0, hi=1000),
        # a full server over one very long prefix
        dict(name="shared_full_256", op="shared", batch=256, groups=1, hq=32, hkv=8, d=128, dtype=BF16, page=64,
             plo=65521, phi=65521, lo=1, hi=2048),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["index", "select", "mask", "shared"])
    dtype = rng.choice([F16, BF16])
    d = rng.choice([64, 128])
    page = rng.choice([64, 128, 256])
    hkv, group = rng.choice([(1, 1), (1, 8), (2, 4), (4, 1), (8, 4), (8, 2), (5, 3), (2, 7)])
    if op == "index":
        most = _spread(rng, 1, 8191)
        return dict(op=op, batch=_spread(rng, 1, 16 if most > 64 else 64), hkv=hkv, d=d, dtype=dtype, page=page, lo=0,
                    hi=_spread(rng, 1, 4096), least=rng.randint(1, most), most=most)
    sinks, recent = rng.randint(0, 2), rng.randint(0, 3)
    if op == "select":
        hi = _spread(rng, 2048, 262144)
        return dict(op=op, batch=_spread(rng, 1, max(1, min(64, 2 ** 21 // hi))), hq=hkv * group, hkv=hkv, d=d,
                    dtype=dtype, page=page, lo=rng.randint(hi // 2, hi), hi=hi,
                    chosen=sinks + recent + _spread(rng, 1, min(150, hi // BLOCK // 3)), sinks=sinks, recent=recent)
    if op == "mask":
        sk = _spread(rng, 1000, 16384)
        sq = rng.choice([sk, sk, max(400, sk // 3), sk + 37])
        return dict(op=op, batch=rng.choice([1, 2]), hq=hkv * group, hkv=hkv, sq=sq, sk=sk, d=d, dtype=dtype,
                    causal=rng.random() < 0.75, topk=sinks + recent + _spread(rng, 1, sk // BLOCK // 3), sinks=sinks,
                    recent=recent, dense=rng.random() < 0.5)
    batch, phi, hi = _spread(rng, 1, 128), _spread(rng, 1, 32768), _spread(rng, 1, 2048)
    return dict(op=op, batch=batch, groups=min(batch, rng.choice([1, 1, 2, 3, 5])), hq=hkv * group, hkv=hkv, d=d,
                dtype=dtype, page=page, plo=rng.randint(1, phi), phi=phi, lo=rng.randint(0, hi), hi=hi)


# ------------------------------------------------------------------------------ inputs


def _gen(seed, device):
    return torch.Generator(device=device).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=g.device)


def _int(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=g.device)


def _rows(g, dtype, *shape):
    """Queries, keys or values [..., d] as a model writes them: some channels are strong."""
    x = _randn(g, *shape)
    x *= torch.exp(0.5 * _randn(g, *shape[-2:]))
    return x.to(dtype)


def _topics(g, dtype, batch, tokens, heads, d):
    """Rows [batch, tokens, heads, d] of a text whose subject moves on every few dozen tokens."""
    step = 48
    subject = _randn(g, batch, -(-tokens // step), heads, d)
    x = subject.repeat_interleave(step, 1)[:, :tokens] + _randn(g, batch, tokens, heads, d)
    x *= torch.exp(0.5 * _randn(g, heads, d))
    return x.to(dtype)


def _tables(need, most, g, pages=0):
    """A block table over shuffled pages (unused entries -1) and the number of pages that there are."""
    pages = pages or int(need.sum()) + 2
    perm = torch.randperm(pages, generator=g, device=g.device)
    col = torch.arange(most, device=g.device)[None]
    first = (torch.cumsum(need, 0) - need)[:, None]
    return torch.where(col < need[:, None], perm[(first + col).clamp(max=pages - 1)], -1).to(torch.int32), pages


def _ceil(n, by):
    return -(-n // by) if isinstance(n, int) else (n + by - 1) // by


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed, dev)
    op, dt, d, hkv = case["op"], getattr(torch, case["dtype"]), case["d"], case["hkv"]
    s = dict(case=case)
    if op == "mask":
        b, sq, sk = case["batch"], case["sq"], case["sk"]
        # the projections' outputs, [batch, tokens, heads, d], seen as [batch, heads, tokens, d]
        s.update(q=_topics(g, dt, b, sq, case["hq"], d).transpose(1, 2),
                 k=_topics(g, dt, b, sk, hkv, d).transpose(1, 2))
        return s
    b, page = case["batch"], case["page"]
    if op == "index":
        new = _int(g, case["least"], case["most"], b)
        lens = _int(g, case["lo"], case["hi"], b) + new
        most = _ceil(case["hi"] + case["most"], page)
        table, pages = _tables(_ceil(lens, page), most, g, b * most)
        s.update(lens=lens.to(torch.int32), new=new.to(torch.int32), table=table,
                 k=_topics(g, dt, pages, page, hkv, d))
        s["index"] = (torch.zeros(pages, page // BLOCK, hkv, d, dtype=torch.int8, device=dev),
                      torch.zeros(pages, page // BLOCK, hkv, device=dev))
        return s
    lens = _int(g, case["lo"], case["hi"], b)
    if op == "select":
        table, pages = _tables(_ceil(lens, page), _ceil(case["hi"], page), g)
        s.update(q=_rows(g, dt, b, case["hq"], d), lens=lens.to(torch.int32), table=table)
        # the index as earlier steps left it
        s["index"] = _to8(_randn(g, pages, page // BLOCK, hkv, d) * torch.exp(0.5 * _randn(g, hkv, d)))
        return s
    groups = case["groups"]
    cuts = torch.randperm(b - 1, generator=g, device=dev)[:groups - 1].sort().values + 1 if groups > 1 else lens[:0]
    ends = torch.tensor([0, b], device=dev)
    starts = torch.cat((ends[:1], cuts, ends[1:]))
    plens = _int(g, case["plo"], case["phi"], groups)
    need = torch.cat((_ceil(plens, page), _ceil(lens, page)))
    table, pages = _tables(need, _ceil(max(case["phi"], case["hi"]), page), g)
    s.update(starts=starts.to(torch.int32), plens=plens.to(torch.int32), lens=lens.to(torch.int32),
             ptable=table[:groups, :_ceil(case["phi"], page)].contiguous(),
             table=table[groups:, :_ceil(case["hi"], page)].contiguous(), most=int((starts[1:] - starts[:-1]).max()),
             q=_rows(g, dt, b, case["hq"], d), k=_rows(g, dt, pages, page, hkv, d), v=_rows(g, dt, pages, page, hkv, d))
    return s


# ------------------------------------------------------------------------------ block summaries
#
# A block of 64 rows is summarised by its mean in 8 bits.  The rows are added in halves (row i to
# row i + 32, then i + 16 and so on), in 32 bits, so that the sum is the same wherever it is
# taken; the mean's codes are its multiples of a 127th of its largest channel.  A score is the
# whole-number product of two summaries' codes times both scales.  A mean that is not finite has
# codes 0 and an infinite scale: such a key block comes first, such a query scores 0 everywhere.


def _halve(x):
    n = x.shape[-2] // 2
    return x[..., :n, :] + x[..., n:, :]


def _to8(x):
    """Codes int8 and scales of x [..., d] in 32 bits."""
    top = x.abs().amax(-1)
    fine = torch.isfinite(top)
    # divided by a tensor: a division by a plain number is a product with its rounded reciprocal
    scale = torch.where(fine, top, 0.0) / torch.tensor(127.0, device=x.device)
    y = x / torch.where(scale > 0, scale, 1.0)[..., None]
    y = torch.where((fine & (scale > 0))[..., None], torch.round(y).clamp(-127, 127), 0.0)
    return y.to(torch.int8), torch.where(fine, scale, math.inf)


def _summary(x, count):
    """x [..., 64, d] with zeros past `count` [...] rows: the summaries of its blocks."""
    total = _halve(_halve(_halve(_halve(_halve(_halve(x))))))[..., 0, :]
    return _to8(total / count.clamp(min=1).float()[..., None])


def _summaries(x):
    """x [B, H, S, d]: codes [B, H, ceil(S / 64), d] and scales."""
    b, h, n, d = x.shape
    blocks = _ceil(n, BLOCK)
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, blocks * BLOCK - n)).view(b, h, blocks, BLOCK, d)
    return _summary(x, (n - torch.arange(blocks, device=x.device) * BLOCK).clamp(max=BLOCK))


def _best(score, may, must, count):
    """Of the places that `may` allows the `must` ones and the best others, `count` in all; ties go to the lowest."""
    rank = torch.where(must & may, math.inf, torch.where(may, score, -math.inf))
    # infinities among the scores: the class of a place goes before its score
    kind = torch.where(must & may, 2, torch.where(may, 1, 0))
    first = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    order = torch.gather(first, -1, torch.sort(torch.gather(kind, -1, first), dim=-1, descending=True, stable=True).indices)
    place = torch.empty_like(order).scatter_(-1, order, torch.arange(order.shape[-1], device=order.device).expand_as(order))
    return may & (must | (place < count))


# ------------------------------------------------------------------------------ plain forms


def _index(s):
    k, page, dev = s["k"], s["case"]["page"], s["k"].device
    codes, scales = s["index"]
    lens, new = s["lens"].long(), s["new"].long()
    blocks = _ceil(s["case"]["most"], BLOCK) + 1               # a sequence's new tokens lie in so many at most
    at = (lens - new)[:, None] // BLOCK + torch.arange(blocks, device=dev)
    on = (at * BLOCK < lens[:, None]) & (new[:, None] > 0)
    seq, nth = torch.nonzero(on, as_tuple=True)
    at = at[seq, nth]
    count = (lens[seq] - at * BLOCK).clamp(max=BLOCK)
    per = page // BLOCK
    where, sub = s["table"].long()[seq, at // per], at % per
    x = k.view(k.shape[0], per, BLOCK, *k.shape[2:])[where, sub].float().transpose(1, 2)     # [n, Hkv, 64, d]
    x = torch.where(torch.arange(BLOCK, device=dev)[:, None] < count[:, None, None, None], x, 0.0)
    codes[where, sub], scales[where, sub] = _summary(x, count[:, None].expand(x.shape[:2]))
    return codes * scales[..., None]


def _score(dot, scale):
    return torch.where(torch.isinf(scale), math.inf, dot * scale)


def _select(s):
    c, dev = s["case"], s["q"].device
    codes, scales = s["index"]
    b, hkv, per = c["batch"], c["hkv"], c["page"] // BLOCK
    lens = s["lens"].long()
    at = torch.arange(s["table"].shape[1] * per, device=dev)
    n = _ceil(lens, BLOCK)[:, None]
    on = at < n
    where = torch.where(on, s["table"].long()[:, at // per], 0)
    kc, ks = codes[where, at % per].transpose(1, 2), scales[where, at % per].transpose(1, 2)     # [B, Hkv, n, d]
    qc, qs = _to8(s["q"].float().view(b, hkv, -1, c["d"]))
    # whole numbers below 2^24: exact in 32 bits whatever the order
    dot = torch.matmul(qc.float(), kc.float().transpose(2, 3)) * torch.where(torch.isinf(qs), 0.0, qs)[..., None]
    score = _score(dot.amax(2), ks)
    must = (at < c["sinks"]) | (at >= n - c["recent"])
    on = on[:, None].expand(b, hkv, -1)
    picked = _best(score, on, must[:, None] & on, c["chosen"])
    most = min(c["chosen"], at.numel())
    first = torch.sort(torch.where(picked, at, at.numel()), dim=-1).values[..., :most]
    first = torch.where(first < at.numel(), first, -1)
    return torch.nn.functional.pad(first, (0, c["chosen"] - most), value=-1).to(torch.int32)


def _mask(s):
    c, dev = s["case"], s["q"].device
    b, hq, sq, d = s["q"].shape
    hkv, sk = s["k"].shape[1:3]
    (qc, qs), (kc, ks) = _summaries(s["q"]), _summaries(s["k"])
    nq, nk = qc.shape[2], kc.shape[2]
    dot = torch.matmul(qc.float().view(b, hkv, -1, d), kc.float().transpose(2, 3)).view(b, hq, nq, nk)
    dot = dot * torch.where(torch.isinf(qs), 0.0, qs)[..., None]
    score = _score(dot, ks.repeat_interleave(hq // hkv, 1)[:, :, None])
    row, col = torch.arange(nq, device=dev)[:, None], torch.arange(nk, device=dev)[None]
    last = (row * BLOCK + BLOCK - 1).clamp(max=sq - 1) + sk - sq if c["causal"] else torch.full_like(row, sk - 1)
    last = torch.div(last, BLOCK, rounding_mode="floor")                       # the last block that a row sees
    must = (col < c["sinks"]) | (col > last - c["recent"])
    if c["dense"]:
        must = must | (row >= nq - 2)
    may = (col <= last).expand(b, hq, nq, nk)
    return _best(score, may, must.expand_as(may), c["topk"]).to(torch.uint8)


def _softmax_parts(x):
    """exp(x - max), its sum and the max; a row of -inf gives zeros, 0 and -inf."""
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    return e, e.sum(-1, keepdim=True), top


def _attend(q, rows, pages, lens, page):
    """q [n, Hkv, r, d] over each n's first lens tokens of `pages` [n, m]: (sum of p v, sum of p, max)."""
    dev = q.device
    pos = torch.arange(pages.shape[1] * page, device=dev)[None]
    on = pos < lens[:, None]
    where = torch.where(on, pages.long()[:, pos[0] // page], 0)
    k = rows[0][where, pos % page].float().permute(0, 2, 3, 1)
    x = torch.matmul(q / math.sqrt(q.shape[-1]), k)
    del k
    e, total, top = _softmax_parts(torch.where(on[:, None, None], x, -math.inf))
    del x
    return torch.matmul(e, rows[1][where, pos % page].float().transpose(1, 2)), total, top


def _shared(s):
    c, dev = s["case"], s["q"].device
    b, hq, d = s["q"].shape
    hkv, page, most, rows = c["hkv"], c["page"], s["most"], (s["k"], s["v"])
    starts = s["starts"].long()
    q = s["q"].float().view(b, hkv, -1, d)
    # the sequences of a group side by side: one product with the prefix for all their heads
    at = starts[:-1, None] + torch.arange(most, device=dev)
    qg = q[at.clamp(max=b - 1)].transpose(1, 2).flatten(2, 3)                    # [P, Hkv, most G, d]
    parts = [t.view(t.shape[0], hkv, most, hq // hkv, -1).transpose(1, 2)
             for t in _attend(qg, rows, s["ptable"], s["plens"], page)]
    seq = torch.arange(b, device=dev)
    group = torch.searchsorted(starts[1:], seq, right=True)
    o1, l1, m1 = [t[group, seq - starts[group]] for t in parts]
    o2, l2, m2 = _attend(q, rows, s["table"], s["lens"], page)
    top = torch.maximum(m1, m2)
    top = torch.where(top == -math.inf, 0.0, top)
    w1, w2 = torch.exp(m1 - top), torch.exp(m2 - top)
    total = l1 * w1 + l2 * w2
    return ((o1 * w1 + o2 * w2) / torch.where(total == 0, 1.0, total)).view(b, hq, d).to(s["q"].dtype)


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"index": _index, "select": _select, "mask": _mask, "shared": _shared}[op](s)
    import block_sparse_attention_gb300 as bsa
    if op == "index":
        bsa.bsattn_index_update(s["k"], s["lens"], s["new"], s["table"], s["index"])
        return s["index"][0] * s["index"][1][..., None]
    if op == "select":
        return bsa.bsattn_decode_select(s["q"], s["index"], s["lens"], s["table"], c["chosen"], sinks=c["sinks"],
                                        recent=c["recent"])
    if op == "mask":
        return bsa.bsattn_mask_from_qk(s["q"], s["k"], c["topk"], c["causal"], sinks=c["sinks"], recent=c["recent"],
                                       use_dense_for_last_block=c["dense"])
    return bsa.bsattn_decode_shared(s["q"], s["k"], s["v"], s["plens"], s["ptable"], s["starts"], s["lens"],
                                    s["table"])


# ------------------------------------------------------------------------------ work


def work(case):
    op, d, hkv, b = case["op"], case["d"], case["hkv"], case["batch"]
    if op == "index":
        new = b * (case["least"] + case["most"]) / 2
        rows = new + b * min(BLOCK // 2, case["hi"])           # and what stands before them in their first blocks
        blocks = new / BLOCK + b / 2
        return dict(bytes=int(rows * hkv * d * 2 + blocks * (hkv * (d + 4) + 4) + 8 * b), flops=int(rows * hkv * d))
    if op == "select":
        hq = case["hq"]
        blocks = b * ((case["lo"] + case["hi"]) / 2 / BLOCK + 0.5)
        return dict(bytes=int(blocks * (hkv * (d + 4) + 4) + 2 * b * hq * d + 4 * b * hkv * case["chosen"]),
                    flops=int(blocks * hq * d * 2))
    hq = case["hq"]
    if op == "mask":
        sq, sk = case["sq"], case["sk"]
        nq, nk = _ceil(sq, BLOCK), _ceil(sk, BLOCK)
        # under the causal rule row r of blocks sees the blocks up to that of its last position
        last = np.minimum(np.arange(nq, dtype=np.int64) * BLOCK + BLOCK, sq) + sk - sq
        pairs = int(np.clip(-(-last // BLOCK), 0, nk).sum()) if case["causal"] else nq * nk
        return dict(bytes=b * (2 * d * (hq * sq + hkv * sk) + hq * nq * nk),
                    flops=b * (d * (hq * sq + hkv * sk) + 2 * d * hq * pairs))
    prefix, mine = (case["plo"] + case["phi"]) / 2, (case["lo"] + case["hi"]) / 2
    return dict(bytes=int(4 * hkv * d * (case["groups"] * prefix + b * mine) + 4 * b * hq * d),
                flops=int(4 * d * b * hq * (prefix + mine)))


# ------------------------------------------------------------------------------ 64-bit definitions


def _f32(x):
    """x, computed in 64 bits from 32-bit numbers by one operation, as the definition rounds it."""
    return x.float().double()


def _exact8(x):
    """Codes and scales of x [..., d] in 64 bits."""
    top = x.abs().amax(-1, keepdim=True)
    ok = torch.isfinite(top)
    scale = _f32(torch.where(ok, top, 0.0) / torch.full_like(top, 127.0))
    code = torch.where(scale > 0, torch.round(_f32(x / torch.where(scale > 0, scale, 1.0))), 0.0).clamp(-127, 127)
    return torch.where(ok, code, 0.0), torch.where(ok, scale, math.inf)[..., 0]


def _exact_summary(rows):
    """Codes and scale of the n <= 64 rows [..., n, d] of a block."""
    n = rows.shape[-2]
    x = torch.zeros(*rows.shape[:-2], BLOCK, rows.shape[-1], dtype=torch.float64, device=rows.device)
    x[..., :n, :] = rows.double()
    for half in (32, 16, 8, 4, 2, 1):
        x = _f32(x[..., :half, :] + x[..., half:2 * half, :])
    return _exact8(_f32(x[..., 0, :] / torch.full_like(x[..., 0, :], float(n))))


def _exact_blocks(x):
    """Codes and scales of all blocks of x [B, H, S, d]."""
    parts = []
    whole = x.shape[2] // BLOCK
    if whole:
        parts.append(_exact_summary(x[:, :, :whole * BLOCK].unflatten(2, (whole, BLOCK))))
    if x.shape[2] % BLOCK:
        parts.append(_exact_summary(x[:, :, None, whole * BLOCK:]))
    return tuple(torch.cat(p, 2) for p in zip(*parts))


def _exact_scores(qc, qs, kc, ks):
    """Scores [r, n] of query summaries [r, d] against key summaries [n, d]."""
    x = _f32((qc @ kc.T) * torch.where(torch.isinf(qs), 0.0, qs)[:, None])
    return x, torch.where(torch.isinf(ks), math.inf, _f32(x * torch.where(torch.isinf(ks), 0.0, ks)))


def _exact_choice(score, forced, count):
    """The forced places of a row and the best others up to `count`, as a sorted list."""
    forced = sorted(set(forced))
    rest = np.ones(len(score), dtype=bool)
    rest[forced] = False
    left = np.nonzero(rest)[0]
    best = left[np.argsort(-score[left], kind="stable")[:max(count - len(forced), 0)]]
    return sorted(forced + best.tolist())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "index":
        codes, scales = s["index"][0].double(), s["index"][1].double()
        lens, new, table, page = s["lens"].tolist(), s["new"].tolist(), s["table"].tolist(), case["page"]
        for b, n in enumerate(lens):
            first = (n - new[b]) // BLOCK
            for j in range(first, _ceil(n, BLOCK) if new[b] else first):
                p, r = table[b][j * BLOCK // page], j * BLOCK % page
                rows = s["k"][p, r:r + min(BLOCK, n - j * BLOCK)].transpose(0, 1)
                codes[p, r // BLOCK], scales[p, r // BLOCK] = _exact_summary(rows)
        return codes * scales[..., None]
    if op == "select":
        codes, scales = s["index"][0], s["index"][1].double()
        group, per = case["hq"] // case["hkv"], case["page"] // BLOCK
        out = torch.full((case["batch"], case["hkv"], case["chosen"]), -1, dtype=torch.int32)
        for b, n in enumerate(s["lens"].tolist()):
            n = _ceil(n, BLOCK)
            j = torch.arange(n, device=codes.device)
            at = s["table"][b].long()[j // per], j % per
            forced = list(range(min(case["sinks"], n))) + list(range(max(0, n - case["recent"]), n))
            for h in range(case["hkv"]):
                qc, qs = _exact8(s["q"][b, h * group:(h + 1) * group].double())
                x, _ = _exact_scores(qc, qs, codes[at[0], at[1], h].double(), scales[at[0], at[1], h])
                ks = scales[at[0], at[1], h]
                x = torch.where(torch.isinf(ks), math.inf, _f32(x.amax(0) * torch.where(torch.isinf(ks), 0.0, ks)))
                picks = _exact_choice(x.cpu().numpy(), forced, case["chosen"])[:case["chosen"]]
                out[b, h, :len(picks)] = torch.tensor(picks, dtype=torch.int32)
        return out
    if op == "mask":
        (qc, qs), (kc, ks) = _exact_blocks(s["q"]), _exact_blocks(s["k"])
        nq, nk, past = qc.shape[2], kc.shape[2], case["sk"] - case["sq"]
        group = case["hq"] // case["hkv"]
        out = torch.zeros(case["batch"], case["hq"], nq, nk, dtype=torch.uint8)
        for b in range(case["batch"]):
            for h in range(case["hq"]):
                _, x = _exact_scores(qc[b, h], qs[b, h], kc[b, h // group], ks[b, h // group])
                x = x.cpu().numpy()
                for r in range(nq):
                    n = (min(r * BLOCK + BLOCK, case["sq"]) - 1 + past) // BLOCK + 1 if case["causal"] else nk
                    forced = list(range(min(case["sinks"], n))) + list(range(max(0, n - case["recent"]), n))
                    if case["dense"] and r >= nq - 2:
                        forced = list(range(n))
                    if n > 0:
                        out[b, h, r, _exact_choice(x[r, :n], forced, case["topk"])] = 1
        return out
    q, page, hkv = s["q"], case["page"], case["hkv"]
    group, d = case["hq"] // hkv, case["d"]
    starts, lens, plens = s["starts"].tolist(), s["lens"].tolist(), s["plens"].tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)

    def tokens(table, n, h):
        j = torch.arange(n, device=q.device)
        at = table.long()[j // page], j % page
        return s["k"][at[0], at[1], h].double(), s["v"][at[0], at[1], h].double()

    for p, n in enumerate(plens):
        for h in range(hkv):
            k, v = tokens(s["ptable"][p], n, h)
            for b in range(starts[p], starts[p + 1]):
                heads = slice(h * group, (h + 1) * group)
                k2, v2 = tokens(s["table"][b], lens[b], h)
                if n + lens[b] == 0:
                    continue
                x = q[b, heads].double() / math.sqrt(d)
                w = torch.softmax(torch.cat((x @ k.T, x @ k2.T), 1), 1)
                out[b, heads] = w[:, :n] @ v + w[:, n:] @ v2
    return out
