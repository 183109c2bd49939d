"""Serving operators around the block-sparse attention: their measured cases and plain forms.

Three groups that a paged serving loop uses next to the sparse prefill and decode:

  plan            block tables and slot maps built on the GPU from request lengths
  kv4_append      K/V of new tokens rounded into a paged 4-bit cache, and the rows read back
  kv4_decode      one query token per sequence over that cache (every block, chosen blocks,
                  or a sliding window with sinks)
  window_prefill  causal attention with a sliding window and a few first tokens (sinks)
  window_decode   the same rule for one query token per sequence over a paged 16-bit cache

The plain forms are elementary torch operations in 32 bits, rounded once at the end.  With
`own` set, `run` makes the calls that a program makes of block_sparse_attention_gb300.
"""
import math

import numpy as np
import torch

own = False

F16, BF16 = "float16", "bfloat16"

# ------------------------------------------------------------------------------ cases


def listed():
    return [
        # one decode step of eight running sequences: one new token each
        dict(name="plan_step_8", op="plan", batch=8, page=64, lo=8192, hi=65536, prompts=0, longest=1,
             spare=0),
        # a full scheduler tick: running sequences, and prompts of up to 4096 tokens cut in
        dict(name="plan_mixed_2000", op="plan", batch=2000, page=64, lo=0, hi=16384, prompts=120,
             longest=4096, spare=33),
        # the K/V of one decode step, a few of the batch's rows being padding (slot -1)
        dict(name="append_step_61", op="kv4_append", tokens=61, heads=8, d=128, dtype=BF16, page=64,
             padded=3),
        # the K/V of a batch of prompts
        dict(name="append_prompt_65521", op="kv4_append", tokens=65521, heads=8, d=128, dtype=BF16,
             page=64, padded=0),
        # one user, a context of 16k tokens, every block: what a single chat costs per token
        dict(name="kv4_one_16385", op="kv4_decode", batch=1, hq=32, hkv=8, d=128, dtype=BF16, page=64,
             lo=16385, hi=16385, chosen=0, window=0, sinks=0),
        # eight sequences with 64 chosen blocks for each kv head, as the sparse decode workload has it
        dict(name="kv4_chosen_8", op="kv4_decode", batch=8, hq=32, hkv=8, d=128, dtype=BF16, page=128,
             lo=8192, hi=65536, chosen=64, window=0, sinks=0),
        # sixteen long ragged contexts, every block
        dict(name="kv4_long_16", op="kv4_decode", batch=16, hq=32, hkv=8, d=128, dtype=BF16, page=64,
             lo=8192, hi=65536, chosen=0, window=0, sinks=0),
        # a chunk of a prompt after 8192 cached tokens, ragged at both ends
        dict(name="window_chunk_257", op="window_prefill", batch=1, hq=8, hkv=2, sq=257, sk=8449, d=128,
             dtype=BF16, window=1024, sinks=4),
        # a batch of prompts, head dimension 64
        dict(name="window_batch_4x8191", op="window_prefill", batch=4, hq=16, hkv=16, sq=8191, sk=8191,
             d=64, dtype=F16, window=1024, sinks=4),
        # one long prompt of a 32-head model
        dict(name="window_long_16384", op="window_prefill", batch=1, hq=32, hkv=8, sq=16384, sk=16384,
             d=128, dtype=BF16, window=4096, sinks=4),
        # a decode step of eight sequences with a short window
        dict(name="window_step_8", op="window_decode", batch=8, hq=32, hkv=8, d=128, dtype=BF16, page=64,
             lo=500, hi=65536, window=1024, sinks=4),
        # a decode step of a full server
        dict(name="window_step_192", op="window_decode", batch=192, hq=32, hkv=8, d=128, dtype=BF16,
             page=64, lo=500, hi=16384, window=4096, sinks=64),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "kv4_append", "kv4_decode", "window_prefill", "window_decode"])
    dtype = rng.choice([F16, BF16])
    d = rng.choice([64, 128])
    page = rng.choice([64, 128, 256])
    hkv, group = rng.choice([(1, 1), (1, 8), (2, 4), (4, 1), (8, 4), (8, 2), (5, 3), (2, 7)])
    if op == "plan":
        batch = _spread(rng, 1, 2000)
        return dict(op=op, batch=batch, page=rng.choice([16, 64, 128]), lo=0, hi=_spread(rng, 100, 16384),
                    prompts=rng.randint(0, max(1, batch // 16)), longest=_spread(rng, 1, 4096),
                    spare=rng.randint(0, 300))
    if op == "kv4_append":
        tokens = _spread(rng, 1, 65521)
        return dict(op=op, tokens=tokens, heads=hkv, d=d, dtype=dtype, page=page,
                    padded=rng.randint(0, max(1, tokens // 20)))
    if op == "kv4_decode":
        batch = _spread(rng, 1, 16)
        hi = _spread(rng, 64, 65536)
        kind = rng.choice(["all", "chosen", "window"])
        return dict(op=op, batch=batch, hq=hkv * group, hkv=hkv, d=d, dtype=dtype, page=page,
                    lo=rng.randint(1, hi), hi=hi, chosen=_spread(rng, 1, 96) if kind == "chosen" else 0,
                    window=_spread(rng, 1, 8192) if kind == "window" else 0,
                    sinks=rng.choice([0, 1, 4, 100]) if kind == "window" else 0)
    window, sinks = _spread(rng, 1, 4096), rng.choice([0, 1, 4, 64, 129])
    if op == "window_prefill":
        sk = _spread(rng, 1, 8192)
        sq = rng.choice([sk, sk, max(1, sk // 3), min(sk, 1), sk + 37])
        return dict(op=op, batch=rng.choice([1, 2]), hq=hkv * group, hkv=hkv, sq=sq, sk=sk, d=d,
                    dtype=dtype, window=window, sinks=sinks)
    hi = _spread(rng, 64, 16384)
    return dict(op=op, batch=_spread(rng, 1, 128), hq=hkv * group, hkv=hkv, d=d, dtype=dtype, page=page,
                lo=rng.randint(1, hi), hi=hi, window=window, sinks=sinks)


# ------------------------------------------------------------------------------ inputs


def _gen(seed, device):
    return torch.Generator(device=device).manual_seed(seed)


def _kv(shape, dtype, g):
    """Keys or values as a model writes them: a spread of scales over the channels, some strong."""
    d, dev = shape[-1], g.device
    by_channel = torch.exp(0.5 * torch.randn(shape[-2], d, generator=g, device=dev))
    x = torch.randn(shape, generator=g, device=dev)
    x *= by_channel
    return x.to(dtype)


def _pages(lens, page, most, spare, g):
    """A block table over shuffled pages (unused entries -1) and the number of pages there are."""
    need = (lens + page - 1) // page
    total = int(need.sum()) + spare
    perm = torch.randperm(max(total, 1), generator=g, device=g.device).to(torch.int32)
    col = torch.arange(most, device=g.device)[None]
    first = (torch.cumsum(need, 0) - need)[:, None]
    table = torch.where(col < need[:, None], perm[(first + col).clamp(max=perm.numel() - 1)], -1)
    return table.to(torch.int32).contiguous(), max(total, 1), perm, int(need.sum())


def _lens(case, g):
    return torch.randint(case["lo"], case["hi"] + 1, (case["batch"],), generator=g, device=g.device)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed, dev)
    s = dict(case=case)
    op = case["op"]
    if op == "plan":
        b, page = case["batch"], case["page"]
        cached = _lens(case, g)
        new = torch.ones(b, dtype=torch.int64, device=dev)
        if case["prompts"]:
            at = torch.randperm(b, generator=g, device=dev)[:case["prompts"]]
            new[at] = torch.randint(1, case["longest"] + 1, (at.numel(),), generator=g, device=dev)
            cached[at] = 0
        held, total = (cached + page - 1) // page, cached + new
        need = (total + page - 1) // page
        most = -(-(max(case["hi"], case["longest"]) + 1) // page)
        pool = torch.randperm(int(need.sum()) + 7, generator=g, device=dev).to(torch.int32)
        col = torch.arange(most, device=dev)[None]
        first = (torch.cumsum(held, 0) - held)[:, None]
        table = torch.where(col < held[:, None], pool[(first + col).clamp(max=pool.numel() - 1)], -1)
        s.update(cached=cached.to(torch.int32), new=new.to(torch.int32), table=table.to(torch.int32).contiguous(),
                 free=pool[int(held.sum()):].clone(), tokens=b + case["prompts"] * case["longest"] + case["spare"])
        s["free_count"] = torch.tensor([s["free"].numel()], dtype=torch.int32, device=dev)
        return s
    dt, d = getattr(torch, case["dtype"]), case["d"]
    if op == "kv4_append":
        t, h, page = case["tokens"], case["heads"], case["page"]
        num_pages = -(-t // page) + 3                       # the last page belongs to no sequence
        slots = torch.randperm((num_pages - 1) * page // 16, generator=g, device=dev)[:-(-t // 16)]
        slots = (slots[:, None] * 16 + torch.arange(16, device=dev)).reshape(-1)[:t].contiguous()
        if case["padded"]:
            slots[torch.randperm(t, generator=g, device=dev)[:case["padded"]]] = -1
        s.update(k=_kv((t, h, d), dt, g), v=_kv((t, h, d), dt, g), slots=slots, k_scale=1.0, v_scale=0.5,
                 cache=_cache(num_pages, h, page, d, dev))
        return s
    hq, hkv = case["hq"], case["hkv"]
    if op == "window_prefill":
        b, sq, sk = case["batch"], case["sq"], case["sk"]
        # the projections' outputs, [batch, tokens, heads, d], seen as [batch, heads, tokens, d]
        s.update(q=_kv((b, sq, hq, d), dt, g).transpose(1, 2), k=_kv((b, sk, hkv, d), dt, g).transpose(1, 2),
                 v=_kv((b, sk, hkv, d), dt, g).transpose(1, 2))
        return s
    b, page = case["batch"], case["page"]
    lens = _lens(case, g)
    table, num_pages, _, _ = _pages(lens, page, -(-case["hi"] // page), 2, g)
    s.update(q=_kv((b, hq, d), dt, g), lens=lens.to(torch.int32), table=table)
    if op == "window_decode":
        s.update(k=_kv((num_pages, page, hkv, d), dt, g), v=_kv((num_pages, page, hkv, d), dt, g))
        return s
    cache = _cache(num_pages, hkv, page, d, dev)
    step = max(1, (1 << 27) // (hkv * page * d))
    for p in range(0, num_pages, step):                     # the cache as earlier steps left it
        n = min(step, num_pages - p)
        for codes, scales, by in ((cache[0], cache[1], 1.0), (cache[2], cache[3], 0.5)):
            x = _kv((n, page, hkv, d), dt, g).transpose(1, 2)
            codes[p:p + n], scales[p:p + n] = _to4(x, by)
    s.update(cache=cache, k_scale=1.0, v_scale=0.5, chosen=None)
    if case["chosen"]:
        n = (lens + 63) // 64
        slots = case["chosen"]
        score = torch.rand(b, hkv, max(int(n.max()), slots), generator=g, device=dev)
        score = torch.where(torch.arange(score.shape[2], device=dev) < n[:, None, None], score, -1.0)
        score.scatter_(2, (n - 1)[:, None, None].expand(b, hkv, 1), 2.0)   # the newest block is in
        best, at = score.sort(dim=2, descending=True)
        s["chosen"] = torch.where(best[:, :, :slots] >= 0, at[:, :, :slots], -1).to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------------------------ the 4-bit format
#
# 16 channels of a token's head share a scale.  A scale is amax / 6 rounded to e4m3, a code the
# nearest e2m1 value (ties to even) of x / scale; both in units of a power of two given for all
# keys or all values.  Two codes a byte, the lower channel in the lower half.


def _cache(pages, heads, page, d, dev):
    codes, scales = (pages, heads, page, d // 2), (pages, heads, page, d // 16)
    return tuple(torch.zeros(s, dtype=torch.uint8, device=dev) for s in (codes, scales, codes, scales))


def _to4(x, by):
    """x [..., d] as codes [..., d / 2] and scales [..., d / 16]."""
    x = x.float().unflatten(-1, (-1, 16)) / by
    # divided by a tensor: a division by a plain number is a product with its rounded reciprocal
    scale = (x.abs().amax(-1) / torch.tensor(6.0, device=x.device)).clamp(max=448).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    y = torch.where(s > 0, x / s, torch.zeros_like(x))
    m = y.abs().clamp(max=6)
    unit = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    half = (torch.round(m / unit) * unit * 2).clamp(max=12).to(torch.int64)      # 0 1 2 3 4 6 8 12
    code = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], device=x.device)[half]
    code = (code + torch.where((y < 0) & (half > 0), 8, 0)).flatten(-2)
    return (code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8), scale.view(torch.uint8)


def _from4(codes, scales, by):
    """The values that codes and scales stand for, in 32 bits."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = codes.to(torch.int32)
    x = table[torch.stack((c & 15, c >> 4), -1).flatten(-2)].unflatten(-1, (-1, 16))
    return (x * (scales.view(torch.float8_e4m3fn).float() * by)[..., None]).flatten(-2)


# ------------------------------------------------------------------------------ plain forms


def _plan(s):
    page, most = s["case"]["page"], s["table"].shape[1]
    cached, new = s["cached"].long(), s["new"].long()
    held, need = (cached + page - 1) // page, (cached + new + page - 1) // page
    end = torch.cumsum(new, 0)
    fits = (need <= most) & (end <= s["tokens"])
    asked = torch.where(fits, need - held, 0)
    more = torch.cumsum(asked, 0)
    first = more - asked
    count = s["free_count"].long()
    served = fits & ((asked == 0) | (more <= count))
    col = torch.arange(most, device=held.device)[None]
    fresh = s["free"].long()[(count - 1 - (first[:, None] + col - held[:, None])).clamp(0, s["free"].numel() - 1)]
    take = served[:, None] & (col >= held[:, None]) & (col < need[:, None])
    s["table"].copy_(torch.where(take, fresh, s["table"].long()))
    at = torch.arange(s["tokens"], device=held.device)
    seq = torch.searchsorted(end, at, right=True)
    inside = seq.clamp(max=new.numel() - 1)
    pos = cached[inside] + at - (end - new)[inside]
    slot = s["table"].long()[inside, (pos // page).clamp(0, most - 1)] * page + pos % page
    slots = torch.where((seq < new.numel()) & served[inside], slot, -1)
    starts = torch.cat((torch.zeros_like(end[:1]), end)).to(torch.int32)
    lens = (cached + torch.where(served, new, 0)).to(torch.int32)
    used = torch.where(served & (asked > 0), more, 0).amax()
    return s["table"], slots, starts, lens, (count - used).to(torch.int32)


def _append(s):
    k4, ks, v4, vs = s["cache"]
    slots, page = s["slots"], s["case"]["page"]
    at = torch.where(slots >= 0, slots, k4.shape[0] * page - 1)            # padding: the page of nobody
    where, row = at // page, at % page
    k4[where, :, row], ks[where, :, row] = _to4(s["k"], s["k_scale"])
    v4[where, :, row], vs[where, :, row] = _to4(s["v"], s["v_scale"])
    on = (slots >= 0)[:, None, None]
    k = _from4(k4[where, :, row], ks[where, :, row], s["k_scale"])
    v = _from4(v4[where, :, row], vs[where, :, row], s["v_scale"])
    return torch.where(on, k, 0.0).to(s["k"].dtype), torch.where(on, v, 0.0).to(s["v"].dtype)


def _softmax_rows(x):
    """exp(x - max) and its sum; a row of -inf gives zeros and a sum of one."""
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    return e, torch.where(total == 0, 1.0, total)


def _attend_one(q, k, v, on):
    """q [B, Hq, d], k and v [B, Hkv, n, d] in 32 bits, on [B, Hkv or 1, n]: [B, Hq, d] in 32 bits."""
    b, hq, d = q.shape
    qg = q.float().view(b, k.shape[1], -1, d)
    x = torch.matmul(qg, k.transpose(2, 3)) / math.sqrt(d)
    e, total = _softmax_rows(torch.where(on[:, :, None], x, -math.inf))
    return (torch.matmul(e, v) / total).view(b, hq, d)


def _kv4_decode(s):
    c = s["case"]
    k4, ks, v4, vs = s["cache"]
    b, page, dev = c["batch"], c["page"], s["q"].device
    lens = s["lens"].long()
    if s["chosen"] is not None:
        blocks = s["chosen"].long()
        pos = (blocks[..., None] * 64 + torch.arange(64, device=dev)).flatten(2)          # [B, Hkv, n]
        on = (blocks >= 0).repeat_interleave(64, 2) & (pos < lens[:, None, None])
    else:
        pos = torch.arange(s["table"].shape[1] * page, device=dev)[None, None]
        on = pos < lens[:, None, None]
        if c["window"]:
            on = on & ((pos < c["sinks"]) | (pos >= lens[:, None, None] - c["window"]))
        pos = pos.expand(b, c["hkv"], -1)
    safe = torch.where(on, pos, 0)
    where = s["table"].long()[torch.arange(b, device=dev)[:, None, None], safe // page]
    head, row = torch.arange(c["hkv"], device=dev)[None, :, None], safe % page
    k = _from4(k4[where, head, row], ks[where, head, row], s["k_scale"])
    v = _from4(v4[where, head, row], vs[where, head, row], s["v_scale"])
    return _attend_one(s["q"], k, v, on.expand(b, c["hkv"], -1)).to(s["q"].dtype)


def _window_decode(s):
    c = s["case"]
    b, page, dev = c["batch"], c["page"], s["q"].device
    lens = s["lens"].long()[:, None]
    # the sinks that lie before the window, then the window
    first = torch.arange(c["sinks"], device=dev)[None]
    near = lens - c["window"] + torch.arange(c["window"], device=dev)[None]
    pos = torch.cat((first.expand(b, -1), near), 1)
    on = torch.cat((first < lens - c["window"], near >= 0), 1)
    pos = torch.where(on, pos, 0)
    where = s["table"].long()[torch.arange(b, device=dev)[:, None], pos // page]
    k = s["k"][where, pos % page].float().transpose(1, 2)
    v = s["v"][where, pos % page].float().transpose(1, 2)
    return _attend_one(s["q"], k, v, on[:, None]).to(s["q"].dtype)


def _window_prefill(s):
    c = s["case"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    b, hq, sq, d = q.shape
    hkv, sk = k.shape[1], k.shape[2]
    past, window = sk - sq, min(c["window"], max(sk, 1))
    block = min(max(128, 1 << (window - 1).bit_length()), 1024, sq)     # query rows that share a stretch of keys
    nb = -(-sq // block)
    span = block + window - 1
    # stretch n holds the keys n block + past - window + 1 and on; zeros where there are none
    lo, hi = past - window + 1, (nb - 1) * block + past - window + 1 + span

    def stretches(x):
        x = torch.nn.functional.pad(x[:, :, max(lo, 0):max(0, min(hi, sk))], (0, 0, max(0, -lo), max(0, hi - sk)))
        return x[:, :, :hi - lo].unfold(2, span, block)       # [B, Hkv, nb, d, span]

    qb = torch.nn.functional.pad(q, (0, 0, 0, nb * block - sq)).reshape(b, hkv, hq // hkv, nb, block, d)
    qb = (qb.transpose(2, 3) / math.sqrt(d)).flatten(3, 4)    # [B, Hkv, nb, G block, d]
    x = torch.matmul(qb, stretches(k)).view(b, hkv, nb, -1, block, span)
    dev = q.device
    n = torch.arange(nb, device=dev)[:, None, None] * block
    pos = n + torch.arange(block, device=dev)[:, None] + past                             # [nb, block, 1]
    key = n + lo + torch.arange(span, device=dev)
    on = (key <= pos) & (key > pos - c["window"]) & (key >= 0) & (key < sk)
    x = torch.where(on[:, None], x, -math.inf)
    far = min(c["sinks"], sk)
    if far:
        y = torch.matmul(qb, k[:, :, None, :far].transpose(3, 4)).view(b, hkv, nb, -1, block, far)
        first = torch.arange(far, device=dev)
        y = torch.where(((first <= pos - c["window"]) & (first <= pos))[:, None], y, -math.inf)
        x = torch.cat((y, x), -1)
    e, total = _softmax_rows(x)
    e = e.flatten(3, 4)
    out = torch.matmul(e[..., far:], stretches(v).transpose(3, 4))
    if far:
        out = out + torch.matmul(e[..., :far], v[:, :, None, :far])
    out = (out / total.flatten(3, 4)).view(b, hkv, nb, -1, block, d).transpose(2, 3)
    return out.reshape(b, hq, nb * block, d)[:, :, :sq].to(s["q"].dtype)


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"plan": _plan, "kv4_append": _append, "kv4_decode": _kv4_decode, "window_prefill": _window_prefill,
                "window_decode": _window_decode}[op](s)
    import block_sparse_attention_gb300 as bsa
    if op == "plan":
        return (s["table"],) + tuple(bsa.bsattn_paged_plan(
            s["cached"], s["new"], s["free"], s["free_count"], s["table"], c["page"], s["tokens"]))
    if op == "kv4_append":
        bsa.bsattn_kv4_append(s["k"], s["v"], s["slots"], s["cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return bsa.bsattn_kv4_gather(s["slots"], s["cache"], s["k"].dtype, k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op == "kv4_decode":
        return bsa.bsattn_decode_paged_kv4(s["q"], s["cache"], s["lens"], s["table"], s["chosen"], window=c["window"],
                                           sinks=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op == "window_prefill":
        return bsa.bsattn_prefill_window(s["q"], s["k"], s["v"], c["window"], c["sinks"])
    return bsa.bsattn_decode_window_paged(s["q"], s["k"], s["v"], s["lens"], s["table"], c["window"], c["sinks"])


# ------------------------------------------------------------------------------ work


def work(case):
    op = case["op"]
    if op == "plan":
        b, page = case["batch"], case["page"]
        tokens = b + case["prompts"] * case["longest"] + case["spare"]
        fresh = b // page + case["prompts"] * (case["longest"] // 2 // page + 1)
        # lengths in, starts and lengths out, the last page of each sequence, new pages twice, slots
        return dict(bytes=b * 4 * 5 + fresh * 8 + tokens * 8, flops=tokens)
    d = case["d"]
    if op == "kv4_append":
        n = 2 * case["tokens"] * case["heads"] * d
        return dict(bytes=2 * n * 2 + 2 * (n // 2 + n // 16) + 8 * case["tokens"], flops=4 * n)
    hq, hkv, b = case["hq"], case["hkv"], case["batch"]
    if op == "window_prefill":
        sq, sk, w = case["sq"], case["sk"], case["window"]
        p = np.arange(sq, dtype=np.int64) + sk - sq
        first = np.maximum(p - w + 1, 0)
        seen = np.maximum(p + 1 - first, 0) + np.clip(np.minimum(case["sinks"], first), 0, None) * (p >= 0)
        return dict(bytes=2 * d * b * (2 * hq * sq + 2 * hkv * sk), flops=int(seen.sum()) * 4 * d * b * hq)
    mean = (case["lo"] + case["hi"]) / 2
    n = mean
    if case.get("chosen"):
        n = min(n, case["chosen"] * 64)
    if case["window"]:
        n = min(n, case["window"] + case["sinks"])
    each = d * 2 if op == "window_decode" else d // 2 + d // 16
    return dict(bytes=int(b * (2 * hkv * n * each + 4 * hq * d)), flops=int(b * hq * n * 4 * d))


# ------------------------------------------------------------------------------ 64-bit definitions


def _two_to(e):
    """2^e for whole e, exactly: the exponent field of a 64-bit number."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact4(x, by):
    """The values of the 4-bit format for x, from its definition: grids written out, in 64 bits."""
    x = x.double().unflatten(-1, (-1, 16)) / by

    def nearest(y, bits, least, most):                        # to `bits` fraction bits, exponent >= least
        e = (torch.frexp(y)[1] - 1).clamp(min=least)
        unit = _two_to(e - bits)
        return (torch.round(y / unit) * unit).clamp(max=most)  # round(): half to even

    six = torch.full((), 6.0, dtype=torch.float64, device=x.device)   # a tensor: divided by, not multiplied
    scale = nearest(x.abs().amax(-1, keepdim=True) / six, 3, -6, 448.0)
    m = nearest(torch.where(scale > 0, x.abs() / scale.clamp(min=2.0 ** -9), 0.0), 1, 0, 6.0)
    return (torch.sign(x) * m * scale * by).flatten(-2)


def _value4(codes, scales, by):
    """The same values from a cache's bytes."""
    lo, hi = codes & 15, codes >> 4
    c = torch.stack((lo, hi), -1).flatten(-2).long()
    e, f = (c >> 1) & 3, c & 1
    x = torch.where(e > 0, (1 + 0.5 * f.double()) * _two_to(e - 1), 0.5 * f.double())
    x = torch.where(c >= 8, -x, x)
    b = scales.long()
    e, f = (b >> 3) & 15, (b & 7).double()
    sc = torch.where(e > 0, (1 + f / 8) * _two_to(e - 7), f / 8 * 2.0 ** -6)
    return x * sc.repeat_interleave(16, -1) * by


def _exact_rows(q, k, v, on):
    """softmax over the keys that `on` leaves, in 64 bits: q [n, d], k and v [m, d], on [n, m]."""
    x = (q.double() @ k.double().T) / math.sqrt(q.shape[-1])
    x = x.masked_fill(~on, -math.inf)
    w = torch.softmax(x, -1)
    return torch.nan_to_num(w, nan=0.0) @ v.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(s)
    if op == "kv4_append":
        on = (s["slots"] >= 0)[:, None, None]
        return tuple(torch.where(on, _exact4(s[n], s[n + "_scale"]), 0.0) for n in ("k", "v"))
    c, q = case, s["q"]
    group = c["hq"] // c["hkv"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    if op == "window_prefill":
        sq, sk = c["sq"], c["sk"]
        step = 4096
        for b in range(c["batch"]):
            for i in range(0, sq, step):
                p = torch.arange(i, min(i + step, sq), device=q.device) + sk - sq
                lo = max(0, int(p[0]) - c["window"] + 1)
                j = torch.arange(lo, max(lo, min(sk, int(p[-1]) + 1)), device=q.device)
                j = torch.cat((torch.arange(min(c["sinks"], lo, sk), device=q.device), j))
                on = (j <= p[:, None]) & ((j < c["sinks"]) | (j > p[:, None] - c["window"]))
                if not j.numel():
                    continue
                for h in range(c["hq"]):
                    out[b, h, i:i + step] = _exact_rows(q[b, h, i:i + step], s["k"][b, h // group, j],
                                                        s["v"][b, h // group, j], on)
        return out
    lens, page = s["lens"].tolist(), c["page"]
    for b, n in enumerate(lens):
        j = torch.arange(n, device=q.device)
        if c["window"]:
            j = j[(j < c["sinks"]) | (j >= n - c["window"])]
        for h in range(c["hkv"]):
            if op == "kv4_decode" and c["chosen"]:
                picks = s["chosen"][b, h]
                j = (picks[picks >= 0].long()[:, None] * 64 + torch.arange(64, device=q.device)).flatten()
                j = j[j < n]
            pages, row = s["table"][b].long()[j // page], j % page
            if op == "kv4_decode":
                k4, ks, v4, vs = s["cache"]
                k = _value4(k4[pages, h, row], ks[pages, h, row], s["k_scale"])
                v = _value4(v4[pages, h, row], vs[pages, h, row], s["v_scale"])
            else:
                k, v = s["k"][pages, row, h], s["v"][pages, row, h]
            at = slice(h * group, (h + 1) * group)
            out[b, at] = _exact_rows(q[b, at], k, v, torch.ones(group, j.numel(), dtype=torch.bool, device=q.device))
    return out


def _exact_plan(s):
    """Sequence by sequence, as a scheduler on the host would do it."""
    page, tokens = s["case"]["page"], s["tokens"]
    cached, new = s["cached"].tolist(), s["new"].tolist()
    free, table = s["free"].tolist()[:int(s["free_count"])], s["table"].cpu().numpy().copy()
    slots = np.full(tokens, -1, dtype=np.int64)
    starts, lens, asked, room, left = [0], [], 0, len(free), len(free)
    for b, (have, more) in enumerate(zip(cached, new)):
        begin, total = starts[-1], have + more
        held, need = -(-have // page), -(-total // page)
        starts.append(begin + more)
        fits = need <= table.shape[1] and begin + more <= tokens
        asked += need - held if fits else 0
        if not fits or (need > held and asked > room):
            lens.append(have)
            continue
        for c in range(held, need):
            table[b, c] = free[room - (asked - (need - held)) - 1 - (c - held)]
        left = min(left, room - asked) if need > held else left
        pos = np.arange(have, total)
        slots[begin:begin + more] = table[b, pos // page].astype(np.int64) * page + pos % page
        lens.append(total)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return torch.from_numpy(table), torch.from_numpy(slots), i32(starts), i32(lens), i32([left])
