"""Plain 64-bit statements of block summaries, block choices and attention over a shared prefix.

Summaries and scores are defined to the last bit: every step is one operation on 32-bit numbers, rounded to
nearest.  Here each step is taken in 64 bits, where sums, products and quotients of 32-bit numbers round to
the same 32-bit number as the exact result does (53 >= 2 * 24 + 2 bits), and then rounded to 32 bits.
"""
import math

import torch

import serving_reference as serving

BLOCK = 64


def _round(x):
    return x.float().double()


def quantise(mean):
    """[..., d] (64-bit values of 32-bit numbers) -> (codes [..., d], scales [...]) in 64 bits."""
    top = mean.abs().amax(-1)
    finite = torch.isfinite(mean).all(-1)
    scale = _round(torch.where(finite, top, 0.0) / torch.full_like(top, 127.0))
    safe = torch.where(scale > 0, scale, 1.0)[..., None]
    codes = torch.round(_round(torch.where(finite[..., None], mean, 0.0) / safe)).clamp(-127, 127)
    codes = torch.where((scale > 0)[..., None], codes, 0.0)
    return codes, torch.where(finite, scale, math.inf)


def summary(rows):
    """Rows [..., n, d], 1 <= n <= 64, of a block."""
    n = rows.shape[-2]
    x = torch.zeros(*rows.shape[:-2], BLOCK, rows.shape[-1], dtype=torch.float64, device=rows.device)
    x[..., :n, :] = rows.double()
    half = BLOCK // 2
    while half:
        x = _round(x[..., :half, :] + x[..., half:, :])
        half //= 2
    return quantise(_round(x[..., 0, :] / torch.full_like(x[..., 0, :], float(n))))


def summaries(x):
    """[..., S, d] -> codes [..., blocks, d] and scales [..., blocks]."""
    parts = [summary(x[..., at:at + BLOCK, :]) for at in range(0, x.shape[-2], BLOCK)]
    return torch.stack([p[0] for p in parts], -2), torch.stack([p[1] for p in parts], -1)


def scores(qc, qs, kc, ks):
    """[n] scores of key summaries [n, d] for a group of query summaries [G, d]."""
    qs = torch.where(torch.isinf(qs), 0.0, qs)
    best = _round((qc @ kc.T) * qs[:, None]).amax(0)
    return torch.where(torch.isinf(ks), math.inf, _round(best * torch.where(torch.isinf(ks), 0.0, ks)))


def choice(score, may, forced, count):
    """Sorted places: those of `forced` that `may` allows, then the best others up to `count`."""
    place = [j for j in range(len(score)) if may[j]]
    picked = [j for j in place if j in forced]
    others = sorted((j for j in place if j not in forced), key=lambda j: (-score[j], j))
    return sorted(picked + others[:max(0, count - len(picked))])


def select(q, codes, scales, lens, table, max_sel, sinks, recent, page):
    """bsattn_decode_select on the host: int32 [B, Hkv, max_sel]."""
    B, Hq, _ = q.shape
    pages, per, hkv, _ = codes.shape
    out = torch.full((B, hkv, max_sel), -1, dtype=torch.int32)
    qc, qs = quantise(q.double())
    codes, scales = codes.double(), scales.double()
    for b in range(B):
        n = -(-min(max(int(lens[b]), 0), table.shape[1] * page) // BLOCK)
        where = [int(table[b, j // per]) for j in range(n)]
        may = [0 <= p < pages for p in where]
        rows = [(p if ok else 0) * per + j % per for j, (p, ok) in enumerate(zip(where, may))]
        forced = set(range(min(sinks, n))) | set(range(max(0, n - recent), n))
        for g in range(hkv):
            at = slice(g * (Hq // hkv), (g + 1) * (Hq // hkv))
            x = scores(qc[b, at], qs[b, at], codes.flatten(0, 1)[rows, g], scales.flatten(0, 1)[rows, g]) if n else []
            picks = choice([float(v) for v in x], may, forced, max_sel)[:max_sel]
            out[b, g, :len(picks)] = torch.tensor(picks, dtype=torch.int32)
    return out


def mask(q, k, topk, causal, sinks, recent, dense):
    """bsattn_mask_from_qk on the host: uint8 [B, Hq, nq, nk]."""
    B, Hq, Sq, _ = q.shape
    hkv, Sk = k.shape[1:3]
    (qc, qs), (kc, ks) = summaries(q), summaries(k)
    nq, nk = qc.shape[2], kc.shape[2]
    out = torch.zeros(B, Hq, nq, nk, dtype=torch.uint8)
    for b in range(B):
        for h in range(Hq):
            g = h // (Hq // hkv)
            for r in range(nq):
                x = scores(qc[b, h, r:r + 1], qs[b, h, r:r + 1], kc[b, g], ks[b, g]).tolist()
                n = nk
                if causal:
                    n = (min(r * BLOCK + BLOCK, Sq) - 1 + Sk - Sq) // BLOCK + 1
                n = max(n, 0)
                forced = set(range(min(sinks, n))) | set(range(max(0, n - recent), n))
                if dense and r >= nq - 2:
                    forced = set(range(n))
                out[b, h, r, choice(x[:n], [True] * n, forced, topk)] = 1
    return out


def shared(q, k_pages, v_pages, plens, ptable, starts, lens, table):
    """Outputs and bounds [B, Hq, d] of bsattn_decode_shared (see serving_reference for the bound)."""
    B, Hq, d = q.shape
    page, hkv = k_pages.shape[1], k_pages.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)

    def rows(pages, n):
        j = torch.arange(n, device=q.device)
        where = pages.long()[j // page]
        ok = (where >= 0) & (where < k_pages.shape[0])
        return where[ok], (j % page)[ok]

    for p in range(len(plens)):
        pw, pr = rows(ptable[p], int(plens[p]))
        for b in range(int(starts[p]), int(starts[p + 1])):
            w, r = rows(table[b], int(lens[b]))
            w, r = torch.cat((pw, w)), torch.cat((pr, r))
            for g in range(hkv):
                at = slice(g * (Hq // hkv), (g + 1) * (Hq // hkv))
                k, v = k_pages[w, r, g], v_pages[w, r, g]
                on = torch.ones(Hq // hkv, len(w), dtype=torch.bool, device=q.device)
                # the largest weight of each part of the keys is 1 or more, and a row's result the mean of its parts'
                out[b, at], bound[b, at] = serving.attend(q[b, at], k, v, on, q.dtype, q.dtype, 1.0)
    return out, bound
