"""Plain 64-bit statements of the paged-serving operators, for the tests of their kernels.

Error bounds.  With u(t) = torch.finfo(t).eps / 2, the largest relative error of one rounding to t, an
attention output o = sum p v / sum p computed with scores in 32 bits, weights rounded to `weights` before
the second product and the result rounded to `dtype` is off by at most

    u(dtype) |o| + (u(weights) + 2 ds + (n + 8) 2^-23) a,      a = sum p |v| / sum p

where ds bounds the error of a score: d products summed in 32 bits (2^-23 each step, as the tensor cores
may truncate) and the scaling, so ds = (d + 4) 2^-23 max_j sum_i |q_i k_ij| / sqrt(d); a relative error of
ds in every weight moves numerator and denominator by that much each, and n terms are summed in 32 bits.
A weight in fp16 below 2^-14 is subnormal: its rounding is off by up to half of their spacing, 2^-25, in
absolute terms.  With the largest weight of a row at least `top` (1 in the prefill; 2^12 in the decodes, which
scale the weights by that, and the sum with them), that adds 2^-25 / top sum |v| over the n keys (the sum of
the weights is at least `top`).  Nothing is added to this but the smallest subnormal of the output's type.
"""
import math

import torch


def half_eps(dtype):
    return torch.finfo(dtype).eps / 2


def attend(q, k, v, on, dtype, weights, top_weight=1.0):
    """q [n, d], k and v [m, d], on [n, m] bool: the outputs [n, d] in 64 bits (0 for a row with no key)
    and the bound on a kernel's error."""
    d = q.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    # masked places may hold anything
    used = on.any(0)[:, None]
    k, v = torch.where(used, k, 0.0), torch.where(used, v, 0.0)
    x = (q @ k.T) / math.sqrt(d)
    size = torch.where(on, (q.abs() @ k.abs().T) / math.sqrt(d), 0.0).amax(1, keepdim=True) if on.shape[1] else \
        torch.zeros(q.shape[0], 1, dtype=torch.float64, device=q.device)
    x = torch.where(on, x, -math.inf)
    top = x.amax(1, keepdim=True) if on.shape[1] else torch.full_like(size, -math.inf)
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(1, keepdim=True)
    total = torch.where(total == 0, 1.0, total)
    out, spread = p @ v / total, p @ v.abs() / total
    ds = (d + 4) * 2.0 ** -23 * size
    n = on.sum(1, keepdim=True)
    bound = half_eps(dtype) * out.abs() + (half_eps(weights) + 2 * ds + (n + 8) * 2.0 ** -23) * spread
    if weights == torch.float16:
        bound = bound + 2.0 ** -25 / top_weight * (on.double() @ v.abs())
    return out, bound + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def check(got, want, bound):
    off = (got.double() - want).abs()
    worst = ((off - bound) / bound.clamp(min=1e-300)).max().item() if off.numel() else 0.0
    assert torch.isfinite(got.double()).all()
    assert bool((off <= bound).all()), f"off by {off.max().item():.3g}, {worst + 1:.3g} times the bound"


def window_prefill(q, k, v, window, sinks):
    """Outputs and bounds [B, Hq, Sq, d] of causal attention with a sliding window and sinks."""
    B, Hq, Sq, _ = q.shape
    group = Hq // k.shape[1]
    Sk = k.shape[2]
    p = torch.arange(Sq, device=q.device)[:, None] + Sk - Sq
    j = torch.arange(Sk, device=q.device)[None]
    on = (j <= p) & ((j < sinks) | (j > p - window))
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b in range(B):
        for h in range(Hq):
            out[b, h], bound[b, h] = attend(q[b, h], k[b, h // group], v[b, h // group], on, q.dtype, q.dtype)
    return out, bound


def decode(q, rows, lens, visible, weights):
    """Outputs and bounds [B, Hq, d] of one query token per sequence.  rows(b, g) -> (k, v) [n, d] of its
    tokens; visible(b, g, n) -> bool [n]."""
    B, Hq, _ = q.shape
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    groups = rows.groups
    for b in range(B):
        n = int(lens[b])
        for g in range(groups):
            at = slice(g * (Hq // groups), (g + 1) * (Hq // groups))
            k, v = rows(b, g, n)
            on = visible(b, g, n)[None].expand(Hq // groups, n)
            out[b, at], bound[b, at] = attend(q[b, at], k, v, on, q.dtype, weights, 2.0 ** 12)
    return out, bound


def windowed(n, window, sinks, device):
    j = torch.arange(n, device=device)
    return (j < sinks) | (j >= n - window)


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def nearest(x, grid):
    """The index of the grid value nearest to each x >= 0, the even index on a tie; past the end the last."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    up = torch.searchsorted(grid, x).clamp(max=grid.numel() - 1)          # first grid value >= x
    down = (up - 1).clamp(min=0)
    a, b = (x - grid[down]).abs(), (grid[up] - x).abs()
    tie = torch.where(down % 2 == 0, down, up)
    return torch.where(x > grid[-1], grid.numel() - 1, torch.where(a == b, tie, torch.where(a < b, down, up)))


def e4m3_grid():
    """All 127 finite magnitudes of e4m3, by code."""
    return [(1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6 for e in range(16) for m in range(8)][:127]


def quantise(x, unit):
    """x [..., d] -> (codes [..., d/2], scales [..., d/16]) uint8 by the format's definition, in 64 bits."""
    x = x.double().unflatten(-1, (-1, 16)) / unit
    grid = e4m3_grid()
    six = torch.full((), 6.0, dtype=torch.float64, device=x.device)
    amax = x.abs().amax(-1)
    scale = nearest(torch.where(torch.isfinite(amax), amax, 0.0) / six, grid)
    s = torch.tensor(grid, dtype=torch.float64, device=x.device)[scale][..., None]
    mag = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0)
    bad = ~torch.isfinite(x).all(-1)
    code = nearest(torch.where(bad[..., None], 0.0, mag), E2M1)
    code = torch.where((x < 0) & (code > 0), code + 8, code).flatten(-2)
    scale = torch.where(bad, 0x7f, scale)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), scale.to(torch.uint8)


def dequantise(codes, scales, unit):
    """The values that codes and scales stand for, in 64 bits (NaN for a scale 0x7f)."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    x = torch.tensor(E2M1 + [-a for a in E2M1], dtype=torch.float64, device=codes.device)[c]
    s = torch.tensor(e4m3_grid() + [math.nan], dtype=torch.float64, device=codes.device)[scales.long()]
    return x * s.repeat_interleave(16, -1) * unit


def plan(cached, new, free, count, table, page, max_tokens):
    """Sequence by sequence on the host: (table, slots, starts, seqlens, free_left, bad, no_space)."""
    table = [list(r) for r in table]
    slots, starts, lens = [-1] * max_tokens, [0], []
    asked, left, bad, full = 0, count, False, False
    for b, (have, more) in enumerate(zip(cached, new)):
        begin = starts[-1]
        starts.append(min(begin + max(more, 0), 2 ** 31 - 1))
        lens.append(have)
        if have < 0 or more < 0:
            bad = True
            continue
        held, need = -(-have // page), -(-(have + more) // page)
        if need > len(table[b]) or begin + more > max_tokens or have + more > 2 ** 31 - 1:
            full = True
            continue
        asked += need - held
        if need > held and asked > count:
            full = True
            continue
        if need > held:
            left = count - asked
        for c in range(held, need):
            table[b][c] = free[count - 1 - (asked - (need - held)) - (c - held)]
        for i in range(more):
            page_no = table[b][(have + i) // page]
            if page_no < 0:
                bad = True
            else:
                slots[begin + i] = page_no * page + (have + i) % page
        lens[-1] = have + more
    return table, slots, starts, lens, left, bad, full
