"""The paged 4-bit cache: page plan, append, gather and decode, against their 64-bit statements."""
import pytest
import torch

import serving_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def bsa():
    import block_sparse_attention_gb300 as m
    m.load()
    return m


def _rand(*shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


# ------------------------------------------------------------------------- plan

def _check_plan(bsa, cached, new, page, max_pages, free, count, max_tokens, table):
    dev = "cuda"
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    t = i32(table) if table else torch.zeros(0, max_pages, dtype=torch.int32, device=dev)
    got = bsa.bsattn_paged_plan(i32(cached), i32(new), i32(free), i32([count]), t, page, max_tokens, ws=ws)
    want = ref.plan(cached, new, free, count, table, page, max_tokens)
    assert t.tolist() == want[0]
    assert got[0].tolist() == want[1]
    assert got[1].tolist() == want[2]
    assert got[2].tolist() == want[3]
    assert got[3].tolist() == [want[4]]
    status = bsa.bsattn_get_device_status(ws)
    assert status == (bsa.BSATTN_ERR_BAD_INDEX if want[5] else 0) | (bsa.BSATTN_ERR_NO_SPACE if want[6] else 0)
    return want


def _case(B, page, max_pages, seed, most_new=40, holes=False):
    g = torch.Generator().manual_seed(seed)
    cached = torch.randint(0, max(1, max_pages * page - most_new), (B,), generator=g).tolist()
    new = torch.randint(0, most_new + 1, (B,), generator=g).tolist()
    pages = torch.randperm(B * max_pages + 5, generator=g).tolist()
    table, at = [], 0
    for n in cached:
        held = -(-n // page)
        table.append(pages[at:at + held] + [-1] * (max_pages - held))
        at += held
    if holes:
        table[B // 2][0] = -1
    return cached, new, table, pages[at:]


@pytest.mark.parametrize("B,page,max_pages,most_new", [(1, 64, 4, 1), (8, 64, 20, 1), (3, 16, 9, 100), (200, 1, 30, 9),
                                                       (511, 64, 7, 300), (700, 48, 5, 20), (5000, 16, 3, 7)])
def test_plan_serves_everyone(bsa, B, page, max_pages, most_new):
    cached, new, table, free = _case(B, page, max_pages, seed=B, most_new=most_new)
    want = _check_plan(bsa, cached, new, page, max_pages, free, len(free), sum(new) + 37, table)
    assert not want[5] and not want[6]


def test_plan_first_tokens_and_nothing(bsa):
    _check_plan(bsa, [0, 0, 5], [0, 1, 0], 4, 3, [9, 8, 7], 3, 4, [[-1] * 3, [-1] * 3, [1, 2, -1]])
    _check_plan(bsa, [], [], 4, 3, [9], 1, 5, [])
    _check_plan(bsa, [3], [0], 4, 1, [], 0, 0, [[0]])
    _check_plan(bsa, [4], [4], 4, 2, [6, 5], 2, 4, [[0, -1]])      # a page ends exactly with the cache


def test_plan_without_room(bsa):
    """Out of pages: those that came first are served, and those that need no page."""
    cached, new, table, free = _case(50, 16, 12, seed=2, most_new=60)
    for count in (0, 1, 17, 40, len(free)):
        want = _check_plan(bsa, cached, new, 16, 12, free, count, sum(new), table)
    tight = _check_plan(bsa, cached, new, 16, 12, free, len(free), sum(new) // 2, table)
    assert tight[6] and -1 in tight[1]
    short = [r[:6] for r in table]
    short = [r + [-1] * (6 - len(r)) for r in short]
    assert _check_plan(bsa, cached, new, 16, 6, free, len(free), sum(new), short)[6] and not want[6]


def test_plan_reports_bad_input(bsa):
    cached, new, table, free = _case(20, 16, 12, seed=3)
    cached[4], new[9] = -1, -7
    assert _check_plan(bsa, cached, new, 16, 12, free, len(free), sum(max(n, 0) for n in new), table)[5]
    cached, new, table, free = _case(20, 16, 12, seed=4, holes=True)
    cached[10] = max(cached[10], 1)
    new[10], cached[10] = 3, 5                      # tokens that go into the unmapped page
    table[10] = [-1] * 12
    assert _check_plan(bsa, cached, new, 16, 12, free, len(free), sum(new), table)[5]
    huge = 2 ** 31 - 1                              # sums past 32 bits
    assert _check_plan(bsa, [0, huge, 3], [huge, huge, 1], 1 << 20, 4, [1, 2, 3], 3, 50, [[-1] * 4] * 3)[6]


def test_plan_is_captured_and_runs_on_any_stream(bsa):
    cached, new, table, free = _case(300, 16, 12, seed=5)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c, n, f, k, t = i32(cached), i32(new), i32(free), i32([len(free)]), i32(table)
    first = [x.clone() for x in bsa.bsattn_paged_plan(c, n, f, k, t, 16, sum(new))]
    t2, side = i32(table), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = bsa.bsattn_paged_plan(c, n, f, k, t2, 16, sum(new))
    with torch.cuda.stream(side):
        graph.replay()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out)) and torch.equal(t, t2)


# ------------------------------------------------------------------------- append and gather

def _special(T, H, d, dtype, seed):
    """Values with exact rounding ties, zeros, subnormals, tiny and huge groups."""
    x = _rand(T, H, d, dtype=dtype, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.0],
                        device="cuda")
    scale = torch.tensor([2.0 ** -9, 0.875 * 2.0 ** -6, 1.0, 1.125, 1.875, 240.0, 448.0], device="cuda")
    pick = scale[torch.randint(0, 7, (T, H, d // 16, 1), generator=g, device="cuda")]
    x[1::3] = (ties * pick).flatten(-2).to(dtype)[1::3]
    x[2::7] *= 2.0 ** -12
    x[0, 0, :16] = 0.0
    x[3, 0, :16] = -0.0
    x[4, 0, :16] = torch.finfo(dtype).smallest_normal
    x[5, 0, :16] = torch.finfo(dtype).max
    # scales on the border between two e4m3 values: amax = 6 * (1 + 1/16) and neighbours
    x[6, 0, :16] = 6.375
    x[6, -1, :16] = 6.0 * 1.1875
    return x


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("unit", [1.0, 0.25, 2.0 ** -16, 2.0 ** 16])
def test_append_is_the_exact_rounding(bsa, d, dtype, unit):
    T, H, page = 301, 3, 64
    k, v = _special(T, H, d, dtype, seed=d), _special(T, H, d, dtype, seed=d + 50)
    cache = bsa.bsattn_kv4_cache(8, H, page, d)
    for c in cache:
        c.fill_(0x5a)
    g = torch.Generator().manual_seed(0)
    slots = torch.randperm(8 * page, generator=g)[:T].cuda()
    slots[7] = -1
    bsa.bsattn_kv4_append(k, v, slots, cache, k_scale=unit, v_scale=1.0)
    wk, ws = ref.quantise(k, unit)
    xk, xs = ref.quantise(v, 1.0)
    on = slots >= 0
    at = slots[on] // page, slots[on] % page
    assert torch.equal(cache.k_scales[at[0], :, at[1]], ws[on])
    assert torch.equal(cache.k_codes[at[0], :, at[1]], wk[on])
    assert torch.equal(cache.v_scales[at[0], :, at[1]], xs[on])
    assert torch.equal(cache.v_codes[at[0], :, at[1]], xk[on])
    rest = torch.ones(8, page, dtype=torch.bool, device="cuda")
    rest[at] = False
    for c in cache:                                     # all other rows are left as they were
        assert (c.transpose(1, 2)[rest] == 0x5a).all()
    gk, gv = bsa.bsattn_kv4_gather(slots, cache, dtype, k_scale=unit, v_scale=1.0)
    want = ref.dequantise(wk, ws, unit).to(dtype)
    want[7] = 0
    assert torch.equal(gk, want)
    want = ref.dequantise(xk, xs, 1.0).to(dtype)
    want[7] = 0
    assert torch.equal(gv, want)


def test_append_every_bf16_and_fp16_value(bsa):
    """All finite 16-bit patterns, each in a group whose largest value sets another scale."""
    for dtype in (BF16, F16):
        bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(dtype)
        x = bits[torch.isfinite(bits.float())]
        g = torch.Generator(device="cuda").manual_seed(1)
        x = x[torch.randperm(x.numel(), generator=g, device="cuda")]
        near = x.float().abs().clamp(2.0 ** -10, 2.0 ** 11).log2().floor()
        x = torch.cat((x, x[near.argsort(stable=True)]))             # also in groups of like size
        x = x[:x.numel() // 128 * 128].view(-1, 1, 128)
        T = x.shape[0]
        cache = bsa.bsattn_kv4_cache(-(-T // 64), 1, 64, 128)
        slots = torch.arange(T, device="cuda")
        bsa.bsattn_kv4_append(x, x.flip(0).contiguous(), slots, cache)
        codes, scales = ref.quantise(x, 1.0)
        assert torch.equal(cache.k_codes.view(-1, 64)[:T], codes[:, 0])
        assert torch.equal(cache.k_scales.view(-1, 8)[:T], scales[:, 0])


def test_append_keeps_infinities_and_nan_visible(bsa):
    x = _rand(4, 2, 64, dtype=BF16, seed=1)
    x[1, 0, 3], x[2, 1, 40] = float("inf"), float("nan")
    cache = bsa.bsattn_kv4_cache(1, 2, 64, 64)
    slots = torch.tensor([5, 0, 63, 9], device="cuda")
    bsa.bsattn_kv4_append(x, x, slots, cache)
    k, v = bsa.bsattn_kv4_gather(slots, cache, BF16)
    bad = torch.zeros_like(k, dtype=torch.bool)
    bad[1, 0, :16] = bad[2, 1, 32:48] = True
    assert torch.equal(k.isnan(), bad) and torch.equal(v.isnan(), bad)


def test_append_strided_rows_and_bad_slots(bsa):
    T, H, d, page = 70, 4, 128, 64
    fused = _rand(T, (8 + 2 * H) * d, dtype=F16, seed=3)
    k = fused[:, 8 * d:(8 + H) * d].unflatten(1, (H, d))
    v = fused[:, (8 + H) * d:].unflatten(1, (H, d))
    cache, ws = bsa.bsattn_kv4_cache(3, H, page, d), torch.zeros(256, dtype=torch.uint8, device="cuda")
    slots = torch.arange(T, device="cuda") * 2
    slots[3], slots[4] = 3 * page, 2 ** 40              # past the cache: skipped and reported
    bsa.bsattn_kv4_append(k, v, slots, cache, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
    gk, gv = bsa.bsattn_kv4_gather(slots, cache, BF16, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
    for got, x in ((gk, k), (gv, v)):
        want = ref.dequantise(*ref.quantise(x, 1.0), 1.0).to(BF16)
        want[3] = want[4] = 0
        assert torch.equal(got, want)
    bsa.bsattn_kv4_append(k[:0], v[:0], slots[:0], cache)
    assert bsa.bsattn_kv4_gather(slots[:0], cache, F16)[0].shape == (0, H, d)
    with pytest.raises(bsa.BsattnError):
        bsa.bsattn_kv4_append(k, v, slots, cache, k_scale=0.3)
    with pytest.raises(TypeError):
        bsa.bsattn_kv4_append(k, v, slots.int(), cache)
    with pytest.raises(ValueError):
        bsa.bsattn_kv4_append(k[..., ::2], v[..., ::2], slots, bsa.bsattn_kv4_cache(3, H, page, 64))


# ------------------------------------------------------------------------- decode

class _Rows4:
    def __init__(self, cache, table, k_unit, v_unit):
        self.c, self.table, self.units, self.groups = cache, table, (k_unit, v_unit), cache.k_codes.shape[1]

    def __call__(self, b, g, n):
        page = self.c.k_codes.shape[2]
        j = torch.arange(n, device="cuda")
        at = self.table[b].long()[j // page], g, j % page
        return (ref.dequantise(self.c.k_codes[at], self.c.k_scales[at], self.units[0]),
                ref.dequantise(self.c.v_codes[at], self.c.v_scales[at], self.units[1]))


def _cache4(lens, Hkv, d, page, seed):
    """A cache of random rows on shuffled pages; rows past each length hold scales that mean NaN."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    total = sum(need) + 2
    perm = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    k4, ks = ref.quantise(_rand(total, Hkv, page, d, dtype=BF16, seed=seed), 1.0)
    v4, vs = ref.quantise(_rand(total, Hkv, page, d, dtype=BF16, seed=seed + 1), 0.5)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        if n and lens[b] % page:
            last = int(perm[at + n - 1])
            ks[last, :, lens[b] % page:] = 0x7f
            vs[last, :, lens[b] % page:] = 0xff
        at += n
    return (k4, ks, v4, vs), table.cuda()


def _decode4(bsa, lens, Hq, Hkv, d, dtype, page, seed, window=0, sinks=0, chosen=None, q_scale=1.0):
    cache, table = _cache4(lens, Hkv, d, page, seed)
    cache = bsa.Kv4Cache(*cache)
    q = _rand(len(lens), Hq, d, dtype=dtype, seed=seed + 7, scale=q_scale)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.zeros(bsa.bsattn_decode_kv4_workspace_size(Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    got = bsa.bsattn_decode_paged_kv4(q, cache, n, table, chosen, window=window, sinks=sinks, k_scale=1.0,
                                      v_scale=0.5, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == 0

    def visible(b, g, m):
        if chosen is not None:
            on = torch.zeros(m + 64, dtype=torch.bool, device="cuda")
            for t in chosen[b, g].tolist():
                if t >= 0:
                    on[64 * t:64 * t + 64] = True
            return on[:m]
        return ref.windowed(m, window, sinks, "cuda") if window else torch.ones(m, dtype=torch.bool, device="cuda")

    # weights are rounded to fp16 there whatever the queries' type; queries are scaled into fp16 exactly
    ref.check(got, *ref.decode(q, _Rows4(cache, table, 1.0, 0.5), lens, visible, F16))
    return got, (q, cache, n, table)


LENS = [0, 1, 31, 32, 33, 63, 64, 65, 100, 1000, 333, 2049]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (32, 1), (100, 33), (64, 200), (5000, 7)])
def test_decode_lengths_and_windows(bsa, d, dtype, window, sinks):
    got, _ = _decode4(bsa, LENS, 8, 2, d, dtype, 64, seed=d + window, window=window, sinks=sinks)
    assert got[0].abs().max() == 0


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (4, 4), (6, 2), (14, 2), (40, 5), (32, 8)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [64, 192])
def test_decode_heads(bsa, Hq, Hkv, d, page):
    _decode4(bsa, [700, 64, 1301], Hq, Hkv, d, BF16, page, seed=Hq + d)


@pytest.mark.parametrize("scale", [1e-3, 30.0, 1e-30, 1e30])
def test_decode_query_sizes(bsa, scale):
    """Queries far outside fp16's range are brought into it by a power of two."""
    if scale == 1e30:                                   # scores past any exponent: one key takes all
        cache, table = _cache4([5], 1, 64, 64, seed=1)
        q = torch.full((1, 2, 64), scale, dtype=BF16, device="cuda")
        n = torch.tensor([1], dtype=torch.int32, device="cuda")
        got = bsa.bsattn_decode_paged_kv4(q, cache, n, table, v_scale=0.5)
        _, v = _Rows4(bsa.Kv4Cache(*cache), table, 1.0, 0.5)(0, 0, 1)
        assert torch.equal(got[0, 0], v[0].to(BF16))
        return
    _decode4(bsa, [500, 77], 8, 2, 128, BF16, 64, seed=3, q_scale=scale)


def test_decode_long_and_ragged(bsa):
    lens = [30000, 3, 12345, 64, 1, 20001, 700, 0, 129]
    got, (q, cache, n, table) = _decode4(bsa, lens, 10, 2, 64, BF16, 64, seed=5)
    for _ in range(5):
        assert torch.equal(got, bsa.bsattn_decode_paged_kv4(q, cache, n, table, k_scale=1.0, v_scale=0.5))


def test_decode_one_long_sequence(bsa):
    _decode4(bsa, [50001], 8, 1, 128, F16, 128, seed=6)
    _decode4(bsa, [50001], 32, 8, 128, BF16, 64, seed=7)


def test_decode_many_sequences(bsa):
    g = torch.Generator().manual_seed(1)
    _decode4(bsa, torch.randint(0, 200, (700,), generator=g).tolist(), 4, 2, 64, F16, 64, seed=8)


@pytest.mark.parametrize("B", [2, 20, 56, 57, 58, 127, 128, 129])
def test_decode_batches_about_the_number_of_parts(bsa, B):
    """Sequences cut for themselves (few of them, or long parts) and end to end, with empty ones among them."""
    for n, d in ((70, 64), (900, 128)):
        lens = [0 if b % 7 == 3 else n + 53 * (b % 5) for b in range(B)]
        got, _ = _decode4(bsa, lens, 8, 8, d, BF16, 64, seed=B + n)
        assert all(got[b].abs().max() == 0 for b in range(B) if lens[b] == 0)
    _decode4(bsa, [0] * B, 8, 8, 64, F16, 64, seed=B)


def test_decode_chosen_blocks(bsa):
    lens = [1000, 64, 0, 3333]
    g = torch.Generator().manual_seed(4)
    for slots in (1, 7, 40):
        idx = torch.full((4, 3, slots), -1, dtype=torch.int32)
        for b, m in enumerate(lens):
            for h in range(3):
                take = min(slots, -(-m // 64))
                idx[b, h, torch.randperm(slots, generator=g)[:take]] = \
                    torch.randperm(-(-m // 64), generator=g)[:take].to(torch.int32)
        idx[0, 1] = -1                                  # nothing chosen: 0
        got, _ = _decode4(bsa, lens, 12, 3, 128, BF16, 64, seed=slots, chosen=idx.cuda())
        assert got[0, 4:8].abs().max() == 0 and got[2].abs().max() == 0


def test_decode_chosen_past_the_end_is_flagged(bsa):
    cache, table = _cache4([130, 130], 1, 64, 64, seed=1)
    q = _rand(2, 2, 64, dtype=F16, seed=2)
    n = torch.tensor([130, 130], dtype=torch.int32, device="cuda")
    ws = torch.zeros(bsa.bsattn_decode_kv4_workspace_size(2, 1, 64), dtype=torch.uint8, device="cuda")
    idx = torch.tensor([[[0, 2]], [[0, 3]]], dtype=torch.int32, device="cuda")
    got = bsa.bsattn_decode_paged_kv4(q, cache, n, table, idx, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
    idx[1, 0, 1] = -1
    assert torch.equal(got, bsa.bsattn_decode_paged_kv4(q, cache, n, table, idx, ws=ws))
    table[0, 1] = 99                                    # an unmapped page
    got = bsa.bsattn_decode_paged_kv4(q, cache, n, table, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX and torch.isfinite(got.float()).all()


def test_decode_shows_nan_tokens(bsa):
    """A token that was not finite when it was appended is seen by those who attend to it, by no one else."""
    cache, table = _cache4([300, 300], 2, 128, 64, seed=2)
    q = _rand(2, 4, 128, dtype=BF16, seed=3)
    n = torch.tensor([300, 300], dtype=torch.int32, device="cuda")
    cache[1][table[1, 1].long(), 0, 9, 2] = 0x7f
    got = bsa.bsattn_decode_paged_kv4(q, cache, n, table)
    assert got[1, :2].isnan().all() and got.isnan().sum() == 256
    got = bsa.bsattn_decode_paged_kv4(q, cache, n, table, window=100, sinks=70)
    assert torch.isfinite(got.float()).all()


def test_decode_streams_and_graphs(bsa):
    calls, want = [], []
    for i, (lens, hq, hkv) in enumerate([([5000, 700], 8, 2), ([90] * 40, 6, 3), ([9000], 8, 1), ([300, 0], 16, 4)]):
        got, c = _decode4(bsa, lens, hq, hkv, 128, BF16, 64, seed=30 + i)
        calls.append(c)
        want.append(got)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for r in range(6):
        for i, c in enumerate(calls):
            with torch.cuda.stream(streams[(i + r) % 4]):
                got.append((i, bsa.bsattn_decode_paged_kv4(*c, k_scale=1.0, v_scale=0.5)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in got)
    graphs, outs = [], []
    for i in (0, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(bsa.bsattn_decode_paged_kv4(*calls[i], k_scale=1.0, v_scale=0.5))
        graphs.append(g)
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[2])


class _Held:
    def __init__(self, k, v):
        self.k, self.v, self.groups = k, v, k[0].shape[1]

    def __call__(self, b, g, n):
        return self.k[b][:, g], self.v[b][:, g]


def test_serving_loop(bsa):
    """Plan, append, decode, step after step, as a server runs them: prompts of several lengths, then one
    token at a time, pages handed out as sequences grow."""
    B, Hq, Hkv, d, page, most = 5, 8, 2, 64, 64, 12
    lens = [0, 0, 0, 0, 0]
    cache = bsa.bsattn_kv4_cache(40, Hkv, page, d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, free = torch.full((B, most), -1, dtype=torch.int32, device="cuda"), i32(list(range(40)))
    count, cached = i32([40]), i32(lens)
    held_k = [torch.zeros(0, Hkv, d, dtype=torch.float64, device="cuda") for _ in range(B)]
    held_v = [torch.zeros(0, Hkv, d, dtype=torch.float64, device="cuda") for _ in range(B)]
    for step, new in enumerate([[200, 1, 64, 63, 0], [1, 1, 1, 1, 130], [1] * 5, [1] * 5, [100, 0, 64, 1, 1]]):
        cap = 400
        slots, starts, seqlens, left = bsa.bsattn_paged_plan(cached, i32(new), free, count, table, page, cap)
        k, v = _rand(cap, Hkv, d, dtype=BF16, seed=step), _rand(cap, Hkv, d, dtype=BF16, seed=step + 100)
        bsa.bsattn_kv4_append(k, v, slots, cache, k_scale=0.5, v_scale=0.25)
        at = 0
        for b, m in enumerate(new):
            held_k[b] = torch.cat((held_k[b], ref.dequantise(*ref.quantise(k[at:at + m], 0.5), 0.5)))
            held_v[b] = torch.cat((held_v[b], ref.dequantise(*ref.quantise(v[at:at + m], 0.25), 0.25)))
            at += m
            lens[b] += m
        assert seqlens.tolist() == lens and starts.tolist()[-1] == sum(new)
        cached, count = seqlens, left
        q = _rand(B, Hq, d, dtype=BF16, seed=step + 200)
        for window, sinks in ((0, 0), (50, 3)):
            got = bsa.bsattn_decode_paged_kv4(q, cache, seqlens, table, window=window, sinks=sinks, k_scale=0.5,
                                              v_scale=0.25)
            on = lambda b, g, n: ref.windowed(n, window or n, sinks, "cuda")  # noqa: E731,B023
            ref.check(got, *ref.decode(q, _Held(held_k, held_v), lens, on, F16))
    # a cached prefix read back for a prefill over it
    j = torch.arange(lens[0], device="cuda")
    rows = table[0].long()[j // page] * page + j % page
    pk, pv = bsa.bsattn_kv4_gather(rows, cache, BF16, k_scale=0.5, v_scale=0.25)
    assert torch.equal(pk.double(), held_k[0]) and torch.equal(pv.double(), held_v[0])
    q = _rand(1, Hq, 40, d, dtype=BF16, seed=1)
    kk, vv = pk.transpose(0, 1)[None], pv.transpose(0, 1)[None]
    ref.check(bsa.bsattn_prefill_window(q, kk, vv, 90, 4), *ref.window_prefill(q, kk, vv, 90, 4))


def test_cache_rows_past_32_bit_offsets(bsa):
    """Pages whose codes lie past 2^32 bytes: append, gather and decode at the cache's far end."""
    Hkv, d, page = 8, 128, 64
    pages = (1 << 32) // (Hkv * page * d // 2) + 4
    codes = [torch.empty(pages, Hkv, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(pages, Hkv, page, d // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = bsa.Kv4Cache(codes[0], scales[0], codes[1], scales[1])
    table = torch.tensor([[pages - 1, 1, pages - 2]], dtype=torch.int32, device="cuda")
    j = torch.arange(150, device="cuda")
    slots = table[0].long()[j // page] * page + j % page
    k, v = _rand(150, Hkv, d, dtype=BF16, seed=1), _rand(150, Hkv, d, dtype=BF16, seed=2)
    bsa.bsattn_kv4_append(k, v, slots, cache)
    gk, gv = bsa.bsattn_kv4_gather(slots, cache, BF16)
    assert torch.equal(gk.double(), ref.dequantise(*ref.quantise(k, 1.0), 1.0))
    q = _rand(1, 16, d, dtype=BF16, seed=3)
    n = torch.tensor([150], dtype=torch.int32, device="cuda")
    got = bsa.bsattn_decode_paged_kv4(q, cache, n, table)
    ref.check(got, *ref.decode(q, _Held([gk.double()], [gv.double()]), [150], lambda b, g, m: ref.windowed(m, m, 0, "cuda"), F16))


def test_sizes_that_do_not_fit_are_refused(bsa):
    cache, table = _cache4([70], 2, 64, 64, seed=1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        bsa.bsattn_paged_plan(i32([0]), i32([1]), i32([3]), i32([1]), table, 2 ** 32 + 64, 8)
    with pytest.raises(bsa.BsattnError):
        bsa.bsattn_paged_plan(i32([0]), i32([1]), i32([3]), i32([1]), table, 64, -1)
    with pytest.raises(TypeError):
        bsa.bsattn_kv4_gather(torch.zeros(1, dtype=torch.int64, device="cuda"), cache, torch.float32)
    q = _rand(1, 4, 64, dtype=F16, seed=2)
    for bad in (dict(block_indices=i32([[[0], [0]]]), window=3), dict(k_scale=0.7)):
        with pytest.raises(bsa.BsattnError):
            bsa.bsattn_decode_paged_kv4(q, cache, i32([70]), table, **bad)
    for bad in (dict(block_indices=i32([[[0]]])), dict(block_indices=torch.zeros(1, 2, 0, dtype=torch.int32, device="cuda")),
                dict(out=q[:, :2])):
        with pytest.raises(ValueError):
            bsa.bsattn_decode_paged_kv4(q, cache, i32([70]), table, **bad)
    with pytest.raises(ValueError):
        bsa.bsattn_decode_paged_kv4(q, cache[:2] + (cache[3], cache[2]), i32([70]), table)
    want = bsa.bsattn_decode_paged_kv4(q, cache, i32([70]), table)
    assert torch.equal(want, bsa.bsattn_decode_paged_kv4(q, cache, i32([70]), table, window=2 ** 40, sinks=2 ** 33))
