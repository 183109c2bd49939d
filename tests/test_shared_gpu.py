"""Decoding over a shared prefix, against its 64-bit statement."""
import math

import pytest
import torch

import selection_reference as ref
import serving_reference as serving

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F16, BF16 = torch.float16, torch.bfloat16
BUDGET = 2_000_000_000                     # the default


@pytest.fixture(scope="module")
def bsa():
    import block_sparse_attention_gb300 as m
    m.load()
    return m


def _rand(*shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Inputs over shuffled pages; rows past each length are NaN."""

    def __init__(self, sizes, plens, lens, Hq, Hkv, d, dtype, page=64, seed=0, scale=1.0):
        assert sum(sizes) == len(lens) and len(sizes) == len(plens)
        need = [-(-n // page) for n in (*plens, *lens)]
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.k, self.v = (_rand(pages, page, Hkv, d, dtype=dtype, seed=seed + s, scale=1.0) for s in (1, 2))
        tables = []
        for n, m in zip((*plens, *lens), need):
            mine = [perm.pop() for _ in range(m)]
            if n % page:
                self.k[mine[-1], n % page:] = float("nan")
                self.v[mine[-1], n % page:] = float("nan")
            tables.append(mine)
        for p in perm:
            self.k[p] = float("nan")
            self.v[p] = float("nan")
        P = len(sizes)

        def table(rows):
            most = max(1, max(map(len, rows)))
            return _i32([r + [-1] * (most - len(r)) for r in rows]).view(len(rows), most)
        self.ptable, self.table = table(tables[:P]), table(tables[P:])
        self.plens, self.lens = _i32(plens), _i32(lens)
        self.starts = _i32([sum(sizes[:p]) for p in range(P + 1)])
        self.q = _rand(len(lens), Hq, d, dtype=dtype, seed=seed + 3, scale=scale)

    def call(self, bsa, **kw):
        return bsa.bsattn_decode_shared(self.q, self.k, self.v, self.plens, self.ptable, self.starts, self.lens, self.table, **kw)

    def want(self):
        return ref.shared(self.q, self.k, self.v, self.plens, self.ptable, self.starts, self.lens, self.table)

    def check(self, bsa, **kw):
        got = self.call(bsa, **kw)
        serving.check(got, *self.want())
        return got


@pytest.mark.parametrize("plen", [1, 63, 64, 65, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("B", [1, 5, 40, 70])
def test_lengths(bsa, plen, B):
    """One prefix; B = 40 and more fill both query tiles (32 sequences of four heads each)."""
    lens = [(7 * b) % 150 for b in range(B)]
    Case([B], [plen], lens, 8, 2, 128, BF16, seed=plen + B).check(bsa)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (3, 1), (10, 2), (6, 1), (14, 2), (8, 1), (17, 17)])
@pytest.mark.parametrize("d,dtype", [(64, F16), (64, BF16), (128, F16), (128, BF16)])
def test_heads_and_types(bsa, Hq, Hkv, d, dtype):
    for B in (6, 150):
        Case([B], [700], [b % 90 for b in range(B)], Hq, Hkv, d, dtype, page=128, seed=Hq + B).check(bsa)


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
def test_groups(bsa, d, dtype):
    """Prefixes of any lengths, some of nothing, groups of one and of many, and empty ones."""
    sizes, plens = [3, 1, 0, 70, 2, 0, 9], [500, 0, 130, 1100, 64, 77, 1]
    lens = [(31 * b) % 200 * (b % 3 > 0) for b in range(sum(sizes))]
    Case(sizes, plens, lens, 8, 4, d, dtype, seed=1).check(bsa)
    Case([1] * 30, [64 * b for b in range(30)], [b for b in range(30)], 4, 4, d, dtype, seed=2).check(bsa)
    Case([90, 120], [333, 900], [5] * 210, 8, 4, d, dtype, seed=3).check(bsa)


@pytest.mark.parametrize("B", [33, 65, 257, 290])
def test_one_prefix_read_several_times(bsa, B):
    """32 sequences of eight heads a reading: two at a time and more, and of nine and ten some CTAs have one less."""
    lens = [(11 * b) % 70 for b in range(B)]
    Case([B], [2000], lens, 16, 2, 64, BF16, seed=B).check(bsa)
    Case([B], [130], [0] * B, 16, 2, 128, F16, seed=B + 1).check(bsa)


@pytest.mark.parametrize("Hkv", [75, 76, 77, 160, 700])
def test_many_kv_heads(bsa, Hkv):
    """As many as half the SMs and more."""
    Case([5], [300], [0, 3, 64, 65, 200], Hkv, Hkv, 64, F16, seed=Hkv).check(bsa)
    Case([2, 3], [0, 200], [0, 3, 64, 65, 200], Hkv, Hkv, 64, BF16, seed=Hkv).check(bsa)


@pytest.mark.parametrize("plen,own", [(5000, 1), (1, 3000), (40_000, 0), (0, 6000)])
def test_shares_of_the_gpu(bsa, plen, own):
    """Prefixes and own tokens that cost very different amounts, or nothing."""
    for B in (3, 100):
        Case([B], [plen], [own if b % 3 == 0 else 0 for b in range(B)], 8, 2, 128, BF16, seed=B).check(bsa)


def test_many_pieces_a_cta(bsa):
    """More items than CTAs, and items of many CTAs: barriers, rings and accumulators are used again and again."""
    Case([2] * 100, [200 + 3 * p for p in range(100)], [1] * 200, 16, 8, 64, F16, seed=1).check(bsa)
    Case([300], [900], [3] * 300, 32, 4, 64, BF16, seed=2).check(bsa)
    Case([2], [60_001], [10, 0], 8, 1, 128, BF16, page=256, seed=3).check(bsa)
    Case([70], [20_077], [10] * 70, 8, 2, 128, F16, page=64, seed=4).check(bsa)


def test_more_prefixes_than_threads(bsa):
    sizes = [p % 3 for p in range(900)]
    Case(sizes, [(17 * p) % 140 for p in range(900)], [(5 * b) % 70 for b in range(sum(sizes))], 2, 1, 64, BF16, seed=5).check(bsa)


def test_nothing_to_see(bsa):
    got = Case([3, 2], [0, 100], [0, 5, 0, 0, 70], 8, 2, 128, BF16, seed=1).check(bsa)
    assert got[[0, 2]].abs().max() == 0
    assert Case([4], [0], [0] * 4, 8, 2, 64, F16, seed=2).call(bsa).abs().max() == 0
    c = Case([4], [100], [3] * 4, 8, 2, 64, F16, seed=2)
    c.q, c.lens, c.table, c.starts = c.q[:0], c.lens[:0], c.table[:0], _i32([0, 0])
    assert c.call(bsa).shape == (0, 8, 64)


def test_agrees_with_the_window_decode(bsa):
    """No prefix: each sequence's own tokens; a prefix of whole pages in front of them: as if each sequence had it
    for itself.  Both within the bound of the one statement."""
    c = Case([9, 11], [0, 0], [(77 * b) % 3000 for b in range(20)], 8, 2, 128, BF16, seed=3)
    c.check(bsa)
    serving.check(bsa.bsattn_decode_window_paged(c.q, c.k, c.v, c.lens, c.table, 1 << 20), *c.want())
    c = Case([5], [640], [100, 1, 64, 0, 300], 8, 2, 128, BF16, seed=4)
    joined = torch.cat((c.ptable.expand(5, -1), c.table), 1).contiguous()
    c.check(bsa)
    serving.check(bsa.bsattn_decode_window_paged(c.q, c.k, c.v, c.lens + 640, joined, 1 << 20), *c.want())


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("sizes", [[1], [30], [70], [129]])
def test_own_tokens_of_any_lengths(bsa, sizes, d, dtype):
    """Ragged own lengths, none among them, one sequence far longer than the others, with prefixes of few tokens and
    of many: every mix of steps."""
    B = sum(sizes)
    for plen, longest in ((0, 700), (64, 5000), (900, 64), (3001, 3003)):
        lens = [(longest * (b * b + 3) // 7) % 200 * (b % 4 != 1) for b in range(B)]
        lens[B // 2] = longest
        Case(sizes, [plen], lens, 8, 2, d, dtype, page=128, seed=plen + B).check(bsa)


def test_more_row_tiles_than_a_part_keeps(bsa):
    """One long prefix and hundreds of groups of one or two sequences: parts that go through many row tiles."""
    sizes = [3] + [1 + p % 2 for p in range(500)]
    B = sum(sizes)
    Case(sizes, [30_000] + [p % 2 for p in range(500)], [5 * (b % 2) for b in range(B)], 2, 1, 64, BF16, seed=6).check(bsa)


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("B", [6, 70])
def test_large_scores(bsa, B, d, dtype):
    """Scores that keep growing along the prefix: the reference maximum moves and O is rescaled."""
    c = Case([B], [1500], [40] * B, 8, 2, d, dtype, seed=5, scale=2.0)
    for j, page in enumerate(c.ptable[0].tolist()):
        c.k[page] = (c.k[page].float() * (0.05 + 0.12 * j)).to(dtype)
    c.check(bsa)


def test_nan_reaches_those_that_see_it(bsa):
    c = Case([3, 40], [400, 500], [50] * 43, 8, 2, 64, F16, seed=6)
    clean = c.call(bsa)
    c.k[c.ptable[0, 2], 7, 1] = float("nan")                   # head 1 of group 0
    got = c.call(bsa)
    lost = got.isnan().all(-1)
    want = torch.zeros_like(lost)
    want[:3, 4:] = True
    assert torch.equal(lost, want) and torch.equal(got[~lost], clean[~lost])
    # in one channel of one sequence's head 0: its rows alone, whoever is worked on with it
    for at in (2, 20):
        for bad in (float("inf"), float("nan"), -float("inf")):
            c = Case([3, 40], [400, 500], [50] * 43, 8, 2, 64, F16, seed=6)
            clean = c.call(bsa)
            c.v[c.table[at, 0], 3, 0, 9] = bad
            got = c.call(bsa)
            off = ~torch.isfinite(got)
            assert off[at, :4, 9].all() and off.sum() == 4 and torch.equal(got[~off], clean[~off])
    # in the prefix: all rows of the group's head
    c = Case([3, 40], [400, 500], [50] * 43, 8, 2, 128, BF16, seed=7)
    out, bound = c.want()
    c.v[c.ptable[1, 1], 3, 1, 100] = float("inf")
    got = c.call(bsa)
    assert not torch.isfinite(got[3:, 4:, 100]).any()
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[3:, 4:] = False
    serving.check(got[rest], out[rest], bound[rest])


def test_nan_beside_bad_pages(bsa):
    c = Case([40], [500], [150] * 40, 8, 2, 128, BF16, page=64, seed=8)
    c.ptable[0, 2] = -1
    c.table[7, 1] = c.k.shape[0]
    c.table[9, 0] = 2 ** 31 - 1
    out, bound = c.want()
    c.v[c.table[20, 0], 3] = float("nan")
    got = c.call(bsa)
    rest = torch.arange(40, device="cuda") != 20
    serving.check(got[rest], out[rest], bound[rest])
    assert got[20].isnan().all()


@pytest.mark.parametrize("B", [5, 70])
def test_bad_pages_and_lengths(bsa, B):
    """Tokens on pages out of range are left out, and reported; so are lengths past a table or below 0."""
    c = Case([B - 2, 2], [1000, 300], [200] * B, 8, 2, 128, BF16, seed=7)
    ws = torch.zeros(bsa.bsattn_decode_shared_workspace_size(B, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    c.check(bsa, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == 0
    for page in (-1, c.k.shape[0], 2 ** 31 - 1):
        c.ptable[0, 3], c.ptable[0, 10], c.ptable[0, 11] = page, page, page      # half a tile, and a whole one
        c.ptable[1, 4] = page                                                # the last page
        c.table[1, 1] = page
        c.check(bsa, ws=ws)
        assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
    want = c.call(bsa)
    c.plens[1] = 10 ** 6
    c.table[B - 1, 3] = c.table[B - 1, 2]
    got = c.call(bsa, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
    assert torch.equal(got[:B - 2].isnan(), want[:B - 2].isnan())
    c.plens[1] = -4
    c.lens[0] = -2 ** 31
    got = c.call(bsa, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
    c.plens[1] = c.lens[0] = 0
    serving.check(got, *c.want())


def test_bad_groups(bsa):
    """Groups that do not rise from 0 to B are reported; sequences outside all of them have no prefix."""
    c = Case([2, 3], [300, 200], [40] * 5, 8, 2, 64, BF16, seed=8)
    ws = torch.zeros(bsa.bsattn_decode_shared_workspace_size(5, 2, 8, 2, 64), dtype=torch.uint8, device="cuda")
    whole, plens = c.call(bsa, ws=ws), c.plens
    c.plens = torch.zeros_like(plens)
    own = c.check(bsa, ws=ws)
    c.plens = plens
    assert bsa.bsattn_get_device_status(ws) == 0
    for starts, outside in (([1, 2, 5], [0]), ([0, 2, 4], [4]), ([0, 2, 2], [2, 3, 4]), ([5, 5, 5], range(5))):
        c.starts = _i32(starts)
        got = c.call(bsa, ws=ws)
        assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
        for b in range(5):
            if b in outside:
                assert torch.equal(got[b], own[b])
    for starts in ([0, 9, 5], [-7, 2, 5], [0, 4, 2], [3, -2 ** 31, 2 ** 31 - 1], [2 ** 31 - 1, 0, -1]):
        c.starts = _i32(starts)
        c.call(bsa, ws=ws)
        assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
    c.starts = _i32([0, 2, 5])
    assert torch.equal(c.call(bsa, ws=ws), whole)


@pytest.mark.parametrize("B,plen,lens", [(70, 9000, 40), (4, 5000, 700), (40, 300, 9)])
def test_expired_waits(bsa, B, plen, lens):
    """Rows are right or NaN in every channel whatever the budget, and the workspace serves the next call."""
    c = Case([B], [plen], [lens] * B, 8, 2, 128, BF16, seed=9)
    ws = torch.zeros(bsa.bsattn_decode_shared_workspace_size(B, 1, 8, 2, 128), dtype=torch.uint8, device="cuda")
    want, seen = c.call(bsa), 0
    try:
        for budget in (0, 200, 1000, 5000, 20000, 100000):
            bsa.bsattn_set_wait_budget_ns(budget)
            for _ in range(3):
                got = c.call(bsa, ws=ws)
                status = bsa.bsattn_get_device_status(ws)
                seen |= status
                assert status in (0, bsa.BSATTN_ERR_TIMEOUT)
                lost = got.isnan().all(-1)
                assert torch.equal(got[~lost], want[~lost])
                assert status or not lost.any()
    finally:
        bsa.bsattn_set_wait_budget_ns(BUDGET)
    # (a first poll may itself last until the data is there: short calls may find nothing expired)
    assert seen or B < 70
    assert torch.equal(c.call(bsa, ws=ws), want) and torch.equal(c.call(bsa), want)
    assert bsa.bsattn_get_device_status(ws) == 0


def test_one_workspace_for_all_shapes(bsa):
    ws = torch.zeros(bsa.bsattn_decode_shared_workspace_size(300, 9, 32, 8, 128), dtype=torch.uint8, device="cuda")
    for seed, (B, plen, d) in enumerate([(70, 900, 128), (3, 2000, 64), (130, 64, 64), (5, 1, 128), (64, 5000, 128)]):
        Case([B], [plen], [9 * b % 130 for b in range(B)], 16, 4, d, BF16, seed=seed).check(bsa, ws=ws)
    ws[256:] = 0xff
    Case([6, 80], [100, 900], [3] * 86, 16, 4, 64, F16, seed=9).check(bsa, ws=ws)


def test_results_do_not_depend_on_the_order(bsa):
    c = Case([64, 6], [7000, 333], [(50 * b) % 900 for b in range(70)], 32, 8, 128, BF16, seed=10)
    want = c.call(bsa)
    for _ in range(20):
        assert torch.equal(c.call(bsa), want)


def test_output_over_the_queries(bsa):
    for B in (4, 80):
        c = Case([B], [900], [60] * B, 8, 2, 128, BF16, seed=11)
        want = c.call(bsa)
        got = c.call(bsa, out=c.q)
        assert got.data_ptr() == c.q.data_ptr() and torch.equal(got, want)
    with pytest.raises(bsa.BsattnError):
        c.call(bsa, out=c.k.view(-1)[:c.q.numel()].view_as(c.q))


def test_streams_and_graphs(bsa):
    cases = [Case([B], [plen], [40] * B, 8, 2, 64, BF16, seed=plen) for B, plen in ((70, 3000), (4, 900))]
    want = [c.call(bsa) for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(cases[i].call(bsa))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)
    # two graphs that are replayed side by side, each with calls one after the other
    graphs, outs = [torch.cuda.CUDAGraph() for _ in cases], []
    for c, graph in zip(cases, graphs):
        with torch.cuda.graph(graph):
            outs.append([c.call(bsa) for _ in range(3)])
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)
    # what a captured call finds is in the device's word
    cases[1].ptable[0, 1] = -1
    torch.cuda.synchronize()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert bsa.bsattn_get_device_status(bsa.status_workspace("cuda")) == bsa.BSATTN_ERR_BAD_INDEX
    assert not torch.equal(outs[1][0], want[1])


def test_far_pages(bsa):
    """A cache whose rows lie past 32-bit offsets."""
    pages, hkv, d = (1 << 32) // (64 * 8 * 128) + 40, 8, 128
    k = torch.zeros(pages, 64, hkv, d, dtype=F16, device="cuda")
    v = torch.zeros_like(k)
    at = list(range(pages - 20, pages))
    k[pages - 20:], v[pages - 20:] = (_rand(20, 64, hkv, d, dtype=F16, seed=s) for s in (1, 2))
    small = Case([3], [10 * 64], [200, 30, 64], 32, hkv, d, F16, seed=3)
    small.k, small.v = k, v
    small.ptable = _i32([at[:10]])
    small.table = _i32([at[10:14], at[14:15] + [-1] * 3, at[15:16] + [-1] * 3])
    small.check(bsa)


@pytest.mark.parametrize("at", [0, 13_000, 19_999])
@pytest.mark.parametrize("B,group", [(1, 1), (20, 8)])
def test_small_weights_of_a_long_prefix(bsa, B, group, at):
    """One key that has all but a little of the weight and a value of 0, and thousands with 2^-24 to 2^-30 of it each,
    which are all that there is of the result: fp16 weights have to keep them.  80 kv heads: a CTA has some ten
    thousand keys of a head, with the large weight among them.  The largest weight of a row is 2^7 or more."""
    n, hkv, d = 20_000, 80, 64
    c = Case([B], [n], [0] * B, hkv * group, hkv, d, F16, page=64, seed=at)
    j = torch.arange(n, device="cuda")
    where = c.ptable[0].long()[j // 64], j % 64
    g = torch.Generator(device="cuda").manual_seed(at + 1)
    score = -math.log(2.0) * (24 + 6 * torch.rand(n, hkv, generator=g, device="cuda"))
    score[at] = 0
    k, v = torch.zeros(n, hkv, d, device="cuda"), 0.5 + torch.rand(n, hkv, d, generator=g, device="cuda")
    k[..., 0], v[at] = score, 0
    c.k[where], c.v[where] = k.to(F16), v.to(F16)
    c.q.zero_()
    c.q[..., 0] = math.sqrt(d)
    got = c.call(bsa).view(B, hkv, group, d)
    on = torch.ones(1, n, dtype=torch.bool, device="cuda")
    for h in range(hkv):
        out, bound = serving.attend(c.q[0, :1], c.k[where][:, h], c.v[where][:, h], on, F16, F16, 2.0 ** 7)
        assert out.min() > 30 * bound.max()
        serving.check(got[:, h], out, bound)


@pytest.mark.parametrize("B", [3, 70])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_weights_above_the_reference(bsa, B, dtype):
    """Scores just under 2^8 times the first tiles' ones: as much as the reference maximum may lag behind."""
    c = Case([B], [3000], [20] * B, 8, 2, 64, dtype, seed=1)
    c.q.zero_()
    c.q[..., 0] = 8
    for i, page in enumerate(c.ptable[0].tolist()):
        c.k[page, :, :, 0] = 0.0 if i < 4 else 5.53125             # 2^7.98
    c.check(bsa)


@pytest.mark.parametrize("B", [3, 70])
def test_scores_of_which_the_rounding_shows(bsa, B):
    """fp16 scores of some 2^26 in base 2, which 32 bits have to the nearest 8, with maxima that move on by 6: no weight
    passes the largest fp16 number."""
    c = Case([B], [3000], [0] * B, 8, 2, 64, F16, seed=1)
    c.q.zero_()
    c.q[..., 0], c.q[..., 1] = 16384, 1
    c.k[..., 0] = 22_704
    for i, page in enumerate(c.ptable[0].tolist()):
        c.k[page, :, :, 1] = 0 if i < 4 else 32 if i < 20 else 64
    got = c.call(bsa)
    top = c.v[c.ptable[0].long()].nan_to_num(0.0).abs().amax((0, 1)).repeat_interleave(4, 0)[None]
    # a mean of values: weights of one row add up to 1, up to the rounding of each
    assert torch.isfinite(got).all() and (got.abs() <= top * (1 + 2.0 ** -9)).all()


@pytest.mark.parametrize("sizes,plens", [([150, 150], [900, 1300]), ([70, 300, 40], [2000, 129, 640]), ([257, 256], [64, 3001])])
@pytest.mark.parametrize("d,dtype,group", [(64, F16, 4), (128, BF16, 4), (128, F16, 8)])
def test_several_large_groups(bsa, sizes, plens, d, dtype, group):
    """Groups of more than 256 rows a kv head each, several items a group."""
    lens = [(13 * b) % 90 for b in range(sum(sizes))]
    Case(sizes, plens, lens, 2 * group, 2, d, dtype, seed=sizes[0]).check(bsa)


@pytest.mark.parametrize("B", [4, 70])
def test_lengths_past_the_tables(bsa, B):
    """What is past a table is left out, and the rest is as if the length ended with it."""
    c = Case([B - 2, 2], [1024, 1024], [192] * B, 8, 2, 128, BF16, seed=12)
    ws = torch.zeros(bsa.bsattn_decode_shared_workspace_size(B, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    whole, want = c.call(bsa, ws=ws), c.want()
    serving.check(whole, *want)
    assert bsa.bsattn_get_device_status(ws) == 0
    plens, lens = c.plens, c.lens
    for past in (1, 129, 2 ** 31 - 1 - 1024):
        for p in range(2):
            c.plens, c.lens = plens.clone(), lens
            c.plens[p] += past
            got = c.call(bsa, ws=ws)
            assert torch.equal(got, whole) and bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
        for b in (0, B - 1):
            c.plens, c.lens = plens, lens.clone()
            c.lens[b] += past
            got = c.call(bsa, ws=ws)
            assert torch.equal(got, whole) and bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX


@pytest.mark.parametrize("plen,own", [(3000, 0), (0, 700), (500, 300)])
@pytest.mark.parametrize("B", [3, 70])
def test_largest_scores_of_either_part(bsa, B, plen, own):
    """fp16 scores of 2^26 to 2^28 in base 2, which 32 bits have to the nearest 8 or 16: a mean of values all the same."""
    c = Case([B], [plen], [own] * B, 32, 8, 64, F16, seed=plen + B)
    c.q.zero_()
    c.q[..., 0], c.q[..., 1] = 16384, 1
    c.k[..., 0] = torch.tensor([30_000, 30_016, 30_032, 30_048, 44_000, 44_032, 60_000, 60_032], device="cuda").to(F16)
    c.k[..., 1] = (_rand(*c.k.shape[:2], dtype=F16, seed=3).abs() * 32).to(F16)[..., None]
    got = c.call(bsa)
    values = c.v.nan_to_num(0.0).abs().amax((0, 1)).repeat_interleave(4, 0)[None]
    assert torch.isfinite(got).all() and (got.abs() <= values * (1 + 2.0 ** -9)).all()
