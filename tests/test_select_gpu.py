"""Block summaries, the blocks chosen by them and the masks made of them, against their 64-bit statement: equal to
the last bit and the last block."""
import pytest
import torch

import selection_reference as ref
import serving_reference as serving

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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(lens, page, pages, seed, most=None):
    """A block table of shuffled distinct pages, -1 past each sequence's."""
    need = [-(-n // page) for n in lens]
    most = most or max(max(need), 1)
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    assert sum(need) <= pages
    rows = []
    for n in need:
        rows.append([perm.pop() for _ in range(n)] + [-1] * (most - n))
    return _i32(rows).view(len(lens), most)


def _same(a, b):
    return torch.equal(a.cpu().double(), b.cpu().double())


# ------------------------------------------------------------------------- summaries

def _check_update(bsa, k, lens, new, table, marker=77):
    pages, page, hkv, d = k.shape
    index = bsa.bsattn_block_index(pages, hkv, page, d)
    index.codes.fill_(marker)
    index.scales.fill_(-3.0)
    want_c, want_s = index.codes.double().cpu(), index.scales.double().cpu()
    for b, (n, m) in enumerate(zip(lens, new)):
        if m <= 0:
            continue
        for j in range((n - m) // 64, -(-n // 64)):
            p, r = int(table[b, j * 64 // page]), j * 64 % page
            rows = k[p, r:r + min(64, n - 64 * j)].transpose(0, 1)
            want_c[p, r // 64], want_s[p, r // 64] = (x.cpu() for x in ref.summary(rows))
    bsa.bsattn_index_update(k, _i32(lens), _i32(new), table, index)
    assert _same(index.codes, want_c)
    assert _same(index.scales, want_s)
    assert bsa.bsattn_get_device_status(bsa.status_workspace("cuda")) == 0
    return index


@pytest.mark.parametrize("d,dtype", [(64, F16), (64, BF16), (128, F16), (128, BF16)])
@pytest.mark.parametrize("hkv", [1, 3, 8, 17])
@pytest.mark.parametrize("page", [64, 192])
def test_update_types_heads_pages(bsa, d, dtype, hkv, page):
    lens, new = [1, 64, 65, 500, 0, 129, 63], [1, 64, 2, 437, 0, 129, 0]
    k = _rand(40, page, hkv, d, dtype=dtype, seed=d + hkv)
    _check_update(bsa, k, lens, new, _table(lens, page, 40, 1))


def test_update_many_sequences(bsa):
    """More sequences than threads, most with a token each, some with none and one with many."""
    lens = [(37 * b) % 200 for b in range(700)]
    new = [min(n, b % 3) for b, n in enumerate(lens)]
    new[123] = lens[123]
    k = _rand(2900, 64, 2, 64, dtype=BF16, seed=3)
    _check_update(bsa, k, lens, new, _table(lens, 64, 2900, 2))


def test_update_more_blocks_than_all_warps_look_up_at_once(bsa):
    k = _rand(2300, 64, 17, 64, dtype=F16, seed=5)
    _check_update(bsa, k, [2200 * 64 - 3, 70], [2200 * 64 - 3, 70], _table([2200 * 64 - 3, 70], 64, 2300, 4))


def test_update_one_token_at_a_time(bsa):
    """Token by token is the same as all at once; what stands past the end has no effect."""
    k = _rand(4, 64, 2, 128, dtype=BF16, seed=5)
    table = _i32([[2, 0, 3]])
    index = bsa.bsattn_block_index(4, 2, 64, 128)
    poisoned = k.clone()
    for n in range(1, 151):
        now = poisoned.clone()
        for j in range(3):
            now[table[0, j], max(0, min(64, n - 64 * j)):] = float("nan")
        bsa.bsattn_index_update(now, _i32([n]), _i32([1]), table, index)
    want = _check_update(bsa, k, [150], [150], table, marker=0)
    assert torch.equal(index.codes[table[0].long()], want.codes[table[0].long()])
    assert torch.equal(index.scales[table[0].long()], want.scales[table[0].long()])


def test_update_extreme_values(bsa):
    """Infinities, NaN, sums past the largest number, subnormals and zeros."""
    k = _rand(8, 64, 1, 64, dtype=BF16, seed=6)
    k[0, 5, 0, 3] = float("inf")
    k[1, 60, 0, 0] = float("nan")
    k[2] = 3e38
    k[3] = 0
    k[4] = (k[4].float() * 1e-39).to(BF16)
    k[5] = torch.finfo(BF16).smallest_normal * 2.0 ** -7
    k[6, 0, 0, 0], k[6, 1, 0, 0] = float("inf"), -float("inf")
    k[7] = (k[7].float() * 1e37).to(BF16)
    index = _check_update(bsa, k, [64] * 8, [64] * 8, _i32([[p] for p in range(8)]))
    assert torch.isinf(index.scales[[0, 1, 2, 6]]).all() and not index.codes[[0, 1, 2, 3, 6]].any()
    # one row of the block alone: the infinity stands past the end
    _check_update(bsa, k, [5], [5], _i32([[0]]))


def test_update_reports_what_is_out_of_range(bsa):
    k = _rand(4, 64, 2, 64, dtype=F16, seed=7)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run(lens, new, table):
        index = bsa.bsattn_block_index(4, 2, 64, 64)
        bsa.bsattn_index_update(k, _i32(lens), _i32(new), _i32(table), index, ws=ws)
        return index, bsa.bsattn_get_device_status(ws)

    good, status = run([100], [100], [[1, 2]])
    assert status == 0
    for lens, new, table in (([100, 100], [100, 100], [[1, 2], [-1, -1]]), ([100, 64], [100, 64], [[1, 2], [4, 0]]),
                             ([100, -5], [100, 3], [[1, 2], [3, 3]]), ([100, 5], [100, -3], [[1, 2], [3, 3]])):
        index, status = run(lens, new, table)
        assert status == bsa.BSATTN_ERR_BAD_INDEX
        assert torch.equal(index.codes, good.codes) and torch.equal(index.scales, good.scales)
    # past the table: what is in it; more new tokens than there are: all
    index, status = run([1000], [1000], [[1, 2]])
    assert status == bsa.BSATTN_ERR_BAD_INDEX and torch.equal(index.scales != 0, good.scales != 0)
    index, status = run([100], [101], [[1, 2]])
    assert status == bsa.BSATTN_ERR_BAD_INDEX and torch.equal(index.codes, good.codes)


def test_update_far_rows(bsa):
    """A cache whose rows lie past 32-bit offsets."""
    pages = (1 << 32) // (64 * 8 * 128) + 3
    k = torch.zeros(pages, 64, 8, 128, dtype=F16, device="cuda")
    k[pages - 1] = _rand(64, 8, 128, dtype=F16, seed=8)
    index = bsa.bsattn_block_index(pages, 8, 64, 128)
    bsa.bsattn_index_update(k, _i32([64]), _i32([1]), _i32([[pages - 1]]), index)
    codes, scales = ref.summary(k[pages - 1].transpose(0, 1))
    assert _same(index.codes[pages - 1, 0], codes) and _same(index.scales[pages - 1, 0], scales)
    assert not index.codes[:pages - 1].any()


# ------------------------------------------------------------------------- decode choice

def _random_index(bsa, pages, per, hkv, d, seed):
    codes, scales = ref.quantise(_rand(pages, per, hkv, d, dtype=torch.float32, seed=seed).double())
    return bsa.BlockIndex(codes.to(torch.int8).contiguous(), scales.float().contiguous())


def _check_select(bsa, q, index, lens, table, max_sel, sinks, recent, status=0):
    page = 64 * index.codes.shape[1]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = bsa.bsattn_decode_select(q, index, _i32(lens), table, max_sel, sinks, recent, ws=ws)
    want = ref.select(q.cpu(), index.codes.cpu(), index.scales.cpu(), lens, table.cpu(), max_sel, sinks, recent, page)
    assert torch.equal(got.cpu(), want)
    assert bsa.bsattn_get_device_status(ws) == status
    return got


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 2), (5, 1), (14, 2), (8, 1), (24, 8)])
@pytest.mark.parametrize("d,dtype", [(64, F16), (64, BF16), (128, F16), (128, BF16)])
def test_select_heads_and_types(bsa, hq, hkv, d, dtype):
    lens = [0, 1, 64, 700, 5000, 2111]
    index = _random_index(bsa, 130, 1, hkv, d, seed=hq)
    q = _rand(6, hq, d, dtype=dtype, seed=hq + d)
    _check_select(bsa, q, index, lens, _table(lens, 64, 130, 3), 9, 1, 2)


@pytest.mark.parametrize("page", [64, 128, 320])
@pytest.mark.parametrize("max_sel,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (7, 3, 4), (8, 0, 1), (31, 1, 1),
                                                  (64, 2, 2), (1000, 0, 0)])
def test_select_counts(bsa, page, max_sel, sinks, recent):
    lens = [4000, 63, 640, 4097, 448]
    index = _random_index(bsa, 160, page // 64, 2, 64, seed=page)
    q = _rand(5, 6, 64, dtype=BF16, seed=max_sel)
    _check_select(bsa, q, index, lens, _table(lens, page, 160, 4, most=70), max_sel, sinks, recent)


def test_select_equal_scores(bsa):
    """Equal scores, in part or all: the lower block first."""
    index = _random_index(bsa, 50, 1, 1, 64, seed=1)
    table = _i32([list(range(50))])
    q = _rand(1, 4, 64, dtype=F16, seed=2)
    for k in (1, 5, 20, 49):
        zero = bsa.BlockIndex(torch.zeros_like(index.codes), torch.ones_like(index.scales))
        got = _check_select(bsa, q, zero, [3200], table, k, 0, 0)
        assert got[0, 0].tolist() == list(range(k))
        _check_select(bsa, q * 0, index, [3200], table, k, 0, 1)
        # runs of the same summary
        some = bsa.BlockIndex(index.codes[torch.arange(50) // 7 * 7].contiguous(), index.scales[torch.arange(50) // 7 * 7].contiguous())
        _check_select(bsa, q, some, [3200], table, k, 1 if k > 1 else 0, 0)
        # the same two scores in turn, one of them the other's negative
        signs = bsa.BlockIndex(index.codes[:1].repeat(50, 1, 1, 1) * torch.where(torch.arange(50, device="cuda") % 2 == 0, 1, -1)
                               .to(torch.int8)[:, None, None, None], torch.ones_like(index.scales))
        _check_select(bsa, q[:, :1].contiguous(), signs, [3200], table, k, 0, 0)


def test_select_extreme_scores(bsa):
    """Summaries of blocks and queries that are not finite; scores that overflow, or underflow to 0."""
    index = _random_index(bsa, 60, 1, 2, 64, seed=3)
    index.codes[[3, 41]] = 0
    index.scales[[3, 41]] = float("inf")
    index.scales[10:14] = 1e30
    index.scales[20:30] *= 1e-38
    table = _i32([list(range(60))] * 4)
    q = _rand(4, 8, 64, dtype=BF16, seed=4)
    q[1, 0, 5] = float("nan")
    q[1, 5] = float("inf")
    q[2] = (q[2].float() * 1e37).to(BF16)
    q[3] = (q[3].float() * 1e-38).to(BF16)
    for k in (1, 2, 3, 6, 30, 59):
        got = _check_select(bsa, q, index, [60 * 64] * 4, table, k, 0, 0)
        if k > 1:
            # (in sequence 2 other scores are infinite too, and the lower block comes first)
            for b in (0, 1, 3):
                assert (got[b] == 3).any(-1).all() and (got[b] == 41).any(-1).all()


@pytest.mark.parametrize("d", [64, 128])
def test_select_largest_products(bsa, d):
    """Codes at both ends of their range, so that sums are as large as they get, and scores one apart."""
    g = torch.Generator().manual_seed(d)
    codes = torch.full((60, 1, 2, d), 127, dtype=torch.int8)
    codes[20:40] = -127
    codes[40:] = torch.where(torch.rand(20, 1, 2, d, generator=g) < 0.5, 127, -127).to(torch.int8)
    for j in range(60):                                     # one less in one channel
        codes[j, 0, :, j % d] -= torch.sign(codes[j, 0, :, j % d]) * (j % 3)
    index = bsa.BlockIndex(codes.cuda(), torch.ones(60, 1, 2, device="cuda"))
    table = _i32([list(range(60))] * 3)
    q = torch.ones(3, 16, d, dtype=BF16, device="cuda")
    q[1] = -1
    q[2] = torch.where(_rand(16, d, dtype=BF16, seed=d) < 0, -1.0, 1.0).to(BF16)
    q[:, 3, ::2] *= 0.5
    for k in (1, 7, 10, 21, 33, 59):
        _check_select(bsa, q, index, [60 * 64] * 3, table, k, 0, 0)


def test_select_reports_what_is_out_of_range(bsa):
    index = _random_index(bsa, 20, 1, 2, 64, seed=5)
    q = _rand(4, 4, 64, dtype=F16, seed=6)
    bad = bsa.BSATTN_ERR_BAD_INDEX
    table = _table([640, 640, 0, 0], 64, 20, 5)
    _check_select(bsa, q, index, [640, 600, 0, 0], table, 4, 1, 1)
    _check_select(bsa, q, index, [640, -3, 0, 0], table, 4, 1, 1, status=bad)
    _check_select(bsa, q, index, [641, 2 ** 31 - 1, 0, 0], table, 4, 1, 1, status=bad)
    _check_select(bsa, q, index, [640, 640, 0, 64], table, 4, 1, 1, status=bad)             # -1 in the table
    for page in (-7, 20, 2 ** 31 - 1):
        table[0, 9] = page                                                              # a forced block
        table[1, 3] = page
        for k in (3, 9, 10, 40):
            _check_select(bsa, q, index, [640, 640, 0, 0], table, k, 1, 1, status=bad)


@pytest.mark.parametrize("d,page", [(64, 256), (128, 64)])
def test_select_long(bsa, d, page):
    """Several hundred thousand tokens, and the longest table that the call takes."""
    lens = [400_000, 250_001]
    pages = -(-650_001 // page) + 2
    index = _random_index(bsa, pages, page // 64, 2, d, seed=7)
    q = _rand(2, 8, d, dtype=BF16, seed=8)
    _check_select(bsa, q, index, lens, _table(lens, page, pages, 6), 200, 1, 4)
    width = 3_000_000 // page
    wide = torch.arange(width, dtype=torch.int32, device="cuda").remainder(pages).repeat(2, 1)
    got = bsa.bsattn_decode_select(q, index, _i32([width * page, 10]), wide, 100, 1, 1)
    # every summary is there many times: of equal scores the lower block
    whole = ref.select(q[:1].cpu(), index.codes.cpu(), index.scales.cpu(), [pages * page], wide[:1, :pages].cpu(), 100, 0, 0, page)
    times = -(-width // pages)
    best = [j for j in whole[0, 0].tolist()]
    assert got[0, 0, 0] == 0 and got[0, 0, -1] == width * page // 64 - 1
    assert {int(j) % (pages * page // 64) for j in got[0, 0, 1:-1].tolist()} <= set(best) | {0} and times > 1
    assert got[1, 0].tolist() == [0] + [-1] * 99


@pytest.mark.parametrize("B,hkv,width", [(1, 8, 768), (1, 8, 769), (2, 8, 2047), (2, 8, 2048), (9, 8, 2300), (1, 8, 4500),
                                         (19, 8, 2050), (25, 8, 2100), (40, 8, 2047), (80, 8, 2048), (50, 3, 900)])
@pytest.mark.parametrize("d", [64, 128])
def test_select_rows_of_one_cta_and_of_several(bsa, B, hkv, width, d):
    """Tables of few and many blocks, rows that fill the GPU or do not, sequences much shorter than the table."""
    lens = [(width * 64, 1, 33 * 64 + 1, 0, 517 * 64, 1024 * 64 - 5)[b % 6] if b < 12 else 64 * (b % 50) for b in range(B)]
    lens = [min(n, width * 64) for n in lens]
    pages = sum(-(-n // 64) for n in lens) + 1
    index = _random_index(bsa, pages, 1, hkv, d, seed=width)
    q = _rand(B, 2 * hkv, d, dtype=BF16, seed=B)
    _check_select(bsa, q, index, lens, _table(lens, 64, pages, 9, most=width), 70, 1, 3)


# ------------------------------------------------------------------------- masks

def _check_mask(bsa, q, k, topk, causal, sinks, recent, dense):
    got = bsa.bsattn_mask_from_qk(q, k, topk, causal, sinks, recent, dense)
    want = ref.mask(q, k, topk, causal, sinks, recent, dense)
    assert torch.equal(got.cpu(), want)
    return got


@pytest.mark.parametrize("Sq,Sk", [(1, 1), (64, 64), (65, 65), (1, 700), (257, 1000), (1000, 1000), (700, 300), (1100, 1111)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("topk,sinks,recent,dense", [(4, 1, 1, False), (0, 0, 0, False), (3, 0, 0, True), (2, 2, 3, False),
                                                     (100, 0, 0, False), (1, 0, 1, True)])
def test_mask_lengths_and_rules(bsa, Sq, Sk, causal, topk, sinks, recent, dense):
    q, k = _rand(1, 2, Sq, 64, dtype=BF16, seed=Sq), _rand(1, 2, Sk, 64, dtype=BF16, seed=Sk + 1)
    _check_mask(bsa, q, k, topk, causal, sinks, recent, dense)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 2), (5, 1), (10, 5)])
@pytest.mark.parametrize("d,dtype", [(64, F16), (128, F16), (128, BF16)])
def test_mask_heads_and_types(bsa, Hq, Hkv, d, dtype):
    q, k = _rand(2, Hq, 900, d, dtype=dtype, seed=Hq), _rand(2, Hkv, 1300, d, dtype=dtype, seed=Hkv)
    _check_mask(bsa, q, k, 5, True, 1, 2, False)


def test_mask_strided_views(bsa):
    """Projections' layouts, a fused row, heads that share memory, and gaps between rows."""
    fused = _rand(2, 600, 8 * 64, dtype=BF16, seed=1)
    q = fused[..., :4 * 64].unflatten(-1, (4, 64)).transpose(1, 2)
    k = fused[..., 4 * 64:6 * 64].unflatten(-1, (2, 64)).transpose(1, 2)
    got = _check_mask(bsa, q, k, 3, True, 1, 1, True)
    assert torch.equal(got, bsa.bsattn_mask_from_qk(q.contiguous(), k.contiguous(), 3, True, 1, 1, True))
    shared = k[:, :1].expand(2, 4, 600, 64)
    assert torch.equal(bsa.bsattn_mask_from_qk(q, shared, 3, True), bsa.bsattn_mask_from_qk(q, k[:, :1], 3, True))
    gaps = _rand(1, 2, 300, 80, dtype=BF16, seed=2)[..., 8:72]
    _check_mask(bsa, gaps, gaps, 2, False, 0, 0, False)
    with pytest.raises(ValueError):
        bsa.bsattn_mask_from_qk(fused[..., ::2].unflatten(-1, (4, 64)).transpose(1, 2), k, 3, True)
    with pytest.raises(bsa.BsattnError):
        bsa.bsattn_mask_from_qk(_rand(1, 2, 300, 68, dtype=BF16, seed=2)[..., :64], k[:1], 2, False)


@pytest.mark.parametrize("Sk", [130 * 64 + 5, 225_300 + 64])
def test_mask_long_rows(bsa, Sk):
    """Rows of keys past one read of a warp, and past what 16 rows have room for."""
    q, k = _rand(1, 1, 600, 64, dtype=BF16, seed=3), _rand(1, 1, Sk, 64, dtype=BF16, seed=4)
    _check_mask(bsa, q, k, 50, True, 1, 2, True)
    _check_mask(bsa, q, k, 700, False, 0, 0, False)


def test_mask_of_many_heads(bsa):
    """More CTAs than SMs."""
    q, k = _rand(2, 40, 1100, 64, dtype=BF16, seed=3), _rand(2, 8, 1300, 64, dtype=BF16, seed=4)
    _check_mask(bsa, q, k, 5, True, 1, 1, True)
    _check_mask(bsa, q[:, :, :1030], k[:, :, :1030], 3, False, 0, 2, False)


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
def test_mask_of_many_blocks(bsa, d, dtype):
    """Dozens of blocks for every SM."""
    q, k = _rand(1, 50, 3300, d, dtype=dtype, seed=5), _rand(1, 50, 3201, d, dtype=dtype, seed=6)
    _check_mask(bsa, q, k, 6, True, 1, 1, False)


def test_mask_output_at_any_address(bsa):
    q, k = _rand(1, 2, 300, 64, dtype=F16, seed=3), _rand(1, 2, 1024, 64, dtype=F16, seed=4)
    want = bsa.bsattn_mask_from_qk(q, k, 5, True)
    flat = torch.full((want.numel() + 3,), 9, dtype=torch.uint8, device="cuda")
    for at in range(4):
        flat.fill_(9)
        out = flat[at:at + want.numel()].view(want.shape)
        assert torch.equal(bsa.bsattn_mask_from_qk(q, k, 5, True, out=out), want)
        assert (flat[:at] == 9).all() and (flat[at + want.numel():] == 9).all()


def test_mask_extreme_values(bsa):
    q, k = _rand(1, 2, 700, 64, dtype=BF16, seed=5), _rand(1, 2, 700, 64, dtype=BF16, seed=6)
    q[0, 0, 70] = float("nan")
    q[0, 1, 300, 3] = float("inf")
    k[0, 0, 200, 1] = float("inf")
    k[0, 1, 500] = float("nan")
    k[0, 1, 64:128] = 0
    q[0, 1, 640:] = (q[0, 1, 640:].float() * 1e38).to(BF16)
    k[0, 1, 640:] = (k[0, 1, 640:].float() * 1e30).to(BF16)
    for topk in (1, 2, 5):
        _check_mask(bsa, q, k, topk, False, 0, 0, False)
        _check_mask(bsa, q, k, topk, True, 1, 1, False)
    _check_mask(bsa, torch.zeros_like(q), k[:, :, :0].new_zeros(1, 2, 700, 64), 4, True, 0, 1, False)


def test_mask_empty(bsa):
    q = _rand(1, 2, 100, 64, dtype=BF16, seed=7)
    assert bsa.bsattn_mask_from_qk(q, q[:, :, :0], 4, True).shape == (1, 2, 2, 0)
    assert bsa.bsattn_mask_from_qk(q[:, :, :0], q, 4, True).shape == (1, 2, 0, 2)
    assert bsa.bsattn_mask_from_qk(q[:0], q[:0], 4, True).shape == (0, 2, 2, 2)


# ------------------------------------------------------------------------- as they are used

def _rows_of(k_pages, v_pages, table, groups):
    page = k_pages.shape[1]

    def rows(b, g, n):
        j = torch.arange(n, device="cuda")
        at = table[b].long()[j // page], j % page
        return k_pages[at[0], at[1], g], v_pages[at[0], at[1], g]
    rows.groups = groups
    return rows


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
def test_a_server_step(bsa, d, dtype):
    """Plan pages, write rows, summarise, choose and attend, for a prompt and for tokens after it; over 16 and
    over 4 bits."""
    B, Hq, Hkv, page, pages, max_pages, max_sel = 3, 8, 2, 128, 60, 16, 6
    k_pages, v_pages = (torch.full((pages, page, Hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    index = bsa.bsattn_block_index(pages, Hkv, page, d)
    cache4 = bsa.bsattn_kv4_cache(pages, Hkv, page, d)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    free, left = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0).contiguous(), _i32([pages])
    cached = _i32([0] * B)
    for step, new in enumerate(([1500, 700, 64], [1, 1, 1], [1, 1, 1], [70, 1, 0])):
        new_lens, T = _i32(new), sum(new)
        slots, starts, lens, left = bsa.bsattn_paged_plan(cached, new_lens, free, left, table, page, T)
        k, v = _rand(T, Hkv, d, dtype=dtype, seed=10 * step), _rand(T, Hkv, d, dtype=dtype, seed=10 * step + 1)
        k_pages.view(-1, Hkv, d)[slots], v_pages.view(-1, Hkv, d)[slots] = k, v
        bsa.bsattn_kv4_append(k, v, slots, cache4)
        bsa.bsattn_index_update(k_pages, lens, new_lens, table, index)
        q = _rand(B, Hq, d, dtype=dtype, seed=10 * step + 2)
        chosen = bsa.bsattn_decode_select(q, index, lens, table, max_sel)
        n = lens.tolist()
        assert torch.equal(chosen.cpu(), ref.select(q.cpu(), index.codes.cpu(), index.scales.cpu(), n, table.cpu(), max_sel, 1, 1, page))

        def seen(b, g, m):
            on = torch.zeros(-(-m // 64) * 64, dtype=torch.bool, device="cuda")
            for j in chosen[b, g].tolist():
                if j >= 0:
                    on[64 * j:64 * j + 64] = True
            return on[:m]
        got = bsa.bsattn_decode_paged(q, k_pages, v_pages, lens, chosen, table)
        serving.check(got, *serving.decode(q, _rows_of(k_pages, v_pages, table, Hkv), n, seen, dtype))
        flat_k, flat_v = (x.view(pages * page, Hkv, d) for x in (k_pages, v_pages))
        assert not torch.isnan(bsa.bsattn_decode_paged_kv4(q, cache4, lens, table, chosen)).any()
        # every block chosen: the whole sequence
        every = bsa.bsattn_decode_select(q, index, lens, table, 64)
        whole = bsa.bsattn_decode_window_paged(q, k_pages, v_pages, lens, table, 1 << 20)
        near = bsa.bsattn_decode_paged(q, k_pages, v_pages, lens, every, table)
        size = max(float(flat_v[slots].abs().max()), 1.0)
        assert (near.double() - whole.double()).abs().max() <= 2 * serving.half_eps(dtype) * 2 * size + 1e-4 * size
        cached = lens
    assert bsa.bsattn_get_device_status(bsa.status_workspace("cuda")) == 0


@pytest.mark.parametrize("d,dtype,S", [(64, F16, 1000), (128, BF16, 777)])
def test_a_sparse_prompt(bsa, d, dtype, S):
    """The mask is what the sparse prefill takes, and with every block in it the prefill is dense."""
    q, k, v = (_rand(1, 4, S, d, dtype=dtype, seed=s) for s in (1, 2, 3))
    mask = bsa.bsattn_mask_from_qk(q, k, 4, True, use_dense_for_last_block=True)
    got = bsa.bsattn_prefill(q, k, v, mask, True)
    i = torch.arange(S, device="cuda")
    for h in range(4):
        on = mask[0, h].bool().repeat_interleave(64, 0).repeat_interleave(64, 1)[:S, :S] & (i <= i[:, None])
        serving.check(got[0, h], *serving.attend(q[0, h], k[0, h], v[0, h], on, dtype, dtype))
    full = bsa.bsattn_mask_from_qk(q, k, 1000, True)
    assert torch.equal(full[0, 0].cpu(), torch.ones_like(full[0, 0].cpu()).tril())


def test_calls_on_other_streams_and_in_graphs(bsa):
    index = _random_index(bsa, 130, 1, 2, 64, seed=1)
    lens = [5000, 2111]
    table, n = _table(lens, 64, 130, 3), _i32(lens)
    q = _rand(2, 8, 64, dtype=BF16, seed=2)
    x, y = _rand(1, 4, 3000, 64, dtype=BF16, seed=3), _rand(1, 2, 3000, 64, dtype=BF16, seed=4)
    k_pages = _rand(130, 64, 2, 64, dtype=BF16, seed=5)
    fresh = bsa.bsattn_block_index(130, 2, 64, 64)

    def calls(to):
        bsa.bsattn_index_update(k_pages, n, n, table, to)
        return (bsa.bsattn_decode_select(q, index, n, table, 9), bsa.bsattn_decode_select(q, to, n, table, 9),
                bsa.bsattn_mask_from_qk(x, y, 7, True))
    want = calls(fresh)
    torch.cuda.synchronize()
    # on two streams at once
    streams = [torch.cuda.Stream() for _ in range(2)]
    other = [bsa.bsattn_block_index(130, 2, 64, 64) for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s, to in zip(streams, other):
        with torch.cuda.stream(s):
            got.append([calls(to) for _ in range(20)][-1])
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    # captured, with new inputs in the same places
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = calls(fresh)
    q.copy_(_rand(2, 8, 64, dtype=BF16, seed=12))
    x.copy_(_rand(1, 4, 3000, 64, dtype=BF16, seed=13))
    k_pages.copy_(_rand(130, 64, 2, 64, dtype=BF16, seed=15))
    graph.replay()
    torch.cuda.synchronize()
    again = calls(bsa.bsattn_block_index(130, 2, 64, 64))
    assert all(torch.equal(a, b) for a, b in zip(captured, again))
    assert not torch.equal(captured[0], want[0]) and not torch.equal(captured[2], want[2])


# ------------------------------------------------------------------------- ties between CTAs, the widest tables

@pytest.mark.parametrize("B,hkv,width", [(5, 8, 2048), (1, 8, 2048), (1, 8, 4096), (25, 8, 2048), (50, 8, 2048)])
def test_select_equal_scores_of_several_ctas(bsa, B, hkv, width):
    """Rows of two, four and eight CTAs, and of one for long tables: of equal scores the lower block comes first, across
    the places where one CTA's blocks end and the next one's begin."""
    index = _random_index(bsa, width, 1, hkv, 64, seed=width + B)
    table = torch.arange(width, dtype=torch.int32, device="cuda").repeat(B, 1)
    lens = [width * 64 if b == 0 else 64 * 700 - 3 if b == 1 else 64 * (b % 40) for b in range(B)]
    q = _rand(B, 2 * hkv, 64, dtype=BF16, seed=B)
    zero = bsa.BlockIndex(torch.zeros_like(index.codes), torch.ones_like(index.scales))
    for k in (1, 255, 256, 257, 511, 512, 513, 1024, 1025, 2047):
        got = bsa.bsattn_decode_select(q, zero, _i32(lens), table, k, 0, 0).cpu()
        for b, n in enumerate(lens):
            n = min(-(-n // 64), k)
            want = torch.tensor(list(range(n)) + [-1] * (k - n), dtype=torch.int32)
            assert torch.equal(got[b], want.expand(hkv, k))
    runs = torch.arange(width, device="cuda") // 100 * 100
    some = bsa.BlockIndex(index.codes[runs].contiguous(), index.scales[runs].contiguous())
    turns = torch.arange(width, device="cuda") % 3
    few = bsa.BlockIndex(index.codes[turns].contiguous(), index.scales[turns].contiguous())
    for k in (130, 512, 777):
        _check_select(bsa, q, some, lens, table, k, 1, 2)
        _check_select(bsa, q, few, lens, table, k, 0, 1)


@pytest.mark.parametrize("d", [64, 128])
def test_select_widest_table(bsa, d):
    """More rows than two CTAs an SM each, in a table for 3000000 tokens, one of them as long as that."""
    width, hkv, B = 46875, 8, 39
    lens = [width * 64 - 5 if b == 7 else 3000 * 64 if b == 20 else 64 * (b % 9) for b in range(B)]
    pages = sum(-(-n // 64) for n in lens) + 1
    index = _random_index(bsa, pages, 1, hkv, d, seed=d)
    q = _rand(B, hkv, d, dtype=BF16, seed=d)
    table = _table(lens, 64, pages, 11, most=width)
    _check_select(bsa, q, index, lens, table, 90, 1, 3)
    same = bsa.BlockIndex(torch.zeros_like(index.codes), torch.ones_like(index.scales))
    got = bsa.bsattn_decode_select(q, same, _i32(lens), table, 40_000, 0, 1)
    want = torch.tensor(list(range(39_999)) + [width - 1], dtype=torch.int32)
    assert torch.equal(got[7].cpu(), want.expand(hkv, 40_000))


@pytest.mark.parametrize("big", [2 ** 32 + 64, 2 ** 31, 2 ** 32])
def test_mask_sizes_past_32_bits(bsa, big):
    """Broadcast views whose sizes a C int would cut off."""
    x = _rand(1, 1, 64, 64, dtype=BF16, seed=1)
    one = x[:, :, :1]
    with pytest.raises(ValueError):
        bsa.bsattn_mask_from_qk(x, one.expand(1, 1, big, 64), 4, True)
    with pytest.raises(ValueError):
        bsa.bsattn_mask_from_qk(one.expand(1, 1, big, 64), x, 4, True)
    with pytest.raises(ValueError):
        bsa.bsattn_mask_from_qk(one.expand(big, 1, 1, 64), one.expand(big, 1, 1, 64), 4, True)
    with pytest.raises(ValueError):
        bsa.bsattn_mask_from_qk(one.expand(1, big, 1, 64), one, 4, True)


def test_index_of_a_4bit_cache(bsa):
    """Pages gathered from a 4-bit cache and summarised as pages of their own, each as a sequence."""
    pages, page, hkv, d, lens = 12, 128, 2, 64, [300, 128, 61]
    table, cache = _table(lens, page, pages, 5), bsa.bsattn_kv4_cache(pages, hkv, page, d)
    slots = torch.cat([table[b].long()[torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page
                       for b, n in enumerate(lens)])
    k, v = (_rand(len(slots), hkv, d, dtype=BF16, seed=s) for s in (1, 2))
    bsa.bsattn_kv4_append(k, v, slots, cache)
    mine = torch.tensor([int(p) for b, n in enumerate(lens) for p in table[b, :-(-n // page)]], device="cuda")
    rows = _i32([min(page, n - at) for n in lens for at in range(0, n, page)])
    whole = (mine[:, None] * page + torch.arange(page, device="cuda")).view(-1)
    got, _ = bsa.bsattn_kv4_gather(whole, cache, BF16)
    got = got.view(len(mine), page, hkv, d)
    scratch = bsa.bsattn_block_index(len(mine), hkv, page, d)
    bsa.bsattn_index_update(got, rows, rows, torch.arange(len(mine), dtype=torch.int32, device="cuda")[:, None].contiguous(), scratch)
    index = bsa.bsattn_block_index(pages, hkv, page, d)
    index.codes[mine], index.scales[mine] = scratch.codes, scratch.scales
    for i, n in enumerate(rows.tolist()):
        for sub in range(-(-n // 64)):
            codes, scales = ref.summary(got[i, 64 * sub:min(64 * sub + 64, n)].transpose(0, 1))
            assert _same(index.codes[mine[i], sub], codes) and _same(index.scales[mine[i], sub], scales)
    q = _rand(3, 4, d, dtype=BF16, seed=3)
    blocks = _check_select(bsa, q, index, lens, table, 2, 0, 1)
    assert torch.isfinite(bsa.bsattn_decode_paged_kv4(q, cache, _i32(lens), table, blocks)).all()
