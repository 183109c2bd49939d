"""Sliding-window attention with sinks, prefill and decode, against its 64-bit statement."""
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


def _prefill(bsa, B, Hq, Hkv, Sq, Sk, d, dtype, window, sinks, seed=0, scale=1.0):
    q = _rand(B, Hq, Sq, d, dtype=dtype, seed=seed, scale=scale)
    k = _rand(B, Hkv, Sk, d, dtype=dtype, seed=seed + 1)
    v = _rand(B, Hkv, Sk, d, dtype=dtype, seed=seed + 2)
    got = bsa.bsattn_prefill_window(q, k, v, window, sinks)
    ref.check(got, *ref.window_prefill(q, k, v, window, sinks))
    return got


# ------------------------------------------------------------------------- prefill

@pytest.mark.parametrize("Sq,Sk", [(1, 1), (1, 300), (127, 127), (128, 128), (129, 129), (257, 1000), (300, 300),
                                   (200, 150), (5, 2), (640, 640)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (128, 128), (129, 130), (10000, 0), (10000, 4)])
def test_prefill_lengths_and_windows(bsa, Sq, Sk, window, sinks):
    _prefill(bsa, 1, 4, 2, Sq, Sk, 128, BF16, window, sinks, seed=Sq + Sk)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (3, 3), (6, 2), (8, 1), (16, 2), (10, 5)])
@pytest.mark.parametrize("d,dtype", [(64, F16), (64, BF16), (128, F16), (128, BF16)])
def test_prefill_heads_and_types(bsa, Hq, Hkv, d, dtype):
    _prefill(bsa, 2, Hq, Hkv, 390, 517, d, dtype, 200, 3, seed=Hq * 100 + Hkv)


def test_prefill_many_items_a_cta(bsa):
    """More items than CTAs: every ring, barrier phase and accumulator is used again and again."""
    _prefill(bsa, 2, 8, 4, 2900, 2900, 128, BF16, 700, 5, seed=3)
    _prefill(bsa, 2, 9, 3, 2950, 2950, 64, F16, 333, 200, seed=4)


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("heads", [(2, 1), (3, 3), (60, 12)])
def test_prefill_few_and_many_query_tiles(bsa, heads, d, dtype):
    """The same lengths with few query tiles (a tile's keys shared out within a CTA) and with many."""
    for Sq, Sk, window, sinks in ((200, 900, 300, 4), (130, 2000, 5000, 0), (256, 1500, 100, 700), (300, 140, 64, 3),
                                  (1, 700, 640, 129), (129, 129, 1, 0)):
        _prefill(bsa, 1, *heads, Sq, Sk, d, dtype, window, sinks, seed=Sq)


def test_prefill_nan_reaches_its_row_from_either_half(bsa):
    q = _rand(1, 1, 100, 128, dtype=BF16, seed=1)
    k, v = _rand(1, 1, 1000, 128, dtype=BF16, seed=2), _rand(1, 1, 1000, 128, dtype=BF16, seed=3)
    for at in (3, 950):                                         # in the first half of the keys, in the second
        bad = k.clone()
        bad[0, 0, at] = float("nan")
        got = bsa.bsattn_prefill_window(q, bad, v, 2000, 0)
        assert torch.equal(got.isnan().any(-1)[0, 0], torch.arange(900, 1000, device="cuda") >= at)


def test_prefill_large_scores_rescale(bsa):
    """Scores that keep growing along a row: the reference maximum moves and O is rescaled."""
    q = _rand(1, 2, 600, 128, dtype=F16, seed=9)
    k = _rand(1, 2, 600, 128, dtype=F16, seed=10)
    v = _rand(1, 2, 600, 128, dtype=F16, seed=11)
    k = (k * torch.linspace(0.05, 3.0, 600, device="cuda")[:, None]).to(F16)
    got = bsa.bsattn_prefill_window(q, k, v, 500, 8)
    ref.check(got, *ref.window_prefill(q, k, v, 500, 8))


def test_prefill_empty_rows_are_zero(bsa):
    got = _prefill(bsa, 1, 2, 1, 300, 30, 64, BF16, 20, 0)
    assert got[:, :, :270].abs().max() == 0
    q = _rand(1, 2, 200, 64, dtype=BF16, seed=0)
    none = bsa.bsattn_prefill_window(q, q[:, :, :0], q[:, :, :0], 4, 1)
    assert none.shape == q.shape and none.abs().max() == 0


def test_prefill_strided_views(bsa):
    """Projections' layouts: [B, S, H, d], a fused QKV row, and an output inside a larger buffer."""
    B, S, Hq, Hkv, d = 2, 333, 4, 2, 64
    fused = _rand(B, S, (Hq + 2 * Hkv) * d, dtype=BF16, seed=5)
    q = fused[..., :Hq * d].unflatten(-1, (Hq, d)).transpose(1, 2)
    k = fused[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d)).transpose(1, 2)
    v = fused[..., (Hq + Hkv) * d:].unflatten(-1, (Hkv, d)).transpose(1, 2)
    room = torch.full((B, S + 3, Hq, d + 8), 7.0, dtype=BF16, device="cuda")
    out = room[:, :S, :, :d].transpose(1, 2)
    got = bsa.bsattn_prefill_window(q, k, v, 100, 2, out=out)
    assert got.data_ptr() == room.data_ptr()
    ref.check(got, *ref.window_prefill(q, k, v, 100, 2))
    assert (room[:, S:] == 7).all() and (room[..., d:] == 7).all()
    with pytest.raises(ValueError):
        bsa.bsattn_prefill_window(q[..., ::2], k[..., ::2], v[..., ::2], 4)
    with pytest.raises(bsa.BsattnError):                      # heads that share memory cannot be mapped
        bsa.bsattn_prefill_window(q, k[:, :1].expand(B, Hkv, S, d), v, 4)


def test_prefill_masked_keys_do_not_matter(bsa):
    """Keys that no row sees: any value, and bit-equal results."""
    q = _rand(1, 2, 130, 128, dtype=BF16, seed=1)
    k = _rand(1, 2, 700, 128, dtype=BF16, seed=2)
    v = _rand(1, 2, 700, 128, dtype=BF16, seed=3)
    a = bsa.bsattn_prefill_window(q, k, v, 40, 4)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, 4:700 - 130 - 39] = 50.0
    v2[:, :, 4:700 - 130 - 39] = -9.0
    assert torch.equal(a, bsa.bsattn_prefill_window(q, k2, v2, 40, 4))
    k2[:, :, 4:700 - 130 - 39] = float("nan")                 # a key may even be NaN
    assert torch.equal(a, bsa.bsattn_prefill_window(q, k2, v2, 40, 4))


@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (3, 3), (64, 16), (30, 30)])
@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_prefill_values_a_row_does_not_see_do_not_matter(bsa, Hq, Hkv, d, dtype, what):
    """Infinities and NaN in V reach the rows that see their key, all of those and no others."""
    S, window, sinks = 777, 200, 3
    q = _rand(1, Hq, S, d, dtype=dtype, seed=1)
    k, v = _rand(1, Hkv, S, d, dtype=dtype, seed=2), _rand(1, Hkv, S, d, dtype=dtype, seed=3)
    want, bound = ref.window_prefill(q, k, v, window, sinks)
    j, p = torch.arange(S, device="cuda"), torch.arange(S, device="cuda")[:, None]
    sees = (j <= p) & ((j < sinks) | (j > p - window))
    for keys in ([500], [1], [127, 128], [640, 700, 776], list(range(600, S)), list(range(0, 300))):
        bad = v.clone()
        bad[:, :, keys, 5:9] = what
        got = bsa.bsattn_prefill_window(q, k, bad, window, sinks)
        hit = sees[:, keys].any(-1)
        ref.check(got[:, :, ~hit], want[:, :, ~hit], bound[:, :, ~hit])
        assert not got[:, :, hit, 5:9].isfinite().any()
    qv = q.transpose(1, 2).contiguous().transpose(1, 2)                 # strided, and over the queries
    kv, bad = k.transpose(1, 2).contiguous().transpose(1, 2), v.transpose(1, 2).contiguous().transpose(1, 2)
    bad[:, :, 700] = what
    bsa.bsattn_prefill_window(qv, kv, bad, window, sinks, out=qv)
    ref.check(qv[:, :, :700], want[:, :, :700], bound[:, :, :700])
    assert not qv[:, :, 700:].isfinite().any()


def test_prefill_nan_query_is_not_hidden(bsa):
    q = _rand(1, 2, 70, 64, dtype=F16, seed=1)
    k, v = _rand(1, 2, 70, 64, dtype=F16, seed=2), _rand(1, 2, 70, 64, dtype=F16, seed=3)
    q[0, 1, 33] = float("nan")
    got = bsa.bsattn_prefill_window(q, k, v, 16, 0)
    assert got[0, 1, 33].isnan().all() and got.isnan().sum() == 64


def test_prefill_streams_and_graph(bsa):
    """Two calls at once on two streams, then a captured call replayed on changed inputs."""
    q = [_rand(1, 8, 1500, 128, dtype=BF16, seed=i) for i in (1, 2)]
    k = _rand(1, 4, 1500, 128, dtype=BF16, seed=5)
    v = _rand(1, 4, 1500, 128, dtype=BF16, seed=6)
    want = [bsa.bsattn_prefill_window(x, k, v, 300, 4) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    got = []
    for s, x in zip(streams, q):
        with torch.cuda.stream(s):
            got.append(bsa.bsattn_prefill_window(x, k, v, 300, 4))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = q[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = bsa.bsattn_prefill_window(x, k, v, 300, 4)
    x.copy_(q[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[1])


# ------------------------------------------------------------------------- decode

class _Rows:
    def __init__(self, k, v, table=None):
        self.k, self.v, self.table, self.groups = k, v, table, k.shape[2]

    def __call__(self, b, g, n):
        if self.table is None:
            return self.k[b, :n, g], self.v[b, :n, g]
        j = torch.arange(n, device=self.k.device)
        page = self.k.shape[1]
        at = self.table[b].long()[j // page], j % page
        return self.k[at[0], at[1], g], self.v[at[0], at[1], g]


def _paged(lens, Hkv, d, dtype, page, seed, fill=float("nan")):
    """A shuffled paged cache; everything past each length holds `fill`."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    total = sum(need) + 2
    perm = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    k = _rand(total, page, Hkv, d, dtype=dtype, seed=seed)
    v = _rand(total, page, Hkv, d, dtype=dtype, seed=seed + 1)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        if n and lens[b] % page:
            last = int(perm[at + n - 1])
            k[last, lens[b] % page:] = fill
            v[last, lens[b] % page:] = fill
        at += n
    return k, v, table.cuda()


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 100, 1000, 333, 2049]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 4), (100, 33), (64, 200), (5000, 0), (5000, 7)])
@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, F16)])
def test_decode_paged_windows(bsa, window, sinks, d, dtype):
    Hq, Hkv = 8, 2
    k, v, table = _paged(LENS, Hkv, d, dtype, 64, seed=window + d)
    q = _rand(len(LENS), Hq, d, dtype=dtype, seed=7)
    lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    got = bsa.bsattn_decode_window_paged(q, k, v, lens, table, window, sinks)
    want = ref.decode(q, _Rows(k, v, table), LENS, lambda b, g, n: ref.windowed(n, window, sinks, "cuda"), dtype)
    ref.check(got, *want)
    assert got[0].abs().max() == 0                              # no token: exactly 0


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (4, 4), (6, 2), (14, 2), (40, 5), (32, 8)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("page", [64, 192])
def test_decode_paged_heads(bsa, Hq, Hkv, dtype, page):
    lens = [700, 64, 1301]
    k, v, table = _paged(lens, Hkv, 128, dtype, page, seed=Hq)
    q = _rand(3, Hq, 128, dtype=dtype, seed=Hq + 1)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = bsa.bsattn_decode_window_paged(q, k, v, n, table, 600, 5)
    ref.check(got, *ref.decode(q, _Rows(k, v, table), lens, lambda b, g, m: ref.windowed(m, 600, 5, "cuda"), dtype))


@pytest.mark.parametrize("window,sinks", [(64, 0), (33, 2), (9999, 3)])
@pytest.mark.parametrize("Smax", [1000, 1003])
def test_decode_contiguous(bsa, window, sinks, Smax):
    """Sequences next to each other, odd strides between them, NaN past every length."""
    lens = [1000, 0, 999, 1, 500, 16]
    q = _rand(6, 8, 128, dtype=BF16, seed=1)
    k, v = _rand(6, Smax, 4, 128, dtype=BF16, seed=2), _rand(6, Smax, 4, 128, dtype=BF16, seed=3)
    for b, n in enumerate(lens):
        k[b, n:] = float("nan")
        v[b, n:] = float("nan")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = bsa.bsattn_decode_window(q, k, v, n, window, sinks)
    ref.check(got, *ref.decode(q, _Rows(k, v), lens, lambda b, g, m: ref.windowed(m, window, sinks, "cuda"), BF16))


def test_decode_masked_tokens_may_be_nan(bsa):
    """Tokens between the sinks and the window: never part of the result, whatever they hold."""
    lens = [900, 451]
    k, v, table = _paged(lens, 2, 128, BF16, 64, seed=3)
    q = _rand(2, 8, 128, dtype=BF16, seed=4)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = bsa.bsattn_decode_window_paged(q, k, v, n, table, 77, 5)
    for b, m in enumerate(lens):
        j = torch.arange(5, m - 77, device="cuda")
        k[table[b].long()[j // 64], j % 64] = float("nan")
        v[table[b].long()[j // 64], j % 64] = float("inf")
    assert torch.equal(a, bsa.bsattn_decode_window_paged(q, k, v, n, table, 77, 5))
    assert torch.isfinite(a.float()).all()


def test_decode_nan_query_is_not_hidden(bsa):
    lens = [900, 451]
    k, v, table = _paged(lens, 2, 128, BF16, 64, seed=3)
    q = _rand(2, 8, 128, dtype=BF16, seed=4)
    q[1, 3] = float("nan")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = bsa.bsattn_decode_window_paged(q, k, v, n, table, 400, 5)
    assert got[1, 3].isnan().all() and got.isnan().sum() == 128


def test_decode_long_and_ragged(bsa):
    """Sequences cut into many pieces next to short ones that share a CTA."""
    lens = [30000, 3, 12345, 64, 1, 20001, 700, 0, 129]
    k, v, table = _paged(lens, 2, 64, BF16, 64, seed=5)
    q = _rand(len(lens), 10, 64, dtype=BF16, seed=6)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = bsa.bsattn_decode_window_paged(q, k, v, n, table, 25000, 64)
    ref.check(got, *ref.decode(q, _Rows(k, v, table), lens, lambda b, g, m: ref.windowed(m, 25000, 64, "cuda"), BF16))
    for _ in range(5):                                          # joined in a fixed order: bit-equal
        assert torch.equal(got, bsa.bsattn_decode_window_paged(q, k, v, n, table, 25000, 64))


def test_decode_many_sequences(bsa):
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 200, (700,), generator=g).tolist()
    k, v, table = _paged(lens, 2, 64, F16, 64, seed=8)
    q = _rand(700, 4, 64, dtype=F16, seed=9)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = bsa.bsattn_decode_window_paged(q, k, v, n, table, 90, 3)
    ref.check(got, *ref.decode(q, _Rows(k, v, table), lens, lambda b, g, m: ref.windowed(m, 90, 3, "cuda"), F16))


@pytest.mark.parametrize("B", [2, 20, 37, 38, 39, 127, 128, 129])
def test_decode_batches_about_the_number_of_parts(bsa, B):
    """Sequences cut for themselves (few of them, or long parts) and end to end, with empty ones among them."""
    for n, window, d in ((70, 40, 64), (900, 600, 128)):
        lens = [0 if b % 7 == 3 else n + 53 * (b % 5) for b in range(B)]
        k, v, table = _paged(lens, 8, d, BF16, 64, seed=B + n)
        q = _rand(B, 8, d, dtype=BF16, seed=B)
        got = bsa.bsattn_decode_window_paged(q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), table,
                                             window, 5)
        ref.check(got, *ref.decode(q, _Rows(k, v, table), lens, lambda b, g, m: ref.windowed(m, window, 5, "cuda"), BF16))
        assert all(got[b].abs().max() == 0 for b in range(B) if lens[b] == 0)


def test_decode_flags_bad_pages_and_lengths(bsa):
    lens = [200, 200, 200]
    k, v, table = _paged(lens, 2, 128, BF16, 64, seed=3)
    q = _rand(3, 4, 128, dtype=BF16, seed=4)
    ws = torch.zeros(bsa.bsattn_decode_window_workspace_size(4, 2, 128), dtype=torch.uint8, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    good = bsa.bsattn_decode_window_paged(q, k, v, n, table, 300, 0, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == 0
    broken = table.clone()
    broken[1, 2] = 10 ** 6                                      # no such page: its tokens are left out
    got = bsa.bsattn_decode_window_paged(q, k, v, n, broken, 300, 0, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
    assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2])
    on = torch.ones(200, dtype=torch.bool, device="cuda")
    on[128:192] = False
    want = ref.decode(q, _Rows(k, v, table), lens, lambda b, g, m: on, BF16)
    ref.check(got[1], want[0][1], want[1][1])
    n[0] = -3                                                   # a negative length: no token, flagged
    got = bsa.bsattn_decode_window_paged(q, k, v, n, table, 300, 0, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
    assert got[0].abs().max() == 0
    want = ref.decode(q, _Rows(k, v, table), [0, 200, 200], lambda b, g, m: ref.windowed(m, 300, 0, "cuda"), BF16)
    ref.check(got, *want)                                       # (other pieces than before: not bit-equal)
    kc, vc = _rand(2, 64, 2, 128, dtype=BF16, seed=1), _rand(2, 64, 2, 128, dtype=BF16, seed=2)
    n = torch.tensor([64, 4000], dtype=torch.int32, device="cuda")   # past the cache: taken as its end
    got = bsa.bsattn_decode_window(q[:2], kc, vc, n, 40, 0, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
    want = ref.decode(q[:2], _Rows(kc, vc), [64, 64], lambda b, g, m: ref.windowed(m, 40, 0, "cuda"), BF16)
    ref.check(got, *want)


def test_decode_streams_graphs_and_shapes(bsa):
    """One workspace zeroed once serves changing shapes; streams and replayed graphs do not share one."""
    shapes = [([5000, 700], 8, 2), ([90] * 40, 6, 3), ([9000], 8, 1), ([300, 0, 2000], 16, 4)]
    ws = torch.zeros(max(bsa.bsattn_decode_window_workspace_size(hq, hkv, 64) for _, hq, hkv in shapes),
                     dtype=torch.uint8, device="cuda")
    calls, want = [], []
    for i, (lens, hq, hkv) in enumerate(shapes * 2):
        k, v, table = _paged(lens, hkv, 64, BF16, 64, seed=20 + i)
        q = _rand(len(lens), hq, 64, dtype=BF16, seed=i)
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        got = bsa.bsattn_decode_window_paged(q, k, v, n, table, 4000, 4, ws=ws)
        ref.check(got, *ref.decode(q, _Rows(k, v, table), lens, lambda b, g, m: ref.windowed(m, 4000, 4, "cuda"), BF16))
        calls.append((q, k, v, n, table))
        want.append(got)
    assert bsa.bsattn_get_device_status(ws) == 0
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for i, c in enumerate(calls):
            with torch.cuda.stream(streams[i % 4]):
                got.append((i, bsa.bsattn_decode_window_paged(*c, 4000, 4)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in got)
    graphs, outs = [], []
    for i in (0, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(bsa.bsattn_decode_window_paged(*calls[i], 4000, 4))
        graphs.append(g)
    for _ in range(10):                                         # replayed side by side
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[2])


def test_last_prefill_row_is_the_decode(bsa):
    """The token that a decode step attends with is the last row of the prefill over the same keys."""
    B, Hq, Hkv, S, d = 2, 8, 2, 777, 128
    q = _rand(B, Hq, S, d, dtype=BF16, seed=1)
    k, v = _rand(B, S, Hkv, d, dtype=BF16, seed=2), _rand(B, S, Hkv, d, dtype=BF16, seed=3)
    full = bsa.bsattn_prefill_window(q, k.transpose(1, 2), v.transpose(1, 2), 200, 4)
    one = bsa.bsattn_decode_window(q[:, :, -1].contiguous(), k, v, torch.full((B,), S, dtype=torch.int32, device="cuda"),
                                   200, 4)
    want, bound = ref.window_prefill(q[:, :, -1:], k.transpose(1, 2), v.transpose(1, 2), 200, 4)
    ref.check(full[:, :, -1:], want, bound)
    ref.check(one[:, :, None], want, bound)


@pytest.mark.parametrize("B", [1, 64])
def test_a_wait_that_expires_is_reported(bsa, B):
    """A budget of no time at all: the kernels give up, report it and leave the context usable.  A wait's
    first poll may itself last until the data is there: one sequence's decode may so come through whole,
    64 sequences' (1 GB in flight at once) cannot."""
    q = _rand(B, 8, 4000, 128, dtype=BF16, seed=1)
    k, v = _rand(B, 8, 4000, 128, dtype=BF16, seed=2), _rand(B, 8, 4000, 128, dtype=BF16, seed=3)
    ws = torch.zeros(bsa.bsattn_decode_window_workspace_size(8, 8, 128), dtype=torch.uint8, device="cuda")
    kd, vd = k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()
    n = torch.full((B,), 4000, dtype=torch.int32, device="cuda")
    want = ref.decode(q[:1, :, 0], _Rows(kd, vd), [4000], lambda b, g, m: ref.windowed(m, 4000, 0, "cuda"), BF16)
    bsa.bsattn_set_wait_budget_ns(0)
    try:
        bsa.bsattn_prefill_window(q, k, v, 1000, 0, ws=ws)
        assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_TIMEOUT
        got = bsa.bsattn_decode_window(q[:, :, 0].contiguous(), kd, vd, n, 4000, 0, ws=ws)
        status = bsa.bsattn_get_device_status(ws)
        if B == 1 and status == 0:
            ref.check(got, *want)
        else:
            assert status == bsa.BSATTN_ERR_TIMEOUT
    finally:
        bsa.bsattn_set_wait_budget_ns(2_000_000_000)
    ws.zero_()
    got = bsa.bsattn_decode_window(q[:, :, 0].contiguous(), kd, vd, n, 4000, 0, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == 0
    ref.check(got[:1], *want)


def test_wait_budget_is_not_the_calls(bsa):
    """A call that takes longer than a wait's budget, with no wait that does: 2.5 ms against 1 ms."""
    q = _rand(4, 32, 16384, 128, dtype=BF16, seed=1)
    k, v = _rand(4, 8, 16384, 128, dtype=BF16, seed=2), _rand(4, 8, 16384, 128, dtype=BF16, seed=3)
    want = bsa.bsattn_prefill_window(q, k, v, 4096, 4)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    bsa.bsattn_set_wait_budget_ns(1_000_000)
    try:
        got = bsa.bsattn_prefill_window(q, k, v, 4096, 4, ws=ws)
        assert bsa.bsattn_get_device_status(ws) == 0
    finally:
        bsa.bsattn_set_wait_budget_ns(2_000_000_000)
    assert torch.equal(got, want)


def test_windows_past_32_bits(bsa):
    """A window or a number of sinks larger than any length is all of it, however it is written."""
    q = _rand(1, 2, 150, 64, dtype=F16, seed=1)
    k, v = _rand(1, 2, 150, 64, dtype=F16, seed=2), _rand(1, 2, 150, 64, dtype=F16, seed=3)
    want = bsa.bsattn_prefill_window(q, k, v, 150, 0)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 32 + 5, 0), (2 ** 40, 2 ** 40), (1, 2 ** 32 + 1)):
        assert torch.equal(want, bsa.bsattn_prefill_window(q, k, v, window, sinks))
    n = torch.tensor([150], dtype=torch.int32, device="cuda")
    args = (q[:, :, -1].contiguous(), k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous(), n)
    want = bsa.bsattn_decode_window(*args, 150, 0)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 32 + 5, 0), (1, 2 ** 32 + 1)):
        assert torch.equal(want, bsa.bsattn_decode_window(*args, window, sinks))
    with pytest.raises(bsa.BsattnError):
        bsa.bsattn_decode_window(*args, -2 ** 40, 0)


def test_in_place_output(bsa):
    """The output may be the queries: every query row is read before its output is written."""
    q = _rand(2, 6, 500, 128, dtype=BF16, seed=1)
    k, v = _rand(2, 3, 700, 128, dtype=BF16, seed=2), _rand(2, 3, 700, 128, dtype=BF16, seed=3)
    want = bsa.bsattn_prefill_window(q, k, v, 100, 3)
    bsa.bsattn_prefill_window(q, k, v, 100, 3, out=q)
    assert torch.equal(q, want)
    lens = [9000, 40]
    kp, vp, table = _paged(lens, 2, 64, BF16, 64, seed=4)
    q = _rand(2, 8, 64, dtype=BF16, seed=5)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = bsa.bsattn_decode_window_paged(q, kp, vp, n, table, 8000, 4)
    bsa.bsattn_decode_window_paged(q, kp, vp, n, table, 8000, 4, out=q)
    assert torch.equal(q, want)


def test_prefill_rows_past_32_bit_offsets(bsa):
    """Batches 2^32 elements apart, heads 2^26, rows 2^20: offsets that only 64 bits hold."""
    shape, stride = (2, 4, 40, 64), (1 << 32, 1 << 26, 1 << 20, 1)
    room = torch.empty((1 << 32) + (1 << 28), dtype=F16, device="cuda")
    q, out = (torch.as_strided(room, shape, stride, at) for at in (0, 128))
    q.copy_(_rand(*shape, dtype=F16, seed=1))
    k, v = _rand(2, 2, 40, 64, dtype=F16, seed=2), _rand(2, 2, 40, 64, dtype=F16, seed=3)
    bsa.bsattn_prefill_window(q, k, v, 9, 1, out=out)
    ref.check(out, *ref.window_prefill(q, k, v, 9, 1))


@pytest.mark.parametrize("big", [2 ** 32 + 64, 2 ** 31, 2 ** 32])
def test_sizes_past_32_bits(bsa, big):
    """Broadcast views whose sizes a C int would cut off."""
    x = torch.zeros(1, 1, 64, 64, dtype=torch.float16, device="cuda")
    one = x[:, :, :1]
    many = one.expand(1, 1, big, 64)
    with pytest.raises(ValueError):
        bsa.bsattn_prefill_window(x, many, many, 100)
    with pytest.raises(ValueError):
        bsa.bsattn_prefill_window(many, x, x, 100, out=many)
    with pytest.raises(ValueError):
        bsa.bsattn_prefill_window(one.expand(big, 1, 1, 64), one.expand(big, 1, 1, 64), one.expand(big, 1, 1, 64), 100,
                                  out=one.expand(big, 1, 1, 64))
