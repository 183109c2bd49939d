"""What the paged-serving calls leave behind: workspaces, status words and outputs after waits that expired,
calls that follow one another, arguments at the edge of what the header allows."""
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F16, BF16 = torch.float16, torch.bfloat16
BUDGET = 2_000_000_000                     # the default
HEADER, TICKETS = 256, 4 * 1024


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


def _decodes(bsa, lens, d=128, Hq=8, Hkv=8):
    """name -> (call(ws=None) over these lengths, workspace size), all over pages in order."""
    B, pages = len(lens), -(-max(lens) // 64)
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    k, v = (_rand(B * pages, 64, Hkv, d, dtype=BF16, seed=s) for s in (1, 2))
    q, n = _rand(B, Hq, d, dtype=BF16, seed=3), _i32(lens)
    cache = bsa.bsattn_kv4_cache(B * pages, Hkv, 64, d)
    bsa.bsattn_kv4_append(k.flatten(0, 1), v.flatten(0, 1), torch.arange(B * pages * 64, device="cuda"), cache)
    flat = [x.view(B, pages * 64, Hkv, d) for x in (k, v)]
    size = bsa.bsattn_decode_window_workspace_size(Hq, Hkv, d)
    return {"paged": (lambda ws=None: bsa.bsattn_decode_window_paged(q, k, v, n, table, max(lens), 0, ws=ws), size),
            "contiguous": (lambda ws=None: bsa.bsattn_decode_window(q, *flat, n, max(lens), 0, ws=ws), size),
            "kv4": (lambda ws=None: bsa.bsattn_decode_paged_kv4(q, cache, n, table, ws=ws),
                    bsa.bsattn_decode_kv4_workspace_size(Hq, Hkv, d))}


@pytest.mark.parametrize("kind", ["paged", "contiguous", "kv4"])
@pytest.mark.parametrize("lens", [[4000] * 64, [9000, 40, 0, 700]])
def test_calls_after_an_expired_wait(bsa, kind, lens):
    """Waits that expire in some CTAs and not in others leave the workspace ready for the next call, the
    binding's own one too; a row is right or NaN in every channel, whatever the budget."""
    call, size = _decodes(bsa, lens)[kind]
    want = call()
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    seen = 0
    try:
        for budget in (0, 200, 500, 1000, 2000, 5000, 20000, 100000):
            bsa.bsattn_set_wait_budget_ns(budget)
            for _ in range(3):
                call()
                got = call(ws)
                status = bsa.bsattn_get_device_status(ws)
                seen |= status
                assert status in (0, bsa.BSATTN_ERR_TIMEOUT)
                assert not ws[HEADER:HEADER + TICKETS].any()
                lost = got.isnan().all(-1)
                assert torch.equal(got[~lost], want[~lost])
                assert status or not lost.any()
    finally:
        bsa.bsattn_set_wait_budget_ns(BUDGET)
    # A first poll may itself last until the data is there, and at 4 bits, where the arithmetic is the longer
    # side, it does; 1 GB of 16-bit rows asked for at once takes longer.
    if len(lens) == 64 and kind != "kv4":
        assert seen
    assert torch.equal(call(), want)
    assert torch.equal(call(ws), want)
    assert bsa.bsattn_get_device_status(ws) == 0


@pytest.mark.parametrize("kind", ["paged", "kv4"])
def test_wait_budget_is_not_the_decodes(bsa, kind):
    """A decode that takes longer than a wait's budget, with no wait that does: 64 sequences of 65536 tokens
    over the pages of four of them, a millisecond or more against a quarter of one."""
    B, Hkv, d, pages = 64, 8, 128, 1024
    k, v = (_rand(4 * pages, 64, Hkv, d, dtype=BF16, seed=s) for s in (1, 2))
    table = torch.arange(4 * pages, dtype=torch.int32, device="cuda").view(4, pages).repeat(B // 4, 1)
    q, n = _rand(B, 32, d, dtype=BF16, seed=3), _i32([64 * pages] * B)
    if kind == "kv4":
        cache = bsa.bsattn_kv4_cache(4 * pages, Hkv, 64, d)
        bsa.bsattn_kv4_append(k.flatten(0, 1), v.flatten(0, 1), torch.arange(4 * pages * 64, device="cuda"), cache)
        size = bsa.bsattn_decode_kv4_workspace_size(32, Hkv, d)
        call = lambda ws: bsa.bsattn_decode_paged_kv4(q, cache, n, table, ws=ws)  # noqa: E731
    else:
        size = bsa.bsattn_decode_window_workspace_size(32, Hkv, d)
        call = lambda ws: bsa.bsattn_decode_window_paged(q, k, v, n, table, 64 * pages, 0, ws=ws)  # noqa: E731
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = call(ws)
    bsa.bsattn_set_wait_budget_ns(250_000)
    try:
        got = call(ws)
        assert bsa.bsattn_get_device_status(ws) == 0
    finally:
        bsa.bsattn_set_wait_budget_ns(BUDGET)
    assert torch.equal(got, want)


def test_status_bits_set_while_the_word_is_read(bsa):
    """Calls on other streams may set bits of a shared word between its reading and its clearing: what one
    reading does not return the next one does."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    word, side = ws.view(torch.int32)[:1], torch.cuda.Stream()
    cached, new, free, count, table = _i32([0]), _i32([5]), _i32([0]), _i32([0]), _i32([[-1]])
    both = bsa.BSATTN_ERR_BAD_INDEX | bsa.BSATTN_ERR_NO_SPACE
    for r in range(400):
        word.fill_(bsa.BSATTN_ERR_BAD_INDEX)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(1 + 400 * r)                  # some time in the 80 us from here on
            bsa.bsattn_paged_plan(cached, new, free, count, table, 64, 5, ws=ws)         # no page for it
        first = bsa.bsattn_get_device_status(ws)
        side.synchronize()
        assert first | bsa.bsattn_get_device_status(ws) == both, f"{first} after {400 * r} cycles"
    assert bsa.bsattn_get_device_status(ws) == 0


@pytest.mark.parametrize("kind", ["plan", "append", "gather", "prefill", "paged", "contiguous", "kv4"])
def test_status_of_captured_calls(bsa, kind):
    """What captured calls without a workspace argument find is read from the device's status word, after
    every replay."""
    dev = torch.device("cuda", torch.cuda.current_device())
    word = bsa.status_workspace(dev)
    bsa.bsattn_get_device_status(word)
    x = _rand(2, 2, 64, dtype=BF16, seed=1)
    cache = bsa.bsattn_kv4_cache(2, 2, 64, 64)
    past = torch.tensor([5, 2 ** 40], device="cuda")        # a slot past the cache
    k, v = _rand(2, 64, 2, 64, dtype=BF16, seed=2), _rand(2, 64, 2, 64, dtype=BF16, seed=3)
    n, table, far = _i32([100, 60]), _i32([[0, 7], [1, 1]]), _i32([100, 60])         # there is no page 7
    p = _rand(64, 8, 4000, 64, dtype=BF16, seed=4)
    calls = {
        "plan": lambda: bsa.bsattn_paged_plan(_zero, _zero, _zero, _zero, _table, 64, 4),
        "append": lambda: bsa.bsattn_kv4_append(x, x, past, cache),
        "gather": lambda: bsa.bsattn_kv4_gather(past, cache, BF16),
        "prefill": lambda: bsa.bsattn_prefill_window(p, p, p, 4000),
        "paged": lambda: bsa.bsattn_decode_window_paged(x, k, v, n, table, 100),
        "contiguous": lambda: bsa.bsattn_decode_window(x, k, v, far, 10),
        "kv4": lambda: bsa.bsattn_decode_paged_kv4(x, cache, n, table),
    }
    _zero, _table = _i32([-1]), _i32([[0]])                 # a negative length
    want = bsa.BSATTN_ERR_TIMEOUT if kind == "prefill" else bsa.BSATTN_ERR_BAD_INDEX
    graph = torch.cuda.CUDAGraph()
    try:
        if kind == "prefill":                               # a budget is taken when the call is made
            bsa.bsattn_set_wait_budget_ns(0)
        with torch.cuda.graph(graph):
            calls[kind]()
    finally:
        bsa.bsattn_set_wait_budget_ns(BUDGET)
    assert bsa.bsattn_get_device_status(word) == 0
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert bsa.bsattn_get_device_status(word) == want
        assert bsa.bsattn_get_device_status(word) == 0


def test_a_workspace_given_to_a_captured_call_has_its_status(bsa):
    x, k = _rand(1, 2, 64, dtype=BF16, seed=1), _rand(1, 64, 2, 64, dtype=BF16, seed=2)
    ws = torch.zeros(bsa.bsattn_decode_window_workspace_size(2, 2, 64), dtype=torch.uint8, device="cuda")
    word, n = bsa.status_workspace(x.device), _i32([65])
    bsa.bsattn_get_device_status(word)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsa.bsattn_decode_window(x, k, k, n, 10, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert bsa.bsattn_get_device_status(word) == 0
    assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX


def _every_call(bsa):
    x, k = _rand(1, 2, 64, dtype=BF16, seed=1), _rand(1, 64, 2, 64, dtype=BF16, seed=2)
    cache, slots, n, table = bsa.bsattn_kv4_cache(1, 2, 64, 64), torch.zeros(1, dtype=torch.int64, device="cuda"), \
        _i32([64]), _i32([[0]])
    return [lambda ws: bsa.bsattn_paged_plan(_i32([0]), _i32([1]), _i32([0]), _i32([1]), _i32([[-1]]), 64, 1, ws=ws),
            lambda ws: bsa.bsattn_kv4_append(x, x, slots, cache, ws=ws),
            lambda ws: bsa.bsattn_kv4_gather(slots, cache, F16, ws=ws),
            lambda ws: bsa.bsattn_prefill_window(k, k, k, 8, ws=ws),
            lambda ws: bsa.bsattn_decode_window(x, k, k, n, 8, ws=ws),
            lambda ws: bsa.bsattn_decode_window_paged(x, k, k, n, table, 8, ws=ws),
            lambda ws: bsa.bsattn_decode_paged_kv4(x, cache, n, table, ws=ws)]


@pytest.mark.parametrize("call", range(7))
def test_workspaces_that_the_kernels_could_not_write_are_refused(bsa, call):
    size = bsa.bsattn_decode_window_workspace_size(2, 2, 64) + bsa.bsattn_decode_kv4_workspace_size(2, 2, 64)
    f = _every_call(bsa)[call]
    for ws in (torch.zeros(size, dtype=torch.uint8),                                      # host memory
               torch.zeros(1, dtype=torch.uint8, device="cuda").expand(size),             # one byte
               torch.zeros(2, size, dtype=torch.uint8, device="cuda").t()):
        with pytest.raises(ValueError):
            f(ws)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    with pytest.raises(bsa.BsattnError):
        f(ws[1:])
    f(ws)
    assert bsa.bsattn_get_device_status(ws) == 0


@pytest.mark.parametrize("T,H,token,head", [(1, 2, 255, None), (3, 1, None, 4), (1, 1, -7, 1)])
def test_append_takes_any_stride_of_a_dimension_of_one(bsa, T, H, token, head):
    d, lib = 64, bsa.load()
    k, v = _rand(T, H, d, dtype=F16, seed=1), _rand(T, H, d, dtype=F16, seed=2)
    slots, ws = torch.arange(T, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    want, got = bsa.bsattn_kv4_cache(1, H, 64, d), bsa.bsattn_kv4_cache(1, H, 64, d)
    bsa.bsattn_kv4_append(k, v, slots, want)
    token, head = H * d if token is None else token, d if head is None else head
    rc = lib.bsattn_kv4_append(k.data_ptr(), v.data_ptr(), token, head, token, head, slots.data_ptr(),
                               *(x.data_ptr() for x in got), 1.0, 1.0, T, H, 1, 64, d, 0, ws.data_ptr(), 256,
                               torch.cuda.current_stream().cuda_stream)
    assert rc == bsa.BSATTN_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("heads", [(4, 2), (3, 3)])
def test_prefill_outputs_between_their_inputs(bsa, heads):
    """Views of one buffer: the queries overwritten in place, and an output in a column of its own."""
    (Hq, Hkv), B, S, d = heads, 2, 300, 64
    fused = _rand(B, S, 2 * Hq + 2 * Hkv, d, dtype=BF16, seed=1)
    q, k, v, out = (x.transpose(1, 2) for x in fused.split((Hq, Hkv, Hkv, Hq), 2))
    want = bsa.bsattn_prefill_window(q.contiguous(), k.contiguous(), v.contiguous(), 100, 3)
    before = fused.clone()
    bsa.bsattn_prefill_window(q, k, v, 100, 3, out=out)
    assert torch.equal(out, want) and torch.equal(fused[:, :, :Hq + 2 * Hkv], before[:, :, :Hq + 2 * Hkv])
    bsa.bsattn_prefill_window(q, k, v, 100, 3, out=q)
    assert torch.equal(q, want) and torch.equal(fused[:, :, Hq:Hq + 2 * Hkv], before[:, :, Hq:Hq + 2 * Hkv])
    with pytest.raises(bsa.BsattnError):
        bsa.bsattn_prefill_window(q, k, v, 100, 3, out=fused[:, :, 1:Hq + 1].transpose(1, 2))
    with pytest.raises(bsa.BsattnError):
        bsa.bsattn_prefill_window(q, k, v, 100, 3, out=fused[:, :, :1].transpose(1, 2).expand(B, Hq, S, d))


@pytest.mark.parametrize("unit,size", [(2.0 ** -16, 2.0 ** 126), (2.0 ** -16, 2.0 ** 127), (2.0 ** -16, 3.3e38),
                                       (2.0 ** -16, -3.3e38), (1.0, 2.0 ** -126), (1.0, 2.0 ** -133),
                                       (2.0 ** 16, 2.0 ** 126), (2.0 ** 16, -3.3e38)])
def test_kv4_decode_queries_of_any_finite_size(bsa, unit, size):
    """bf16 queries up to the type's ends.  Only token 5's key is not 0: with a large query of its sign it takes
    all, with one of the other sign the rest share; a tiny query's scores are 0 to 32 bits, all weights 1."""
    d, n = 64, 9
    cache = bsa.bsattn_kv4_cache(1, 1, 64, d)
    v = _rand(64, 1, d, dtype=BF16, seed=1)
    bsa.bsattn_kv4_append(torch.zeros_like(v), v, torch.arange(64, device="cuda"), cache)
    if unit <= 1:                                                       # above, the score has no 32-bit value
        cache.k_codes[0, 0, 5, 0], cache.k_scales[0, 0, 5, 0] = 2, 1    # 1 * 2^-9 * unit in channel 0
    _, values = bsa.bsattn_kv4_gather(torch.arange(n, device="cuda"), cache, F16)
    q = torch.zeros(1, 1, d, dtype=BF16, device="cuda")
    q[..., 0] = size
    got = bsa.bsattn_decode_paged_kv4(q, cache, _i32([n]), _i32([[0]]), k_scale=unit)[0, 0].double()
    values = values[:, 0].double()
    weight = torch.ones(n, dtype=torch.float64, device="cuda")
    if abs(size) > 1 and unit <= 1:
        weight[torch.arange(n, device="cuda") != 5 if size > 0 else 5] = 0
    want = weight @ values / weight.sum()
    # one rounding to bf16; weights of 2^12 are exact in fp16, sums of n values and one quotient in 32 bits
    bound = torch.finfo(BF16).eps / 2 * want.abs() + (n + 8) * 2.0 ** -23 * (weight @ values.abs()) / weight.sum()
    assert bool(((got - want).abs() <= bound).all())


def test_a_status_word_that_the_caller_has_set_stays_set(bsa):
    x, k, n = _rand(1, 2, 64, dtype=BF16, seed=1), _rand(1, 64, 2, 64, dtype=BF16, seed=2), _i32([65])
    default, mine = bsa.status_workspace(x.device), torch.zeros(256, dtype=torch.uint8, device="cuda")
    bsa.bsattn_get_device_status(default)
    graph = torch.cuda.CUDAGraph()
    bsa.bsattn_set_status_word(mine)
    try:
        with torch.cuda.graph(graph):
            bsa.bsattn_decode_window(x, k, k, n, 10)
        graph.replay()
        assert bsa.bsattn_get_device_status(mine) == bsa.BSATTN_ERR_BAD_INDEX
        bsa.bsattn_decode_window(x, k, k, n, 10)
        assert bsa.bsattn_get_device_status(mine) == bsa.BSATTN_ERR_BAD_INDEX
    finally:
        bsa.bsattn_set_status_word(None)
    assert bsa.bsattn_get_device_status(default) == 0
    ws = torch.zeros(bsa.bsattn_decode_window_workspace_size(2, 2, 64), dtype=torch.uint8, device="cuda")
    bsa.bsattn_decode_window(x, k, k, n, 10, ws=ws)
    assert bsa.bsattn_get_device_status(ws) == bsa.BSATTN_ERR_BAD_INDEX
    assert bsa.bsattn_get_device_status(mine) == 0
