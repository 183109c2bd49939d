"""Argument checks of the paged-serving entry points: they fail before anything is launched."""
import ctypes

import pytest
import torch

import block_sparse_attention_gb300 as bsa

X = 1 << 12          # an aligned address that is never read
INVALID, UNSUPPORTED = bsa.BSATTN_ERR_INVALID_ARG, bsa.BSATTN_ERR_UNSUPPORTED


def _plan(**kw):
    a = dict(cached=X, new=2 * X, free=3 * X, count=4 * X, table=5 * X, slots=6 * X, starts=7 * X, lens=8 * X,
             left=9 * X, B=4, page=64, max_pages=8, cap=16, tokens=8, ws=10 * X, wsb=256, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return bsa.load().bsattn_paged_plan(*a.values())


@pytest.mark.parametrize("kw", [dict(B=-1), dict(page=0), dict(max_pages=0), dict(cap=-1), dict(tokens=-1),
                                dict(ws=None), dict(wsb=16), dict(cached=None), dict(new=None), dict(free=None),
                                dict(count=None), dict(table=None), dict(slots=None), dict(starts=None),
                                dict(lens=None), dict(left=None),
                                dict(lens=X),              # new lengths over the old ones
                                dict(left=4 * X),          # the count over itself
                                dict(starts=8 * X),        # two outputs in one place
                                dict(table=3 * X)])
def test_plan_refuses(kw):
    assert _plan(**kw) == INVALID


def test_plan_refuses_more_sequences_than_it_scans():
    assert _plan(B=8193, cached=X, new=X << 8, free=X << 9, count=X << 10, table=X << 11, slots=X << 13,
                 starts=X << 14, lens=X << 15, left=X << 16) == UNSUPPORTED


def _append(**kw):
    a = dict(k=X, v=X, kt=256, kh=128, vt=256, vh=128, slots=X, kc=X, ks=X, vc=X, vs=X, ku=1.0, vu=1.0, T=3,
             Hkv=2, pages=4, page=64, d=128, dtype=1, ws=X, wsb=256, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return bsa.load().bsattn_kv4_append(*a.values())


def _gather(**kw):
    a = dict(slots=X, kc=X, ks=X, vc=X, vs=X, ku=1.0, vu=1.0, k=X, v=X, T=3, Hkv=2, pages=4, page=64, d=128,
             dtype=1, ws=X, wsb=256, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return bsa.load().bsattn_kv4_gather(*a.values())


@pytest.mark.parametrize("call", [_append, _gather])
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(Hkv=0), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(ku=0.0), INVALID), (dict(vu=-1.0), INVALID),
    (dict(ku=3.0), INVALID), (dict(vu=float("nan")), INVALID), (dict(ku=float("inf")), INVALID),
    (dict(vu=2.0 ** 17), INVALID), (dict(ws=None), INVALID), (dict(wsb=8), INVALID), (dict(slots=None), INVALID),
    (dict(k=None), INVALID), (dict(kc=X + 8), INVALID), (dict(vs=X + 4), INVALID), (dict(k=X + 2), INVALID),
    (dict(T=0), bsa.BSATTN_OK)])
def test_kv4_rows_refuse(call, kw, want):
    assert call(**kw) == want


@pytest.mark.parametrize("kw", [dict(kt=255), dict(kh=4), dict(vt=130), dict(vh=1)])
def test_append_refuses_unaligned_strides(kw):
    assert _append(**kw) == INVALID


def _kv4(**kw):
    a = dict(q=X, kc=X, ks=X, vc=X, vs=X, ku=1.0, vu=1.0, lens=X, idx=None, table=X, window=0, sinks=0, out=X,
             B=1, Hq=8, Hkv=2, pages=4, page=64, max_pages=4, d=128, max_sel=0, dtype=1, ws=X, wsb=1 << 30,
             stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return bsa.load().bsattn_decode_paged_kv4(*a.values())


def _paged(**kw):
    a = dict(q=X, k=X, v=X, lens=X, table=X, window=8, sinks=0, out=X, B=1, Hq=8, Hkv=2, pages=4, page=64,
             max_pages=4, d=128, dtype=1, ws=X, wsb=1 << 30, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return bsa.load().bsattn_decode_window_paged(*a.values())


def _window(**kw):
    a = dict(q=X, k=X, v=X, lens=X, window=8, sinks=0, out=X, B=1, Hq=8, Hkv=2, Smax=64, d=128, dtype=1, ws=X,
             wsb=1 << 30, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return bsa.load().bsattn_decode_window(*a.values())


@pytest.mark.parametrize("call", [_kv4, _paged, _window])
@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=7), INVALID),
    (dict(Hq=18), UNSUPPORTED), (dict(d=80), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(lens=None), INVALID),
    (dict(q=X + 2), INVALID), (dict(out=X + 8), INVALID), (dict(ws=None), INVALID), (dict(wsb=300), INVALID),
    (dict(Hkv=1025, Hq=1025), UNSUPPORTED), (dict(B=0), bsa.BSATTN_OK)])
def test_stream_decodes_refuse(call, kw, want):
    assert call(**kw) == want


@pytest.mark.parametrize("call", [_kv4, _paged])
@pytest.mark.parametrize("kw,want", [(dict(page=0), INVALID), (dict(page=48), UNSUPPORTED), (dict(pages=0), INVALID),
                                     (dict(max_pages=0), INVALID), (dict(table=None), INVALID)])
def test_paged_decodes_refuse(call, kw, want):
    assert call(**kw) == want


def test_decodes_refuse_what_only_they_take():
    assert _kv4(idx=X, max_sel=3, window=5) == INVALID           # two rules of visibility
    assert _kv4(idx=X, max_sel=-1) == INVALID
    assert _kv4(ku=1.5) == INVALID and _kv4(vu=0.0) == INVALID
    assert _kv4(kc=None) == INVALID and _kv4(vs=X + 8) == INVALID
    assert _paged(window=0) == INVALID and _window(window=0) == INVALID
    assert _paged(k=None) == INVALID and _paged(v=X + 8) == INVALID
    assert _window(Smax=-1) == INVALID and _window(k=None) == INVALID
    assert _paged(pages=1 << 20, page=1 << 12) == UNSUPPORTED     # rows past 32 bits
    assert _window(B=1 << 16, Smax=1 << 16) == UNSUPPORTED


def _prefill(strides=None, **kw):
    a = dict(q=X, k=X, v=X, window=8, sinks=0, out=X, B=1, Hq=4, Hkv=2, Sq=64, Sk=64, d=128, strides=None, dtype=1,
             ws=X, wsb=256, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    if strides is not None:
        a["strides"] = (ctypes.c_int64 * 12)(*strides)
    return bsa.load().bsattn_prefill_window(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID), (dict(Sq=-1), INVALID),
    (dict(Sk=-1), INVALID), (dict(window=0), INVALID), (dict(sinks=-1), INVALID), (dict(d=256), UNSUPPORTED),
    (dict(dtype=7), UNSUPPORTED), (dict(ws=None), INVALID), (dict(wsb=4), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(out=X + 8), INVALID), (dict(v=X + 2), INVALID), (dict(B=0), bsa.BSATTN_OK),
    (dict(Sq=0), bsa.BSATTN_OK), (dict(Sq=(1 << 30) + 1), UNSUPPORTED)])
def test_prefill_window_refuses(kw, want):
    assert _prefill(**kw) == want


@pytest.mark.parametrize("at,value", [(1, 0), (2, 0), (2, 132), (5, -128), (8, 4), (10, 0), (11, 0), (11, 130)])
def test_prefill_window_refuses_strides(at, value):
    dense = [4 * 64 * 128, 64 * 128, 128, 2 * 64 * 128, 64 * 128, 128, 2 * 64 * 128, 64 * 128, 128,
             4 * 64 * 128, 64 * 128, 128]
    dense[at] = value
    assert _prefill(strides=dense) == INVALID


def test_workspace_sizes():
    small, big = bsa.bsattn_decode_window_workspace_size(8, 8, 128), bsa.bsattn_decode_window_workspace_size(64, 8, 128)
    assert 256 + 4096 < small < big
    assert bsa.bsattn_decode_kv4_workspace_size(64, 8, 128) > 256 + 4096
    assert bsa.bsattn_decode_kv4_workspace_size(0, 8, 128) == 256


def test_status_of_a_plan_without_space_has_a_name():
    assert bsa.bsattn_status_string(bsa.BSATTN_ERR_NO_SPACE | bsa.BSATTN_ERR_BAD_INDEX) == \
        "BSATTN_ERR_BAD_INDEX|BSATTN_ERR_NO_SPACE"


def test_binding_refuses_host_tensors():
    q = torch.zeros(1, 2, 3, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        bsa.bsattn_prefill_window(q, q, q, 4)
    with pytest.raises(ValueError):
        bsa.bsattn_decode_window(q[0], q, q, torch.zeros(1, dtype=torch.int32), 4)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        bsa.bsattn_paged_plan(i, i, i, i, i[None], 64, 8)
    cache = bsa.bsattn_kv4_cache(1, 2, 64, 64, device="cpu")
    with pytest.raises(ValueError):
        bsa.bsattn_kv4_append(q[0], q[0], torch.zeros(2, dtype=torch.int64), cache)
