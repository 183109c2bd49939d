"""Argument checks of the block-choosing calls and the shared-prefix decode: they fail before anything is launched."""
import ctypes

import pytest
import torch

import block_sparse_attention_gb300 as bsa

X = 1 << 30          # an aligned address that is never read
OK, INVALID, UNSUPPORTED = bsa.BSATTN_OK, bsa.BSATTN_ERR_INVALID_ARG, bsa.BSATTN_ERR_UNSUPPORTED


def _call(name, **kw):
    args = {
        "update": dict(k=X, lens=2 * X, new=3 * X, table=4 * X, codes=5 * X, scales=6 * X, B=4, Hkv=2, pages=8, page=64,
                       max_pages=4, d=128, dtype=1, ws=7 * X, wsb=256, stream=None),
        "select": dict(q=X, codes=2 * X, scales=3 * X, lens=4 * X, table=5 * X, sinks=1, recent=1, out=6 * X, B=4, Hq=8,
                       Hkv=2, pages=8, page=64, max_pages=4, d=128, max_sel=4, dtype=1, ws=7 * X, wsb=256, stream=None),
        "mask": dict(q=X, k=2 * X, topk=4, sinks=1, recent=1, dense=0, causal=1, out=3 * X, B=2, Hq=4, Hkv=2, Sq=200,
                     Sk=300, d=128, strides=None, dtype=1, ws=4 * X, wsb=1 << 24, stream=None),
        "shared": dict(q=X, k=2 * X, v=3 * X, plens=4 * X, ptable=5 * X, starts=6 * X, lens=7 * X, table=8 * X,
                       out=9 * X, B=4, P=1, Hq=8, Hkv=2, pages=8, page=64, max_prefix=4, max_pages=4, d=128, dtype=1,
                       ws=10 * X, wsb=1 << 28, stream=None),
    }[name]
    assert not set(kw) - set(args)
    args.update(kw)
    if args.get("strides") is not None:
        args["strides"] = (ctypes.c_int64 * 6)(*args["strides"])
    f = {"update": "bsattn_index_update", "select": "bsattn_decode_select", "mask": "bsattn_mask_from_qk",
         "shared": "bsattn_decode_shared"}[name]
    return getattr(bsa.load(), f)(*args.values())


@pytest.mark.parametrize("kw", [dict(B=-1), dict(Hkv=0), dict(pages=0), dict(page=0), dict(max_pages=0), dict(k=None),
                                dict(lens=None), dict(new=None), dict(table=None), dict(codes=None), dict(scales=None),
                                dict(ws=None), dict(wsb=8), dict(ws=7 * X + 8), dict(k=X + 2), dict(codes=5 * X + 8),
                                dict(scales=6 * X + 4),
                                dict(codes=X), dict(codes=6 * X), dict(scales=5 * X + 256), dict(codes=2 * X),
                                dict(scales=4 * X)])
def test_update_refuses(kw):
    assert _call("update", **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(page=96), dict(d=96), dict(dtype=2), dict(pages=1 << 26)])
def test_update_does_not_support(kw):
    assert _call("update", **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(pages=0), dict(page=0),
                                dict(max_pages=0), dict(max_sel=0), dict(max_sel=-1), dict(sinks=-1), dict(recent=-1),
                                dict(sinks=3, recent=2), dict(recent=5), dict(sinks=2 ** 31 - 1),
                                dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(q=None), dict(codes=None),
                                dict(scales=None), dict(lens=None), dict(table=None), dict(out=None), dict(ws=None),
                                dict(wsb=255), dict(ws=7 * X + 4), dict(q=X + 8), dict(codes=2 * X + 1), dict(scales=3 * X + 4),
                                dict(out=X), dict(out=2 * X + 64), dict(out=3 * X), dict(out=4 * X), dict(out=5 * X + 4)])
def test_select_refuses(kw):
    assert _call("select", **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(Hq=18), dict(page=32), dict(d=32), dict(dtype=-1), dict(max_pages=46876),
                                dict(page=128, max_pages=23438), dict(max_sel=1 << 27)])
def test_select_does_not_support(kw):
    assert _call("select", **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(Sq=-1), dict(Sk=-1), dict(topk=-1),
                                dict(sinks=-1), dict(recent=-1), dict(q=None), dict(k=None), dict(out=None), dict(ws=None),
                                dict(wsb=256), dict(ws=4 * X + 8), dict(q=X + 8), dict(k=2 * X + 2), dict(out=X),
                                dict(out=2 * X + 100), dict(out=4 * X + 300), dict(ws=X), dict(ws=2 * X),
                                dict(strides=[102400, 25600, 127, 76800, 38400, 128]),
                                dict(strides=[102400, 25600, -128, 76800, 38400, 128]),
                                dict(strides=[102400, 25600, 128, 76800, 4, 128]),
                                # the last head of the second prompt lies over the mask
                                dict(strides=[X - (3 * 25600 + 199 * 128 + 128) + 8, 25600, 128, 76800, 38400, 128],
                                     out=3 * X)])
def test_mask_refuses(kw):
    assert _call("mask", **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(d=96), dict(dtype=2), dict(Sk=450561), dict(Sq=(1 << 30) + 1)])
def test_mask_does_not_support(kw):
    assert _call("mask", wsb=1 << 40, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(B=-1), dict(P=0), dict(P=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(pages=0),
                                dict(page=0), dict(max_prefix=0), dict(max_pages=0), dict(q=None), dict(k=None),
                                dict(v=None), dict(plens=None), dict(ptable=None), dict(starts=None), dict(lens=None),
                                dict(table=None), dict(out=None), dict(ws=None), dict(wsb=1 << 12), dict(ws=10 * X + 8),
                                dict(q=X + 8), dict(out=9 * X + 2), dict(k=2 * X + 8), dict(v=3 * X + 4),
                                dict(out=X + 256), dict(out=2 * X), dict(out=3 * X + 64)])
def test_shared_refuses(kw):
    assert _call("shared", **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(Hq=18), dict(page=96), dict(d=32), dict(dtype=2), dict(pages=1 << 25),
                                dict(Hq=1025, Hkv=1025), dict(B=1 << 29), dict(P=(1 << 24) + 1)])
def test_shared_does_not_support(kw):
    assert _call("shared", wsb=1 << 40, **kw) == UNSUPPORTED


def test_nothing_to_do():
    assert _call("update", B=0) == OK and _call("select", B=0) == OK and _call("shared", B=0) == OK
    assert _call("mask", B=0) == OK and _call("mask", Sq=0) == OK and _call("mask", Sk=0) == OK


def test_workspace_sizes_grow_with_the_work():
    size = bsa.bsattn_decode_shared_workspace_size
    assert size(4, 1, 32, 8, 128) < size(64, 1, 32, 8, 128) < size(2048, 1, 32, 8, 128)
    assert size(4, 1, 32, 8, 64) < size(4, 1, 32, 8, 128)
    assert size(0, 1, 32, 8, 128) == 256
    mask = bsa.bsattn_mask_from_qk_workspace_size
    assert mask(1, 8, 8, 64, 64, 128) < mask(1, 8, 8, 65, 64, 128) <= mask(1, 8, 8, 65, 6400, 128)
    assert mask(0, 8, 8, 64, 64, 128) == mask(1, 8, 8, 0, 64, 128) == 256


def test_binding_wants_cuda_tensors():
    q, lens, table = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    pages = torch.zeros(3, 64, 2, 64, dtype=torch.float16)
    index = bsa.bsattn_block_index(3, 2, 64, 64, device="cpu")
    with pytest.raises(ValueError):
        bsa.bsattn_index_update(pages, lens, lens, table, index)
    with pytest.raises(ValueError):
        bsa.bsattn_decode_select(q, index, lens, table, 4)
    with pytest.raises(ValueError):
        bsa.bsattn_mask_from_qk(q[None], q[None], 4, True)
    with pytest.raises(ValueError):
        bsa.bsattn_decode_shared(q, pages, pages, lens[:1], table[:1], lens, lens, table)
    with pytest.raises(ValueError):
        bsa.bsattn_block_index(3, 2, 96, 64, device="cpu")


def test_reference_choice():
    """The rule itself, worked by hand."""
    import selection_reference as ref
    assert ref.choice([3.0, 1.0, 3.0, 2.0], [True] * 4, set(), 2) == [0, 2]
    assert ref.choice([3.0, 3.0, 3.0, 3.0], [True] * 4, {3}, 2) == [0, 3]
    assert ref.choice([3.0, 9.0, 3.0, 3.0], [True, False, True, True], {1, 3}, 2) == [0, 3]
    assert ref.choice([1.0, 2.0], [True] * 2, {0, 1}, 1) == [0, 1]
    codes, scale = ref.summary(torch.tensor([[1.0, -2.0], [3.0, -6.0]]))
    assert codes.tolist() == [64.0, -127.0] and scale == torch.tensor(4.0 / 127).double()      # 63.5 to even
    assert ref.quantise(torch.tensor([float("inf"), 1.0]).double())[1] == float("inf")


def test_workspace_sizes_of_lengths_near_32_bits():
    most = 2 ** 31 - 1
    mask = bsa.bsattn_mask_from_qk_workspace_size
    assert mask(1, 1, 1, 1 << 30, 64, 64) < mask(1, 1, 1, most - 63, 64, 64) <= mask(1, 1, 1, most, 64, 64) < 1 << 33
    assert mask(1, 1, 1, 64, 1 << 30, 64) < mask(1, 1, 1, 64, most - 63, 64) <= mask(1, 1, 1, 64, most, 64) < 1 << 33
