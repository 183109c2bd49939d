"""More argument checks of the paged-serving entry points: what they must not launch a kernel for."""
import ctypes

import pytest

import block_sparse_attention_gb300 as bsa

X = 1 << 20          # an aligned address that is never read
INVALID = bsa.BSATTN_ERR_INVALID_ARG


def _call(name, **kw):
    """An entry point's return value with addresses that are never read, but for what kw changes."""
    lib = bsa.load()
    args = {
        "plan": dict(cached=X, new=2 * X, free=3 * X, count=4 * X, table=5 * X, slots=6 * X, starts=7 * X, lens=8 * X,
                     left=9 * X, B=4, page=64, max_pages=8, cap=16, tokens=8, ws=10 * X, wsb=256, stream=None),
        "append": dict(k=X, v=2 * X, kt=256, kh=128, vt=256, vh=128, slots=3 * X, kc=4 * X, ks=5 * X, vc=6 * X,
                       vs=7 * X, ku=1.0, vu=1.0, T=3, Hkv=2, pages=4, page=64, d=128, dtype=1, ws=8 * X, wsb=256,
                       stream=None),
        "gather": dict(slots=X, kc=2 * X, ks=3 * X, vc=4 * X, vs=5 * X, ku=1.0, vu=1.0, k=6 * X, v=7 * X, T=3, Hkv=2,
                       pages=4, page=64, d=128, dtype=1, ws=8 * X, wsb=256, stream=None),
        "prefill": dict(q=X, k=2 * X, v=3 * X, window=8, sinks=0, out=4 * X, B=2, Hq=4, Hkv=2, Sq=64, Sk=64, d=128,
                        strides=None, dtype=1, ws=5 * X, wsb=256, stream=None),
        "kv4": dict(q=X, kc=2 * X, ks=3 * X, vc=4 * X, vs=5 * X, ku=1.0, vu=1.0, lens=6 * X, idx=None, table=7 * X,
                    window=0, sinks=0, out=8 * X, B=1, Hq=8, Hkv=2, pages=4, page=64, max_pages=4, d=128, max_sel=0,
                    dtype=1, ws=9 * X, wsb=1 << 30, stream=None),
        "paged": dict(q=X, k=2 * X, v=3 * X, lens=4 * X, table=5 * X, window=8, sinks=0, out=6 * X, B=1, Hq=8, Hkv=2,
                      pages=4, page=64, max_pages=4, d=128, dtype=1, ws=7 * X, wsb=1 << 30, stream=None),
        "contiguous": dict(q=X, k=2 * X, v=3 * X, lens=4 * X, window=8, sinks=0, out=5 * X, B=1, Hq=8, Hkv=2, Smax=64,
                           d=128, dtype=1, ws=6 * X, wsb=1 << 30, stream=None),
    }[name]
    assert not set(kw) - set(args)
    args.update(kw)
    if args.get("strides") is not None:
        args["strides"] = (ctypes.c_int64 * 12)(*args["strides"])
    f = {"plan": lib.bsattn_paged_plan, "append": lib.bsattn_kv4_append, "gather": lib.bsattn_kv4_gather,
         "prefill": lib.bsattn_prefill_window, "kv4": lib.bsattn_decode_paged_kv4,
         "paged": lib.bsattn_decode_window_paged, "contiguous": lib.bsattn_decode_window}[name]
    return f(*args.values())


@pytest.mark.parametrize("name", ["plan", "append", "gather", "prefill", "kv4", "paged", "contiguous"])
@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_workspace_alignment(name, off):
    """A status word at an odd address would be a misaligned atomic once a bit is set."""
    assert _call(name, ws=40 * X + off) == INVALID


@pytest.mark.parametrize("off", [1, 4, 8])
def test_status_word_alignment(off):
    lib = bsa.load()
    assert lib.bsattn_set_status_word(X + off) == INVALID
    assert lib.bsattn_set_status_word(None) == bsa.BSATTN_OK


def _strides(*tensors):
    return [s for t in tensors for s in t]


# [2, 4 or 2, 64, 128] dense, as the entry point's own layout
Q, KV = (4 * 64 * 128, 64 * 128, 128), (2 * 64 * 128, 64 * 128, 128)
ROWS_FIRST = (4 * 64 * 128, 128, 4 * 128)                     # [B, S, H, d] seen as [B, H, S, d]
Q_BYTES, KV_BYTES = 2 * 2 * 4 * 64 * 128, 2 * 2 * 2 * 64 * 128


@pytest.mark.parametrize("out", [
    (4 * 64 * 128, 128, 128),                                  # a head's rows over the next head's
    (4 * 64 * 128, 64 * 128 - 128, 128),                       # the last row of a head over the next one's first
    (128, 64 * 128, 128),                                      # batches over rows
    (4 * 64 * 128, 160, 2 * 160 + 64),                         # heads 0 and 2 a row apart, over each other
])
def test_prefill_window_refuses_an_output_over_itself(out):
    assert _call("prefill", strides=_strides(Q, KV, KV, out)) == INVALID


@pytest.mark.parametrize("kw", [
    dict(out=2 * X), dict(out=3 * X),                          # k, v
    dict(out=2 * X + KV_BYTES - 16), dict(out=3 * X - Q_BYTES + 16),       # by 16 bytes
    dict(out=X + 256), dict(out=X - 16),                       # q, not where it is
    dict(out=X, strides=_strides(Q, KV, KV, ROWS_FIRST)),      # q in another order
    dict(out=2 * X + 64 * 128 * 2 * 2, strides=_strides(Q, (4 * 64 * 128, 64 * 128, 128), KV, Q)),
    dict(B=1, Hq=1, Hkv=1, Sq=1, Sk=1, out=3 * X + 128),
])
def test_prefill_window_refuses_an_output_over_its_inputs(kw):
    assert _call("prefill", **kw) == INVALID


@pytest.mark.parametrize("name", ["kv4", "paged", "contiguous"])
@pytest.mark.parametrize("tensor,off", [("q", 256), ("q", -16), ("k", 0), ("v", 0), ("k", -16), ("v", 16384 - 16)])
def test_stream_decodes_refuse_an_output_over_their_inputs(name, tensor, off):
    """Another CTA may still read what one has overwritten; only q itself is read before it is."""
    at = dict(q=X, k=2 * X, v=4 * X if name == "kv4" else 3 * X)[tensor]
    assert _call(name, B=4, out=at + off) == INVALID


def test_kv4_decode_refuses_an_output_over_its_scales():
    assert _call("kv4", out=3 * X) == INVALID and _call("kv4", out=5 * X + 64) == INVALID
