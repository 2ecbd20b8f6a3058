"""Refusals of the calls on the cache in 8 bits and on drafted trees, before anything is enqueued (no
GPU needed), and the cases' own quantiser."""
import ctypes
import math

import pytest
import torch

from quantized_routed_expert_02_gb300 import moeq4k as m
from tests.cache_cases import quantised, visible
from tests.test_abi_attention_half import BAD_BATCH, BATCH
from tests.test_abi_host import ALIGNED, lib  # noqa: F401

P, S, F, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float, ctypes.c_int  # noqa: E741
OK, SHAPE, NULL, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
CHECK_ONLY = ctypes.c_void_p(-1)
INF, NAN = float("inf"), float("nan")
WS = 48 << 20


def append(lib, qkv=ALIGNED, pos=ALIGNED, freq=ALIGNED, axis=None, axes=1, rot=64, qw=None, kw=None, eps=1e-6,
           q_out=ALIGNED, k=ALIGNED, v=ALIGNED, ks=ALIGNED, vs=ALIGNED, table=ALIGNED, offs=ALIGNED, lens=ALIGNED,
           ws=ALIGNED, ws_bytes=256, **b):
    b = BATCH | b
    lib.moe_rope_append_q8.restype = I
    return lib.moe_rope_append_q8(P(qkv), P(pos), P(freq), P(axis), I(axes), I(rot), I(0), P(qw), P(kw), F(eps),
                                  P(q_out), P(k), P(v), P(ks), P(vs), P(table), P(offs), P(lens), I(b["N"]), I(b["B"]),
                                  I(b["max_pages"]), I(b["num_pages"]), I(b["page"]), I(b["Hq"]), I(b["Hkv"]),
                                  I(b["D"]), I(b["dtype"]), P(ws), S(ws_bytes), CHECK_ONLY)


def attn(lib, q=ALIGNED, k=ALIGNED, v=ALIGNED, ks=ALIGNED, vs=ALIGNED, table=ALIGNED, offs=ALIGNED, lens=ALIGNED,
         tree=None, words=0, most=1, scale=0.1, cap=0.0, window=0, sinks=0, out=ALIGNED, lse=None, ws=ALIGNED,
         ws_bytes=WS, **b):
    b = BATCH | b
    lib.moe_attention_cache.restype = I
    return lib.moe_attention_cache(P(q), P(k), P(v), P(ks), P(vs), P(table), P(offs), P(lens), P(tree), I(words),
                                   I(b["N"]), I(b["B"]), I(most), I(b["max_pages"]), I(b["num_pages"]), I(b["page"]),
                                   I(b["Hq"]), I(b["Hkv"]), I(b["D"]), I(b["dtype"]), F(scale), F(cap), I(window),
                                   I(sinks), P(out), P(lse), P(ws), S(ws_bytes), CHECK_ONLY)


def keep(lib, k=ALIGNED, v=ALIGNED, ks=None, vs=None, table=ALIGNED, offs=ALIGNED, lens=ALIGNED, keep=ALIGNED,
         kept=ALIGNED, most=5, elem=2, ws=ALIGNED, ws_bytes=256, **b):
    b = BATCH | b
    lib.moe_cache_keep.restype = I
    return lib.moe_cache_keep(P(k), P(v), P(ks), P(vs), P(table), P(offs), P(lens), P(keep), P(kept), I(b["B"]),
                              I(most), I(b["max_pages"]), I(b["num_pages"]), I(b["page"]), I(b["Hkv"]), I(b["D"]),
                              I(elem), P(ws), S(ws_bytes), CHECK_ONLY)


@pytest.mark.parametrize("bad", [{}] + BAD_BATCH + [
    dict(axes=0), dict(axes=9), dict(rot=0), dict(rot=8), dict(rot=40), dict(rot=144), dict(rot=128, D=64),
    dict(eps=-1.0), dict(eps=NAN)])
def test_append_shapes(lib, bad):
    assert append(lib, **bad) == (SHAPE if bad else OK)


def test_append_pointers(lib):
    for name in ("qkv", "pos", "freq", "q_out", "k", "v", "ks", "vs", "table", "offs", "lens", "ws"):
        assert append(lib, **{name: 0}) == NULL, name
        step = {"pos": 2, "table": 2, "offs": 2, "lens": 2, "freq": 4, "ws": 128}.get(name, 8)
        assert append(lib, **{name: ALIGNED + step}) == MISALIGNED, name
    assert append(lib, ws_bytes=255) == WORKSPACE


@pytest.mark.parametrize("bad", [{}] + BAD_BATCH + [
    dict(most=0), dict(window=-1), dict(sinks=-1), dict(scale=NAN), dict(scale=INF), dict(cap=-1.0), dict(cap=INF),
    dict(cap=1e-39, scale=3e5), dict(words=1), dict(tree=ALIGNED), dict(tree=ALIGNED, words=33),
    dict(tree=ALIGNED, words=-1)])
def test_attention_shapes(lib, bad):
    for scales in ({}, dict(ks=None, vs=None)):
        assert attn(lib, **bad, **scales) == (SHAPE if bad else OK)


def test_attention_pointers(lib):
    for name in ("q", "k", "v", "table", "offs", "lens", "out", "ws", "ks", "vs"):
        assert attn(lib, **{name: 0}) == NULL, name  # of the scales one alone
    for name in ("q", "k", "v", "out", "ks", "vs"):
        assert attn(lib, **{name: ALIGNED + 8}) == MISALIGNED, name
    assert attn(lib, tree=ALIGNED + 2, words=1) == MISALIGNED and attn(lib, lse=ALIGNED + 2) == MISALIGNED
    assert attn(lib, ws=ALIGNED + 128) == MISALIGNED and attn(lib, ws_bytes=1 << 16) == WORKSPACE
    assert attn(lib, tree=ALIGNED, words=32, sinks=2 ** 31 - 1, window=2 ** 31 - 1) == OK


@pytest.mark.parametrize("bad", [{}, dict(B=0), dict(B=4097), dict(max_pages=0), dict(num_pages=0), dict(page=24),
                                 dict(Hkv=0), dict(Hkv=257), dict(D=96), dict(most=0), dict(most=(1 << 20) + 1),
                                 dict(elem=4), dict(elem=0), dict(num_pages=1 << 30), dict(max_pages=1 << 27)])
def test_keep_shapes(lib, bad):
    assert keep(lib, **bad) == (SHAPE if bad else OK)
    if "elem" not in bad:
        assert keep(lib, **bad, elem=1, ks=ALIGNED, vs=ALIGNED) == (SHAPE if bad else OK)


def test_keep_pointers(lib):
    for name in ("k", "v", "table", "offs", "lens", "keep", "kept", "ws"):
        assert keep(lib, **{name: 0}) == NULL, name
    assert keep(lib, ks=ALIGNED, vs=ALIGNED) == NULL  # 16-bit values have no scales
    assert keep(lib, elem=1) == NULL and keep(lib, elem=1, ks=ALIGNED) == NULL
    assert keep(lib, elem=1, ks=ALIGNED, vs=ALIGNED + 4) == MISALIGNED
    assert keep(lib, k=ALIGNED + 8) == MISALIGNED and keep(lib, ws_bytes=128) == WORKSPACE


# --------------------------------------------------------------------------
# the native module
# --------------------------------------------------------------------------
F16, BF16, I32, I8 = torch.float16, torch.bfloat16, torch.int32, torch.int8


def aligned_bytes(n):
    t = torch.zeros(n + 256, dtype=torch.uint8)
    at = -t.data_ptr() % 256
    return t[at:at + n]


def batch_args():
    return dict(page_table=torch.zeros(1, 2, dtype=I32), q_offs=torch.tensor([0, 3], dtype=I32),
                kv_lens=torch.tensor([5], dtype=I32), ws=aligned_bytes(WS), stream=0)


def codes(names):
    return {n: torch.zeros(4, 2, 16, 64, dtype=I8) for n in names} | {n: torch.zeros(4, 2, 16) for n in
                                                                     ("k_scales", "v_scales")}


def append_args():
    return dict(batch_args(), **codes(("k_codes", "v_codes")), qkv=torch.zeros(3, 8 * 64, dtype=F16),
                pos=torch.zeros(1, 3, dtype=I32), inv_freq=torch.zeros(16, dtype=torch.float64),
                q_out=torch.zeros(3, 4, 64, dtype=F16), axis=torch.zeros(16, dtype=I32), q_norm_w=torch.zeros(64),
                k_norm_w=torch.zeros(64))


def attn_args():
    return dict(batch_args(), **codes(("k_pages", "v_pages")), q=torch.zeros(3, 4, 64, dtype=BF16), max_new=3,
                scale=0.125, out=torch.zeros(3, 4, 64, dtype=BF16), lse=torch.zeros(3, 4), window=4, sinks=1,
                tree=torch.zeros(3, 1, dtype=I32))


def attn16_args():
    return dict(attn_args(), k_pages=torch.zeros(4, 2, 16, 64, dtype=BF16), k_scales=None, v_scales=None,
                v_pages=torch.zeros(4, 2, 16, 64, dtype=BF16))


def keep_args():
    return dict(batch_args(), **codes(("k_pages", "v_pages")), keep=torch.zeros(1, 7, dtype=I32),
                kept=torch.zeros(1, dtype=I32))


def keep16_args():
    return dict(keep_args(), k_pages=torch.zeros(4, 2, 16, 64, dtype=F16), k_scales=None, v_scales=None,
                v_pages=torch.zeros(4, 2, 16, 64, dtype=F16))


CALLS = {"append": (append_args, "moe_rope_append_q8"), "attn": (attn_args, "moe_attention_cache"),
         "attn16": (attn16_args, "moe_attention_cache"), "keep": (keep_args, "moe_cache_keep"),
         "keep16": (keep16_args, "moe_cache_keep")}
BAD = [
    ("append", "qkv", torch.zeros(3, 7 * 64, dtype=F16), ValueError),
    ("append", "qkv", torch.zeros(3, 8 * 64), TypeError),
    ("append", "qkv", None, TypeError),
    ("append", "q_out", torch.zeros(3, 4, 64, dtype=BF16), TypeError),
    ("append", "k_codes", torch.zeros(4, 2, 16, 64, dtype=F16), TypeError),
    ("append", "k_codes", torch.zeros(4, 2, 16, 64, dtype=torch.uint8), TypeError),
    ("append", "v_codes", torch.zeros(4, 2, 16, 128, dtype=I8), ValueError),
    ("append", "k_scales", None, TypeError),
    ("append", "k_scales", torch.zeros(4, 2, 16, dtype=F16), TypeError),
    ("append", "v_scales", torch.zeros(4, 2, 16, 1), ValueError),
    ("append", "v_scales", torch.zeros(4, 16, 2).transpose(1, 2), ValueError),
    ("append", "pos", torch.zeros(1, 2, dtype=I32), ValueError),
    ("append", "axis", torch.zeros(15, dtype=I32), ValueError),
    ("attn", "q", torch.zeros(3, 4, 64), TypeError),
    ("attn", "k_pages", torch.zeros(4, 2, 16, 64, dtype=BF16), TypeError),
    ("attn", "v_pages", torch.zeros(3, 2, 16, 64, dtype=I8), ValueError),
    ("attn", "v_scales", None, TypeError),
    ("attn", "k_scales", None, TypeError),
    ("attn", "tree", torch.zeros(3, dtype=I32), ValueError),
    ("attn", "tree", torch.zeros(2, 1, dtype=I32), ValueError),
    ("attn", "tree", torch.zeros(3, 0, dtype=I32), ValueError),
    ("attn", "tree", torch.zeros(3, 1, dtype=torch.int64), TypeError),
    ("attn", "tree", torch.zeros(3, 2, dtype=I32)[:, ::2], ValueError),
    ("attn", "sinks", 1.5, TypeError),
    ("attn", "sinks", 1 << 40, OverflowError),
    ("attn", "lse", torch.zeros(4, 3), ValueError),
    ("attn16", "k_pages", torch.zeros(4, 2, 16, 64, dtype=I8), TypeError),
    ("attn16", "q", torch.zeros(3, 4, 64, dtype=F16), TypeError),
    ("attn16", "k_scales", torch.zeros(4, 2, 16), TypeError),
    ("keep", "keep", torch.zeros(7, dtype=I32), ValueError),
    ("keep", "keep", torch.zeros(2, 7, dtype=I32), ValueError),
    ("keep", "kept", torch.zeros(1, dtype=torch.int64), TypeError),
    ("keep", "v_scales", None, TypeError),
    ("keep16", "k_pages", torch.zeros(4, 2, 16, 64), TypeError),
    ("keep16", "v_pages", torch.zeros(4, 2, 16, 64, dtype=BF16), TypeError),
    ("keep16", "k_pages", torch.zeros(4, 2, 16, 64, dtype=I8), TypeError),
]


@pytest.mark.parametrize("call,name,value,error", BAD)
def test_bad_argument(call, name, value, error):
    args, fn = CALLS[call]
    with pytest.raises(error):
        getattr(m, fn)(**dict(args(), **{name: value}))


@pytest.mark.parametrize("call", CALLS)
def test_host_tensors_are_refused_last(call):
    """Good arguments on the host: the library would take them, but they are on no CUDA device."""
    args, fn = CALLS[call]
    with pytest.raises(ValueError, match="not the current CUDA device"):
        getattr(m, fn)(**args())


@pytest.mark.parametrize("call,bad", [("attn", dict(max_new=0)), ("attn", dict(window=-1)), ("attn", dict(sinks=-1)),
                                      ("attn", dict(tree=torch.zeros(3, 33, dtype=I32))),
                                      ("keep", dict(keep=torch.zeros(1, 0, dtype=I32)))])
def test_the_library_refuses(call, bad):
    args, fn = CALLS[call]
    with pytest.raises(m.MoeError, match="INVALID_SHAPE"):
        getattr(m, fn)(**dict(args(), **bad))


@pytest.mark.parametrize("call", CALLS)
def test_argument_lists(call):
    args, fn = CALLS[call]
    with pytest.raises(TypeError, match="unexpected keyword"):
        getattr(m, fn)(**args(), other=1)
    with pytest.raises(TypeError, match="missing argument"):
        getattr(m, fn)(next(iter(args().values())))
    with pytest.raises(TypeError, match="takes"):
        getattr(m, fn)(*range(40))


# --------------------------------------------------------------------------
# the cases' own definitions
# --------------------------------------------------------------------------
def test_quantised():
    x = torch.tensor([[0.0, 0.0], [1.0, -0.5], [127.0, 0.5], [127.0, 1.5], [1e-38, 1e-39], [INF, 1.0], [NAN, 1.0]])
    c, d = quantised(x)
    assert c.tolist() == [[0, 0], [127, -64], [127, 0], [127, 2], [0, 0], [0, 0], [0, 0]]
    assert d[:5].tolist() == [0.0, float(torch.tensor(1.0) / 127), 1.0, 1.0, 0.0]
    assert float(d[5]) == INF and math.isnan(float(d[6]))


def test_visible():
    v = lambda *a: visible(*a).int().tolist()  # noqa: E731
    assert v(2, 4, 0, 0, None, 0) == [[1, 1, 1, 0], [1, 1, 1, 1]]
    assert v(2, 4, 2, 1, None, 0) == [[1, 1, 1, 0], [1, 0, 1, 1]]
    assert v(3, 4, 0, 0, [1, 3, 5], 1) == [[1, 1, 0, 0], [1, 1, 1, 0], [1, 1, 0, 1]]
    # window 2: the root (place 1) sees tokens 0 and 1, its children (place 2) of the old ones none
    assert v(3, 4, 2, 0, [1, 3, 5], 1) == [[1, 1, 0, 0], [0, 1, 1, 0], [0, 1, 0, 1]]
    assert v(3, 4, 2, 1, [1, 3, 0], 1) == [[1, 1, 0, 0], [1, 1, 1, 0], [1, 0, 0, 0]]
    # more new tokens than cached ones: the first is not cached and sees nothing
    assert v(3, 2, 0, 0, None, 0) == [[0, 0], [1, 0], [1, 1]]
    assert v(3, 2, 0, 0, [1, 3, 7], 1) == [[0, 0], [1, 0], [1, 1]]
