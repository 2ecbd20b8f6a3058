"""Host-side checks of the attention half's entry points: every refusal comes
back before anything is enqueued (no GPU needed)."""
import ctypes

import pytest

from tests.test_abi_host import ALIGNED, lib, m  # noqa: F401

P, S, F, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float, ctypes.c_int  # noqa: E741
SHAPE, NULL, MISALIGNED, WORKSPACE = 1, 2, 3, 4
INF, NAN = float("inf"), float("nan")


def norm(lib, x=ALIGNED, xt=0, res=None, gamma=ALIGNED, eps=1e-6, T=3, H=512, sum_out=None, y=ALIGNED, yt=0,
         q=None, d=None, sums=None):
    lib.moe_add_rmsnorm.restype = I
    return lib.moe_add_rmsnorm(P(x), I(xt), P(res), P(gamma), F(eps), I(T), I(H), P(sum_out), P(y), I(yt),
                               P(q), P(d), P(sums), P(None))


@pytest.mark.parametrize("bad,code", [
    (dict(T=0), SHAPE), (dict(T=(1 << 22) + 1), SHAPE), (dict(H=0), SHAPE), (dict(H=12), SHAPE),
    (dict(H=16392), SHAPE), (dict(H=264, q=ALIGNED, d=ALIGNED, sums=ALIGNED), SHAPE),
    (dict(xt=3), SHAPE), (dict(yt=-1), SHAPE), (dict(eps=-1e-9), SHAPE), (dict(eps=NAN), SHAPE),
    (dict(eps=INF), SHAPE), (dict(x=0), NULL), (dict(gamma=0), NULL), (dict(y=0), NULL),
    (dict(q=ALIGNED), NULL), (dict(q=ALIGNED, d=ALIGNED), NULL), (dict(d=ALIGNED, sums=ALIGNED), NULL),
    (dict(x=ALIGNED + 8), MISALIGNED), (dict(res=ALIGNED + 4), MISALIGNED), (dict(sum_out=ALIGNED + 8), MISALIGNED),
    (dict(y=ALIGNED + 2), MISALIGNED), (dict(q=ALIGNED + 8, d=ALIGNED, sums=ALIGNED), MISALIGNED),
])
def test_norm_refusals(lib, bad, code):
    assert norm(lib, **bad) == code


BATCH = dict(N=5, B=2, max_pages=4, num_pages=9, page=16, Hq=8, Hkv=2, D=128, dtype=2)
BAD_BATCH = [dict(N=0), dict(N=(1 << 22) + 1), dict(B=0), dict(B=4097), dict(max_pages=0), dict(num_pages=0),
             dict(page=0), dict(page=8), dict(page=24), dict(page=512), dict(Hkv=0), dict(Hq=0), dict(Hq=9),
             dict(Hq=264), dict(Hq=129, Hkv=1), dict(D=96), dict(D=256), dict(D=0), dict(dtype=0), dict(dtype=3),
             dict(num_pages=1 << 30), dict(max_pages=1 << 27)]


def rope(lib, qkv=ALIGNED, pos=ALIGNED, freq=ALIGNED, axis=None, axes=1, rot=64, qw=None, kw=None, eps=1e-6,
         q_out=ALIGNED, k=ALIGNED, v=ALIGNED, table=ALIGNED, offs=ALIGNED, lens=ALIGNED, ws=ALIGNED, ws_bytes=256,
         **b):
    b = BATCH | b
    lib.moe_rope_append.restype = I
    return lib.moe_rope_append(P(qkv), P(pos), P(freq), P(axis), I(axes), I(rot), I(0), P(qw), P(kw), F(eps),
                               P(q_out), P(k), P(v), P(table), P(offs), P(lens), I(b["N"]), I(b["B"]),
                               I(b["max_pages"]), I(b["num_pages"]), I(b["page"]), I(b["Hq"]), I(b["Hkv"]),
                               I(b["D"]), I(b["dtype"]), P(ws), S(ws_bytes), P(None))


@pytest.mark.parametrize("bad", BAD_BATCH + [dict(axes=0), dict(axes=9), dict(rot=0), dict(rot=8), dict(rot=40),
                                             dict(rot=144), dict(rot=128, D=64), dict(eps=-1.0), dict(eps=NAN)])
def test_rope_shapes(lib, bad):
    assert rope(lib, **bad) == SHAPE


def test_rope_pointers(lib):
    for name in ("qkv", "pos", "freq", "q_out", "k", "v", "table", "offs", "lens", "ws"):
        assert rope(lib, **{name: 0}) == NULL, name
        assert rope(lib, **{name: ALIGNED + 2}) == MISALIGNED, name
    for name in ("axis", "qw", "kw"):
        assert rope(lib, **{name: ALIGNED + 2}) == MISALIGNED, name
    for name in ("qkv", "q_out", "k", "v"):
        assert rope(lib, **{name: ALIGNED + 8}) == MISALIGNED, name
    assert rope(lib, freq=ALIGNED + 4) == MISALIGNED
    assert rope(lib, ws=ALIGNED + 128) == MISALIGNED
    assert rope(lib, ws_bytes=255) == WORKSPACE


def attn(lib, q=ALIGNED, k=ALIGNED, v=ALIGNED, table=ALIGNED, offs=ALIGNED, lens=ALIGNED, max_new=1, scale=0.1,
         softcap=0.0, window=0, out=ALIGNED, lse=None, ws=ALIGNED, ws_bytes=48 << 20, **b):
    b = BATCH | b
    lib.moe_attention_paged.restype = I
    return lib.moe_attention_paged(P(q), P(k), P(v), P(table), P(offs), P(lens), I(b["N"]), I(b["B"]), I(max_new),
                                   I(b["max_pages"]), I(b["num_pages"]), I(b["page"]), I(b["Hq"]), I(b["Hkv"]),
                                   I(b["D"]), I(b["dtype"]), F(scale), F(softcap), I(window), P(out), P(lse), P(ws),
                                   S(ws_bytes), P(None))


@pytest.mark.parametrize("bad", BAD_BATCH + [dict(max_new=0), dict(window=-1), dict(scale=NAN), dict(scale=INF),
                                             dict(softcap=-1.0), dict(softcap=INF), dict(softcap=NAN),
                                             dict(softcap=1e-38, scale=1e5)])
def test_attention_shapes(lib, bad):
    assert attn(lib, **bad) == SHAPE


def test_attention_pointers_and_workspace(lib, m):
    for name in ("q", "k", "v", "table", "offs", "lens", "out", "ws"):
        assert attn(lib, **{name: 0}) == NULL, name
        assert attn(lib, **{name: ALIGNED + 2}) == MISALIGNED, name
    for name in ("q", "k", "v", "out"):
        assert attn(lib, **{name: ALIGNED + 8}) == MISALIGNED, name
    assert attn(lib, lse=ALIGNED + 2) == MISALIGNED
    need = m.moe_attention_workspace_bytes(8, 2, 128)
    assert 256 <= need <= 48 << 20
    assert attn(lib, ws_bytes=need - 1) == WORKSPACE
    assert m.moe_attention_workspace_bytes(9, 2, 128) == 0
    assert m.moe_attention_workspace_bytes(8, 2, 80) == 0
    assert all(m.moe_attention_workspace_bytes(h, k, d) <= 48 << 20
               for h, k in ((1, 1), (256, 2), (256, 256), (64, 4)) for d in (64, 128))


def test_codes_refusals(lib):
    f = lib.moe_ffn_q8k_codes
    f.restype = I

    def call(q=ALIGNED, d=ALIGNED, sums=ALIGNED, T=1, ws_bytes=1 << 40):
        return f(P(q), P(d), P(sums), P(ALIGNED), P(ALIGNED), P(ALIGNED), P(ALIGNED), P(ALIGNED), I(T), I(2048),
                 I(128), I(8), I(768), P(ALIGNED), P(ALIGNED), S(ws_bytes), P(None))
    assert call(T=0) == SHAPE
    assert call(q=0) == NULL and call(d=0) == NULL and call(sums=0) == NULL
    assert call(q=ALIGNED + 8) == MISALIGNED and call(d=ALIGNED + 2) == MISALIGNED
    assert call(ws_bytes=1024) == WORKSPACE


def test_status_name(m):
    assert m.status_str(10) == "MOE_ERR_CACHE_RANGE" and m.STATUS_NAMES[10] == "MOE_ERR_CACHE_RANGE"


class Recorder:
    """Stands for the library: keeps the call that it gets."""

    def __getattr__(self, name):
        def take(*args):
            self.call = name, args
            return 0
        return take


@pytest.mark.parametrize("make,bad,code", [
    (norm, dict(eps=-1.0), SHAPE), (norm, dict(x=ALIGNED + 8), MISALIGNED), (rope, dict(rot=8), SHAPE),
    (rope, dict(q_out=0), NULL), (attn, dict(max_new=0), SHAPE), (attn, dict(ws_bytes=1 << 10), WORKSPACE)])
def test_checks_alone(lib, make, bad, code):
    """MOE_CHECK_ONLY in place of a stream: the checks' answer, with nothing enqueued (nor a GPU needed)."""
    def check(**args):
        call = Recorder()
        make(call, **args)
        name, a = call.call
        return getattr(lib, name)(*a[:-1], P(-1))
    assert check() == 0
    assert check(**bad) == code
