"""Host-side refusals of the 4-bit cache's, the rotary and the planning calls: every
call below returns from the checks, before any CUDA call, and no pointer is dereferenced."""

import ctypes

import pytest

from paged_kv_cache_209_gb300.pkv import CacheDesc

FAKE = 0x10000
F = ctypes.c_float
NULL, SHAPE, DTYPE, ALIGN, OVERLAP, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 6, 7, 10


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_209_gb300 import build, pkv
    import os
    if not os.path.exists(pkv.LIB_PATH):
        build.build()
    return pkv.load_library()


def desc(**kw):
    return CacheDesc(**{**dict(num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, dtype=3), **kw})


BAD_DESCS = [(dict(block_size=8), SHAPE), (dict(head_dim=96), SHAPE), (dict(num_kv_heads=0), SHAPE), (dict(num_blocks=0), SHAPE),
             (dict(dtype=1), DTYPE), (dict(dtype=9), DTYPE), (dict(num_blocks=1 << 31), SHAPE),
             (dict(num_blocks=1 << 29, num_kv_heads=4), SHAPE)]


@pytest.mark.parametrize("kw,status", BAD_DESCS)
def test_geometry(lib, kw, status):
    d = ctypes.byref(desc(**kw))
    assert lib.pkv_append_q4(FAKE, FAKE, FAKE, 4, FAKE, d, 0, None) == status
    assert lib.pkv_copy_blocks_q4(FAKE, 1, FAKE, d, 0, None) == status
    assert lib.pkv_gather_q4(FAKE, FAKE, 4, FAKE, None, FAKE, 2, 8, FAKE, FAKE, 1, d, 0, None) == status
    assert lib.pkv_decode_attention_q4(FAKE, FAKE, FAKE, 4, FAKE, 2, 32, F(.1), FAKE, FAKE, 1 << 40, d, 0, None) == status
    assert lib.pkv_multiquery_attention_q4(FAKE, FAKE, FAKE, 4, FAKE, FAKE, 2, 32, 3, F(.1), FAKE, FAKE, 1 << 40, d, 0,
                                           None) == status
    assert lib.pkv_multiquery_q4_workspace_size(2, 32, 4, 3, d) == 0


def test_append_copy_gather(lib):
    d = ctypes.byref(desc())
    app = lambda k=FAKE, v=FAKE, s=FAKE, n=4, c=FAKE: lib.pkv_append_q4(k, v, s, n, c, d, 0, None)  # noqa: E731
    assert app(k=None) == app(v=None) == app(s=None) == app(c=None) == NULL
    assert app(k=FAKE + 2) == app(v=FAKE + 8) == app(s=FAKE + 4) == app(c=FAKE + 8) == ALIGN
    assert app(n=-1) == app(n=1 << 28) == app(n=(1 << 62) + 4) == SHAPE
    assert app(k=None, v=None, s=None, n=0) == 0
    assert lib.pkv_append_q4(FAKE, FAKE, FAKE, 4, FAKE, None, 0, None) == NULL
    cp = lambda p=FAKE, n=1, c=FAKE: lib.pkv_copy_blocks_q4(p, n, c, d, 0, None)  # noqa: E731
    assert cp(p=None) == cp(c=None) == NULL and cp(p=FAKE + 4) == cp(c=FAKE + 4) == ALIGN and cp(n=-1) == cp(n=1 << 60) == SHAPE and cp(n=0) == 0
    ga = lambda **kw: lib.pkv_gather_q4(kw.get("c", FAKE), FAKE, kw.get("w", 4), FAKE, None, kw.get("r", FAKE), 2,  # noqa: E731
                                        kw.get("n", 8), kw.get("o", FAKE), FAKE, kw.get("t", 1), d, kw.get("f", 0), None)
    assert ga(c=None) == ga(r=None) == ga(o=None) == NULL and ga(o=FAKE + 8) == ga(c=FAKE + 4) == ALIGN
    assert ga(w=0) == ga(n=-1) == ga(n=1 << 31) == SHAPE and ga(t=2) == ga(t=3) == DTYPE and ga(n=0) == 0
    assert ga(f=0x80000000) == UNSUPPORTED


def test_attention(lib):
    d = ctypes.byref(desc())
    dec = lambda **kw: lib.pkv_decode_attention_q4(  # noqa: E731
        kw.get("q", FAKE), kw.get("c", FAKE), kw.get("t", FAKE), kw.get("w", 4), kw.get("l", FAKE), kw.get("b", 2),
        kw.get("h", 32), F(kw.get("s", .1)), kw.get("o", FAKE), kw.get("ws", FAKE), kw.get("n", 1 << 40), d, kw.get("f", 0), None)
    mul = lambda **kw: lib.pkv_multiquery_attention_q4(  # noqa: E731
        kw.get("q", FAKE), kw.get("c", FAKE), kw.get("t", FAKE), kw.get("w", 4), kw.get("l", FAKE), kw.get("r", FAKE),
        kw.get("b", 2), kw.get("h", 32), kw.get("m", 3), F(kw.get("s", .1)), kw.get("o", FAKE), kw.get("ws", FAKE),
        kw.get("n", 1 << 40), d, kw.get("f", 0), None)
    for call in (dec, mul):
        for name in ("q", "c", "t", "l", "o", "ws"):
            assert call(**{name: None}) == NULL, name
        for name, off in (("q", 2), ("c", 8), ("t", 2), ("l", 1), ("o", 8), ("ws", 16)):
            assert call(**{name: FAKE + off}) == ALIGN, name
        assert call(h=30) == call(h=0) == call(h=1032) == call(b=-1) == call(w=0) == call(w=1 << 27) == SHAPE
        assert call(w=1 << 21, b=1024) == SHAPE
        assert call(s=float("nan")) == call(s=float("inf")) == SHAPE
        assert call(f=0x80000000) == UNSUPPORTED
        assert call(n=0) == call(n=255) == WORKSPACE
        assert call(b=0) == 0
    assert dec(h=264) == UNSUPPORTED                        # 33 query heads per KV head
    assert mul(m=0) == SHAPE and mul(m=65537) == UNSUPPORTED and mul(r=None) == NULL and mul(r=FAKE + 2) == ALIGN
    size = lib.pkv_multiquery_q4_workspace_size
    assert size(2, 30, 4, 3, d) == size(2, 32, 4, 0, d) == size(2, 32, 4, 65537, d) == size(-1, 32, 4, 3, d) == 0
    assert size(2, 32, 0, 3, d) == size(2, 32, 1 << 27, 3, d) == 0


def test_rotary(lib):
    table = lambda **kw: lib.pkv_rotary_table(kw.get("f", FAKE), kw.get("r", 64), kw.get("p", 0), kw.get("n", 8),  # noqa: E731
                                              F(kw.get("x", 1.0)), kw.get("t", FAKE), None)
    assert table(f=None) == table(t=None) == NULL and table(f=FAKE + 4) == table(t=FAKE + 8) == ALIGN and table(n=0) == 0
    for bad in (dict(r=0), dict(r=3), dict(r=8194), dict(p=-1), dict(n=-1), dict(p=1 << 30, n=1 << 30), dict(n=1 << 31),
                dict(p=1 << 40), dict(x=float("nan"))):
        assert table(**bad) == SHAPE, bad

    def app(dtype=1, **kw):
        g = lambda name, default=FAKE: kw.get(name, default)  # noqa: E731
        return lib.pkv_append_rotary(g("q"), g("qs", 4096), g("k"), g("ks", 1024), g("v"), g("vs", 1024), g("p"), g("t"),
                                     g("np", 100), g("r", 128), 0, g("s"), g("n", 4), g("h", 32), g("o"), g("os", 4096),
                                     g("kc"), g("vc"), g("sc", FAKE if dtype == 2 else None),
                                     ctypes.byref(desc(dtype=dtype, **kw.get("d", {}))), g("fl", 0), None)
    for dtype in (0, 1, 2, 3):
        for name in ("q", "k", "v", "p", "t", "s", "o", "kc"):
            assert app(dtype, **{name: None}) == NULL, name
        for name, off in (("q", 8), ("k", 2), ("v", 4), ("p", 2), ("t", 8), ("s", 4), ("o", 8), ("kc", 8), ("vc", 8)):
            assert app(dtype, **{name: FAKE + off}) == ALIGN, name
        for bad in (dict(r=0), dict(r=3), dict(r=130), dict(np=0), dict(n=-1), dict(n=1 << 26), dict(n=1 << 62), dict(h=-1), dict(h=1025),
                    dict(qs=4088), dict(ks=1016), dict(vs=0), dict(os=-4096), dict(ks=1 << 31), dict(d=dict(head_dim=96))):
            assert app(dtype, **bad) == SHAPE, bad
        assert app(dtype, qs=4097) == app(dtype, ks=1026) == ALIGN
        assert app(dtype, n=0) == 0 and app(dtype, fl=1, n=20000) == UNSUPPORTED
    # q_out over an input or a pool (the host refuses before anything is launched)
    far = {name: FAKE + (i << 32) for i, name in enumerate(("q", "k", "v", "p", "t", "s", "kc", "vc", "sc"), 1)}
    step = 2 * 4096                                         # bytes of a row of q
    for dtype in (1, 2, 3):
        for out in (far["q"] + 16, far["q"] - 16, far["q"] + 4 * step - 16, far["k"], far["k"] - 4 * step + 16, far["v"] + 16, far["p"],
                    far["t"] + 100 * 512 - 16, far["s"] + 16, far["kc"], *([far["vc"]] if dtype != 3 else [])):
            assert app(dtype, **{**far, "o": out}) == OVERLAP, hex(out)
        # parts of one product's output: a wide row, q_out between the parts
        wide = dict(q=FAKE, k=FAKE + 8192, v=FAKE + 10240, qs=8192, ks=8192, vs=8192, os=8192)
        for out in (FAKE + 16, FAKE + 8192, FAKE + 12288 - 16, FAKE + 16384 - 16, FAKE + 3 * 16384 + 16, FAKE - 16):
            assert app(dtype, **{**far, **wide, "o": out}) == OVERLAP, hex(out)
        assert app(dtype, **{**far, **wide, "os": 8200}) == OVERLAP
    assert app(1, vc=None) == app(2, vc=None) == app(2, sc=None) == NULL
    assert app(2, sc=FAKE + 4) == ALIGN
    assert app(7) == DTYPE
    assert lib.pkv_append_rotary(*([FAKE, 8] * 3), FAKE, FAKE, 1, 2, 0, FAKE, 0, 1, FAKE, 8, FAKE, FAKE, None, None, 0, None) == NULL


def test_plan(lib):
    def plan(**kw):
        at = [0x100000 * (i + 1) for i in range(13)]
        names = ("lens", "new", "held", "free", "count", "tables", "slots", "pos", "start", "nlens", "nheld", "ncount", "result")
        p = {**dict(zip(names, at)), **kw}
        g = lambda name, default: kw.get(name, default)  # noqa: E731
        return lib.pkv_plan_step(p["lens"], p["new"], p["held"], p["free"], g("cap", 100), p["count"], p["tables"], g("w", 8),
                                 g("b", 4), g("rows", 40), g("nb", 64), p["slots"], p["pos"], p["start"], p["nlens"],
                                 p["nheld"], p["ncount"], p["result"], g("f", 0), None)
    names = ("lens", "new", "held", "free", "count", "tables", "slots", "pos", "start", "nlens", "nheld", "ncount", "result")
    for name in names:
        assert plan(**{name: None}) == NULL, name
        assert plan(**{name: 0x500002}) == ALIGN, name
    assert plan(slots=0x700004) == ALIGN
    for bad in (dict(b=-1), dict(rows=-1), dict(rows=1 << 31), dict(cap=-1), dict(cap=1 << 31), dict(nb=-1), dict(w=0),
                dict(w=1 << 27)):
        assert plan(**bad) == SHAPE, bad
    assert plan(b=16385) == plan(f=0x80000000) == UNSUPPORTED
    # outputs over inputs, and over each other
    at = 0x100000
    assert plan(nlens=at) == plan(nheld=3 * at + 12) == plan(ncount=5 * at) == plan(start=2 * at - 16) == OVERLAP
    assert plan(tables=4 * at + 396) == plan(pos=7 * at + 316) == plan(result=at * 10 + 12) == OVERLAP
    assert plan(slots=6 * at + 120) == OVERLAP
