"""Host-side refusals of the int8 chunk attention, the reading-back calls and
draft verification: every call here returns from the host checks, before any
CUDA call (the pointers are never dereferenced)."""

import ctypes
import os

import pytest
import torch

FAKE = 0x10000
OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 7, 10


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_209_gb300 import build, pkv
    if not os.path.exists(pkv.LIB_PATH):
        build.build()
    return pkv.load_library()


def desc(**kw):
    from paged_kv_cache_209_gb300.pkv import CacheDesc
    d = dict(num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, dtype=2)
    d.update(kw)
    return ctypes.byref(CacheDesc(**d))


BAD_GEOMETRY = [(dict(block_size=8), SHAPE), (dict(head_dim=96), SHAPE), (dict(num_kv_heads=0), SHAPE),
                (dict(num_blocks=0), SHAPE), (dict(num_blocks=2 ** 40), SHAPE), (dict(dtype=7), DTYPE)]


def chunk(lib, d=None, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, sc=FAKE, tab=FAKE, maxb=16, lens=FAKE, qs=FAKE, batch=2, heads=32, nq=64,
             scale=0.1, out=FAKE, ws=FAKE, wsb=1 << 40, flags=0)
    a.update(kw)
    return lib.pkv_multiquery_attention_q8(a["q"], a["k"], a["v"], a["sc"], a["tab"], a["maxb"], a["lens"], a["qs"],
                                           a["batch"], a["heads"], a["nq"], ctypes.c_float(a["scale"]), a["out"],
                                           a["ws"], a["wsb"], d or desc(), a["flags"], None)


def test_chunk_refusals(lib):
    for kw, status in BAD_GEOMETRY + [(dict(dtype=1), DTYPE), (dict(dtype=0), DTYPE)]:
        assert chunk(lib, desc(**kw)) == status, kw
    for name in ("q", "k", "v", "sc", "tab", "lens", "qs", "out", "ws"):
        assert chunk(lib, **{name: None}) == NULL, name
        assert chunk(lib, **{name: FAKE + 2}) == ALIGN, name
    assert chunk(lib, ws=FAKE + 16) == ALIGN
    for kw in (dict(heads=30), dict(heads=0), dict(heads=1032), dict(nq=0), dict(batch=-1), dict(maxb=0),
               dict(maxb=1 << 27), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert chunk(lib, **kw) == SHAPE, kw
    assert chunk(lib, nq=65537) == UNSUPPORTED
    assert chunk(lib, flags=0x80000000) == UNSUPPORTED
    assert chunk(lib, wsb=64) == WORKSPACE                     # the tile path
    assert chunk(lib, nq=4, wsb=64) == WORKSPACE               # the split path
    assert chunk(lib, batch=0) == OK


def test_chunk_workspace_size(lib):
    size = lambda d=None, batch=4, heads=32, maxb=16, nq=64: lib.pkv_multiquery_q8_workspace_size(  # noqa: E731
        batch, heads, maxb, nq, d or desc())
    assert size() >= 256 and size(desc(head_dim=64), nq=1) >= 256
    assert size(nq=0) == 0 and size(nq=65537) == 0 and size(heads=30) == 0 and size(heads=2048) == 0
    assert size(desc(dtype=1)) == 0 and size(batch=-1) == 0
    # the size for the largest call serves the smaller ones, on either kernel
    for batch, nq in ((1, 1), (4, 8), (1500, 8), (1500, 64)):
        assert size(batch=batch, nq=nq) <= size(batch=1500, nq=512)
    assert size(nq=8) >= lib.pkv_decode_q8_workspace_size(4, 32, 16, 8, desc(), None)


def gather(lib, q8, d=None, **kw):
    a = dict(k=FAKE, v=FAKE, sc=FAKE, tab=FAKE, maxb=16, lens=FAKE, first=FAKE, rs=FAKE, batch=2, rows=64, ko=FAKE,
             vo=FAKE, dt=1, flags=0)
    a.update(kw)
    if q8:
        return lib.pkv_gather_q8(a["k"], a["v"], a["sc"], a["tab"], a["maxb"], a["lens"], a["first"], a["rs"],
                                 a["batch"], a["rows"], a["ko"], a["vo"], a["dt"], d or desc(), a["flags"], None)
    return lib.pkv_gather(a["k"], a["v"], a["tab"], a["maxb"], a["lens"], a["first"], a["rs"], a["batch"], a["rows"],
                          a["ko"], a["vo"], d or desc(dtype=1), a["flags"], None)


@pytest.mark.parametrize("q8", [False, True])
def test_gather_refusals(lib, q8):
    for kw, status in BAD_GEOMETRY:
        assert gather(lib, q8, desc(**dict(dict(dtype=2 if q8 else 1), **kw))) == status, kw
    assert gather(lib, q8, desc(dtype=1 if q8 else 2)) == DTYPE
    for name in ("k", "v", "tab", "lens", "rs", "ko", "vo") + (("sc",) if q8 else ()):
        assert gather(lib, q8, **{name: None}) == NULL, name
        assert gather(lib, q8, **{name: FAKE + 2}) == ALIGN, name
    assert gather(lib, q8, first=FAKE + 2) == ALIGN
    for kw in (dict(batch=-1), dict(rows=-1), dict(rows=1 << 31), dict(maxb=0), dict(maxb=1 << 27)):
        assert gather(lib, q8, **kw) == SHAPE, kw
    assert gather(lib, q8, flags=0x80000000) == UNSUPPORTED
    assert gather(lib, q8, batch=0) == OK and gather(lib, q8, rows=0, ko=None, vo=None) == OK
    if q8:
        assert gather(lib, q8, dt=2) == DTYPE


def verify(lib, **kw):
    a = dict(p=FAKE, ps=1000, pr=10, q=FAKE, qs=1000, qr=8, dt=0, vocab=1000, tok=FAKE, acc=FAKE, smp=FAKE, t0=FAKE,
             d0=FAKE, batch=2, most=4, lens=FAKE, new=FAKE, out=FAKE, num=FAKE, flags=0)
    a.update(kw)
    return lib.pkv_verify_drafts(a["p"], a["ps"], a["pr"], a["q"], a["qs"], a["qr"], a["dt"], a["vocab"], a["tok"],
                                 a["acc"], a["smp"], a["t0"], a["d0"], a["batch"], a["most"], a["lens"], a["new"],
                                 a["out"], a["num"], a["flags"], None)


def test_verify_refusals(lib):
    for name in ("p", "tok", "acc", "smp", "t0", "d0", "lens", "new", "out", "num"):
        assert verify(lib, **{name: None}) == NULL, name
        assert verify(lib, **{name: FAKE + 2}) == ALIGN, name
    assert verify(lib, q=FAKE + 2) == ALIGN and verify(lib, q=FAKE + 1, dt=1) == ALIGN
    for kw in (dict(batch=-1), dict(vocab=0), dict(vocab=(1 << 20) + 1, ps=1 << 21, qs=1 << 21), dict(ps=999),
               dict(qs=999), dict(ps=1 << 31), dict(qs=1 << 31), dict(most=-1), dict(most=65536), dict(pr=-1),
               dict(qr=-1), dict(pr=1 << 31), dict(qr=1 << 31)):
        assert verify(lib, **kw) == SHAPE, kw
    assert verify(lib, dt=2) == DTYPE
    assert verify(lib, flags=0x80000000) == UNSUPPORTED
    assert verify(lib, batch=0, p=None, out=None) == OK


def test_binding_refuses_host_tensors(lib):
    from paged_kv_cache_209_gb300 import pkv
    kc, vc = torch.zeros((3, 2, 16, 64), dtype=torch.int8), torch.zeros((3, 2, 64, 16), dtype=torch.int8)
    sc, kp = torch.zeros((3, 2, 2, 16)), torch.zeros((3, 2, 16, 64))
    t, n, st = (torch.zeros(s, dtype=torch.int32) for s in ((1, 2), (1,), (2,)))
    q, ws, u = torch.zeros((5, 4, 64), dtype=torch.bfloat16), torch.zeros(1024, dtype=torch.uint8), torch.zeros(1)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_multiquery_attention_q8(q, kc, vc, sc, t, n, st, 0.1, 5, workspace=ws)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_gather_q8(kc, vc, sc, t, n, st, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_gather(kp, kp, t, n, st, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_verify_drafts(torch.zeros((2, 10)), torch.zeros((1, 10)), n, u, u, st, st, 1)


def test_binding_refuses_wrong_types_and_shapes(lib, monkeypatch):
    """The checks behind the device check, on host tensors (-1 is a host tensor's device number)."""
    from paged_kv_cache_209_gb300 import pkv
    monkeypatch.setattr(pkv, "_here", lambda: -1)
    kc, vc = torch.zeros((3, 2, 16, 64), dtype=torch.int8), torch.zeros((3, 2, 64, 16), dtype=torch.int8)
    sc = torch.zeros((3, 2, 2, 16))
    t, n, st = (torch.zeros(s, dtype=torch.int32) for s in ((1, 2), (1,), (2,)))
    q = torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    ws = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError, match="contiguous"):
        pkv.pkv_multiquery_attention_q8(q.transpose(0, 1), kc, vc, sc, t, n, st, 0.1, 5, workspace=ws)
    with pytest.raises(ValueError, match="v_codes"):
        pkv.pkv_multiquery_attention_q8(q, kc, kc, sc, t, n, st, 0.1, 5, workspace=ws)
    with pytest.raises(ValueError, match="bf16"):
        pkv.pkv_multiquery_attention_q8(q.float(), kc, vc, sc, t, n, st, 0.1, 5, workspace=ws)
    with pytest.raises(ValueError, match="int32"):
        pkv.pkv_multiquery_attention_q8(q, kc, vc, sc, t.long(), n, st, 0.1, 5, workspace=ws)
    with pytest.raises(ValueError, match="out"):
        pkv.pkv_multiquery_attention_q8(q, kc, vc, sc, t, n, st, 0.1, 5, out=q[:4], workspace=ws)
    with pytest.raises(ValueError, match="row_start"):
        pkv.pkv_gather_q8(kc, vc, sc, t, n, st[:1], 4)
    with pytest.raises(ValueError, match="unsupported"):
        pkv.pkv_gather_q8(kc, vc, sc, t, n, st, 4, out_dtype=torch.float16)
    kp = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_out"):
        pkv.pkv_gather(kp, kp, t, n, st, 4, k_out=torch.zeros((3, 2, 64), dtype=torch.bfloat16))
    p, u = torch.zeros((2, 10)), torch.zeros(1)
    tok = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="draft_probs"):
        pkv.pkv_verify_drafts(p, p, tok, u, u, st, st, 1)
    with pytest.raises(ValueError, match="consecutive"):
        pkv.pkv_verify_drafts(p.t(), None, tok, u, u, st, st, 1)
    with pytest.raises(ValueError, match="accept_uniform is float32"):
        pkv.pkv_verify_drafts(p, p[:1], tok, u.double(), u, st, st, 1)
