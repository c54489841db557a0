"""Calls with ``stream=`` that allocate their workspace and outputs themselves, while the
current stream is busy: what it still does with memory that is free again, and when it
would get to a fill, must not matter."""

import numpy as np
import pytest
import torch

import cases
import test_gpu_chunk_q8 as T
from test_gpu_chunk_q8 import pkv  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

DIRTY = 64 << 20


def calls(pkv):  # noqa: F811
    """name -> call(**kw) returning a tuple of tensors, inputs on the device."""
    cu = lambda x: (x if torch.is_tensor(x) else torch.from_numpy(np.ascontiguousarray(x))).cuda()  # noqa: E731
    c = cases.random_case(41, [700, 90, 3000], 8, 2, 128, torch.bfloat16)
    m = cases.multiquery_case(42, [700, 90, 300], [4, 2, 3], 8, 2, 128, torch.bfloat16)
    g = cases.grouped_case(43, [0, 0, 0, -1], [8], [40, 7, 90, 60], 8, 2, 128, torch.bfloat16)
    few, many = T.make(44, [700, 90, 300], [4, 2, 3], 8, 2, 128), T.make(45, [700, 90, 2000], [40, 80, 200], 8, 2, 128)
    few["tables"] = np.pad(few["tables"], ((0, 0), (0, 6000)), constant_values=-1)    # the kernel that splits the cache
    f, y = T.device(few), T.device(many)
    cd, md = {k: cu(v) for k, v in c.items() if k in ("q", "k_pool", "v_pool", "tables", "lens")}, \
        {k: cu(v) for k, v in m.items() if k in ("q", "k_pool", "v_pool", "tables", "lens", "query_start")}
    gd = {k: cu(v) for k, v in g.items() if k in ("q", "k_pool", "v_pool", "tables", "lens", "prefix_group", "group_blocks")}
    rows = torch.tensor([0, 700, 790, 1090], dtype=torch.int32).cuda()
    rng = np.random.default_rng(46)
    p, q = cu(rng.random((9, 4000), np.float32)), cu(rng.random((6, 4000), np.float32))
    tok, acc, sam = cu(rng.integers(0, 4000, 6).astype(np.int32)), cu(rng.random(6, np.float32)), cu(rng.random(3, np.float32))
    ts, ds, lens = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 3, 6, 9], [0, 2, 4, 6], [9, 9, 9]))
    one = lambda fn: (lambda **kw: (fn(**kw),))  # noqa: E731
    attn = (cd["q"], cd["k_pool"], cd["v_pool"], cd["tables"], cd["lens"], c["scale"])
    return {
        "decode": one(lambda **kw: pkv.pkv_decode_attention(*attn, **kw)),
        "decode_noalloc": one(lambda **kw: pkv.pkv_decode_attention_noalloc(*attn, **kw)),
        "decode_prefixed": one(lambda **kw: pkv.pkv_decode_attention_prefixed(
            gd["q"], gd["k_pool"], gd["v_pool"], gd["tables"], gd["lens"], g["scale"], gd["prefix_group"],
            gd["group_blocks"], 8, **kw)),
        "multiquery": one(lambda **kw: pkv.pkv_multiquery_attention(
            md["q"], md["k_pool"], md["v_pool"], md["tables"], md["lens"], md["query_start"], m["scale"], 4, **kw)),
        "decode_q8": one(lambda **kw: pkv.pkv_decode_attention_q8(
            f["q"], f["kc"], f["vc"], f["sc"], f["tables"], f["lens"], few["scale"], query_start=f["start"],
            max_query_len=4, **kw)),
        "multiquery_q8 split": one(lambda **kw: T.call(pkv, few, f, **kw)),
        "multiquery_q8 tiles": one(lambda **kw: T.call(pkv, many, y, **kw)),
        "gather": lambda **kw: pkv.pkv_gather(md["k_pool"], md["v_pool"], md["tables"], md["lens"], rows, 1090, **kw),
        "gather_q8": lambda **kw: pkv.pkv_gather_q8(f["kc"], f["vc"], f["sc"], f["tables"], f["lens"], rows, 1090, **kw),
        "verify_drafts": lambda **kw: pkv.pkv_verify_drafts(p, q, tok, acc, sam, ts, ds, 2, context_lens=lens, **kw),
    }


NAMES = ["decode", "decode_noalloc", "decode_prefixed", "multiquery", "decode_q8", "multiquery_q8 split",
         "multiquery_q8 tiles", "gather", "gather_q8", "verify_drafts"]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_that_a_call_makes_belongs_to_its_stream(pkv, name, raw):  # noqa: F811
    every = calls(pkv)
    assert sorted(every) == sorted(NAMES)
    call = every[name]
    want = call()
    shapes = [(t.shape, t.dtype) for t in want]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # free memory of the current stream: dirty blocks of many sizes, and blocks of the outputs'
    # sizes that it has yet to write
    torch.cuda.empty_cache()
    dirty = [torch.full((DIRTY >> i,), 0x55, dtype=torch.uint8, device="cuda") for i in range(0, 16, 2)]
    late = [torch.empty(s, dtype=t, device="cuda") for s, t in shapes]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                           # about 0.1 s
    for t in late:
        t.fill_(7)
    del dirty, late, t
    got = call(stream=side.cuda_stream if raw else side)
    side.synchronize()
    early = [t.clone() for t in got]
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, early):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert pkv.pkv_device_status(clear=True) == 0


def test_outputs_are_there_for_the_current_stream(pkv):  # noqa: F811
    """A result that the current stream reads late, dropped at once: the next call's is other memory."""
    call = calls(pkv)["multiquery_q8 split"]
    want = call()[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    copies = []
    for _ in range(4):
        out = call(stream=side)[0]
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(20_000_000)
        copies.append(out.clone())
        del out
        with torch.cuda.stream(side):
            torch.full_like(want, 7)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in copies)


def test_the_default_stream_as_a_handle(pkv):  # noqa: F811
    call = calls(pkv)["gather"]
    assert all(torch.equal(a, b) for a, b in zip(call(), call(stream=0)))
