"""Calls from two host threads at once, on two streams, of batches as different as they can be: whatever a launch sets up
on the host, the other thread's launches go through, and both threads' results are those of a call alone. (Calls go
through the C ABI, as Python's lock would keep them apart.)"""

import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def in_turn_and_at_once(calls, outputs, times=1500):
    """Each call alone, then every call `times` times from a thread of its own."""
    streams = [torch.cuda.Stream() for _ in calls]
    for call, stream in zip(calls, streams):
        assert call(stream.cuda_stream) == 0
    torch.cuda.synchronize()
    alone = [[t.clone() for t in some] for some in outputs]
    for some in outputs:
        for t in some:
            t.zero_()
    torch.cuda.synchronize()
    found, start = [set() for _ in calls], threading.Barrier(len(calls))

    def work(i):
        start.wait()
        for _ in range(times):
            found[i].add(calls[i](streams[i].cuda_stream))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert found == [{0} for _ in calls]
    for some, want in zip(outputs, alone):
        assert all(torch.equal(a, b) for a, b in zip(some, want))


def attention_q4(pkv, batch, q_heads, head_dim, new):
    """One token of context more than there are new ones, every sequence's table naming the same block."""
    g = torch.Generator(device="cuda").manual_seed(batch)
    cache = torch.randint(0, 256, (4, 1, 16 * head_dim + 128), dtype=torch.uint8, device="cuda", generator=g)
    cache[..., 16 * head_dim:] = torch.full((4, 1, 32), 0.25, device="cuda").view(torch.uint8)
    q = torch.randn((batch * new, q_heads, head_dim), device="cuda", generator=g).to(torch.bfloat16)
    tables = torch.full((batch, 1), 2, dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), new + 1, dtype=torch.int32, device="cuda")
    start = torch.arange(0, batch * new + 1, new, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    desc = pkv.CacheDesc(4, 16, 1, head_dim, pkv.PKV_INT4)
    size = pkv.pkv_multiquery_q4_workspace_size(batch, q_heads, 1, new, cache)
    work = torch.zeros(size, dtype=torch.uint8, device="cuda")
    lib = pkv.load_library()

    def call(stream, keep=(cache, q, tables, lens, start, work)):
        return lib.pkv_multiquery_attention_q4(q.data_ptr(), cache.data_ptr(), tables.data_ptr(), 1, lens.data_ptr(), start.data_ptr(),
                                               batch, q_heads, new, 0.1, out.data_ptr(), work.data_ptr(), size, ctypes.byref(desc),
                                               0, stream)
    return call, [out]


@pytest.mark.parametrize("q_heads,head_dim,new", [(4, 128, 1), (4, 64, 2), (4, 128, 4), (8, 64, 4)])
def test_attention_q4(pkv, q_heads, head_dim, new):
    made = [attention_q4(pkv, batch, q_heads, head_dim, new) for batch in (1024, 1)]
    torch.cuda.synchronize()
    in_turn_and_at_once([c for c, _ in made], [o for _, o in made])


def test_attention_q4_with_one_and_two_warps_a_block(pkv):
    """16 and 32 rows share a kernel, and differ in its shared memory."""
    made = [attention_q4(pkv, 600, 4, 128, 4), attention_q4(pkv, 600, 8, 128, 4)]
    torch.cuda.synchronize()
    in_turn_and_at_once([c for c, _ in made], [o for _, o in made])


def plan(pkv, batch):
    ints = lambda value, n=batch: torch.full((n,), value, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, new, held, free, left, tables = ints(5), ints(1), ints(1), ints(3, 8), ints(8, 1), ints(2)
    slots = torch.zeros(batch, dtype=torch.int64, device="cuda")
    out = [slots, ints(0), ints(0, batch + 1), ints(0), ints(0), ints(0, 1), ints(0, 2)]
    lib = pkv.load_library()

    def call(stream, keep=(lens, new, held, free, left, tables)):
        return lib.pkv_plan_step(lens.data_ptr(), new.data_ptr(), held.data_ptr(), free.data_ptr(), 8, left.data_ptr(),
                                 tables.data_ptr(), 1, batch, batch, 4, *(t.data_ptr() for t in out), 0, stream)
    return call, out


def test_plan_step(pkv):
    """Batches whose sums take 131 and 48 KB."""
    made = [plan(pkv, batch) for batch in (16384, 6100)]
    torch.cuda.synchronize()
    in_turn_and_at_once([c for c, _ in made], [o for _, o in made])


def pools_of(pkv, kind, head_dim, g):
    rows = torch.randn((2, 4, 1, 16, head_dim), device="cuda", generator=g)
    if kind == "q8":
        codes = torch.randint(-128, 128, (4, 1, 16, head_dim), dtype=torch.int8, device="cuda", generator=g)
        return [codes, codes.transpose(2, 3).contiguous(), torch.full((4, 1, 2, 16), 0.01, device="cuda")], pkv.PKV_INT8
    return [rows[0].to(torch.bfloat16), rows[1].to(torch.bfloat16)], pkv.PKV_BF16


def older_attention(pkv, kind, batch, head_dim, new):
    """Decode (new 0) or multi-query attention over bf16 or int8 pools."""
    g = torch.Generator(device="cuda").manual_seed(batch)
    pools, dtype = pools_of(pkv, kind, head_dim, g)
    rows = batch * max(new, 1)
    q = torch.randn((rows, 4, head_dim), device="cuda", generator=g).to(torch.bfloat16)
    tables = torch.full((batch, 1), 2, dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), 9, dtype=torch.int32, device="cuda")
    start = torch.arange(0, rows + 1, max(new, 1), dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    desc = pkv.CacheDesc(4, 16, 1, head_dim, dtype)
    lib = pkv.load_library()
    at = [p.data_ptr() for p in pools]
    most = max(new, 1)
    if kind == "q8":
        size = lib.pkv_decode_q8_workspace_size(batch, 4, 1, most, ctypes.byref(desc), None)
    elif new:
        size = lib.pkv_multiquery_workspace_size(batch, 4, 1, most, ctypes.byref(desc), None)
    else:
        size = lib.pkv_decode_workspace_size(batch, 4, 1, ctypes.byref(desc), None)
    work = torch.zeros(size, dtype=torch.uint8, device="cuda")
    rest = (0.1, out.data_ptr(), work.data_ptr(), size, ctypes.byref(desc), 0, None)

    def call(stream, keep=(pools, q, tables, lens, start, work)):
        if kind == "q8":
            return lib.pkv_decode_attention_q8(q.data_ptr(), *at, tables.data_ptr(), 1, lens.data_ptr(), start.data_ptr(), batch, 4, most,
                                               *rest, stream)
        if new:
            return lib.pkv_multiquery_attention(q.data_ptr(), *at, tables.data_ptr(), 1, lens.data_ptr(), start.data_ptr(), batch, 4, most,
                                                *rest, stream)
        return lib.pkv_decode_attention(q.data_ptr(), *at, tables.data_ptr(), 1, lens.data_ptr(), batch, 4, *rest, stream)
    return call, [out]


@pytest.mark.parametrize("kind,head_dim,new", [("bf16", 128, 0), ("bf16", 64, 0), ("bf16", 128, 3), ("bf16", 64, 3), ("q8", 128, 1),
                                               ("q8", 128, 3)])
def test_older_attention(pkv, kind, head_dim, new):
    made = [older_attention(pkv, kind, batch, head_dim, new) for batch in (1024, 1)]
    torch.cuda.synchronize()
    in_turn_and_at_once([c for c, _ in made], [o for _, o in made])
