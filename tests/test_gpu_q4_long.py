"""Long contexts and large tensors: offsets past 32 bits in the 4-bit cache, in q and in the rotary table; queries
turned in place; graphs that share a workspace."""

import numpy as np
import pytest
import torch

from oracle import quant4 as Q
from oracle import rotary as R
from q4_cases import B, check, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def pool():
    """250000 blocks of 8 heads of 128: 4.4 GB, the last 17408 bytes of it past 2^32."""
    yield torch.full((250000, 8, Q.record_bytes(128)), 0x5a, dtype=torch.uint8, device="cuda")
    torch.cuda.empty_cache()


@pytest.mark.parametrize("news", [[1, 1], [4, 2], [8, 7], [100, 40]])
def test_blocks_far_into_the_pool(pkv, pool, news):
    s = make(1, [900, 333], news, 32, 8, 128)
    want = reference(s)
    near = s["cache"].shape[0]
    pool[-near:] = s["cache"]
    far = torch.where(s["tables"] >= 0, s["tables"] + (pool.shape[0] - near), s["tables"])
    for cache, tables in ((s["cache"], s["tables"]), (pool, far)):
        got = pkv.pkv_multiquery_attention_q4(s["q"], cache, tables, s["lens"], s["start"], s["scale"], max(news))
        check(got, *want)
    k, v = pkv.pkv_gather_q4(pool, far, s["lens"], torch.tensor([0, 900, 1233], dtype=torch.int32, device="cuda"), 1233)
    k1, v1 = pkv.pkv_gather_q4(s["cache"], s["tables"], s["lens"], torch.tensor([0, 900, 1233], dtype=torch.int32, device="cuda"), 1233)
    assert torch.equal(k, k1) and torch.equal(v, v1)


def test_append_and_copy_far_into_the_pool(pkv, pool):
    last = pool.shape[0] - 1
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn((5, 8, 128), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    small = torch.full((1, 8, Q.record_bytes(128)), 0x5a, dtype=torch.uint8, device="cuda")
    pool[last] = 0x5a
    slots = torch.tensor([15, 0, 3, 7, 8], device="cuda")
    pkv.pkv_append_q4(k, v, slots, small)
    pkv.pkv_append_q4(k, v, slots + B * last, pool)
    assert torch.equal(pool[last], small[0])
    pkv.pkv_copy_blocks_q4(torch.tensor([[last, 1], [1000, last - 1]], device="cuda"), pool)
    assert torch.equal(pool[1], small[0]) and torch.equal(pool[last - 1], pool[1000])
    pool[1] = 0x5a


@pytest.mark.parametrize("batch,n,q_heads", [(1, 262145, 4), (1, 262145, 16), (2, 131072, 8)])
def test_long_contexts(pkv, batch, n, q_heads):
    """(Bounds of tests/q4_cases.py: a CTA takes some hundreds of blocks of these, so sums stay as short as there.)"""
    s = make(3, [n] * batch, [1] * batch, q_heads, 1, 64, garbage=False)
    check(pkv.pkv_decode_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["scale"]), *reference(s, decode=True), mean=False)


def test_a_long_context_in_few_ctas(pkv):
    """So many long sequences that a CTA takes whole ones: each warp sums thousands of tokens. All tables name the same
    blocks, so that the pool stays small."""
    s = make(4, [16384], [1], 4, 1, 128, garbage=False)
    want, bound = reference(s, decode=True)
    many = 1024
    got = pkv.pkv_decode_attention_q4(s["q"].expand(many, -1, -1).contiguous(), s["cache"], s["tables"].expand(many, -1).contiguous(),
                                      s["lens"].expand(many).contiguous(), s["scale"])
    check(got, want.expand(many, -1, -1), bound.expand(many, -1, -1), mean=False)


def test_rotary_over_more_than_2_31_elements(pkv):
    tokens, heads, kv, d = 530000, 32, 1, 128
    q = torch.empty((tokens, heads, d), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty((tokens, kv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (q, k, v):
        x.normal_()
    table = pkv.pkv_rotary_table(pkv.pkv_rotary_frequencies(d).cuda(), 1 << 20)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    slots = torch.arange(tokens, device="cuda")
    cache = torch.zeros((-(-tokens // B), kv, Q.record_bytes(d)), dtype=torch.uint8, device="cuda")
    out = pkv.pkv_append_rotary(q, k, v, pos, table, slots, cache)
    for at in (0, 262144 - 8, tokens - 16):
        few = torch.zeros_like(cache[:1])
        alone = pkv.pkv_append_rotary(q[at:at + 16], k[at:at + 16], v[at:at + 16], pos[at:at + 16], table, slots[:16], few)
        assert torch.equal(out[at:at + 16], alone)
        if at % B == 0:
            assert torch.equal(cache[at // B], few[0])
    again = pkv.pkv_append_rotary(q, k, v, pos, table, slots, cache, q_out=q)
    assert again.data_ptr() == q.data_ptr() and torch.equal(again, out)


def test_table_of_more_than_2_32_bytes(pkv):
    f = pkv.pkv_rotary_frequencies(128).cuda()
    n = (1 << 23) + 7
    table = pkv.pkv_rotary_table(f, n)
    last = pkv.pkv_rotary_table(f, 9, first_position=n - 9)
    assert torch.equal(table[-9:], last)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary", [(128, 128), (128, 64), (64, 16), (64, 10), (128, 126)])
@pytest.mark.parametrize("tokens", [3, 600])
def test_in_place(pkv, interleaved, d, rotary, tokens):
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn((tokens, 24 * d), device="cuda", generator=g).to(torch.bfloat16)
    q, k, v = (x.view(tokens, -1, d) for x in (qkv[:, :16 * d], qkv[:, 16 * d:20 * d], qkv[:, 20 * d:]))
    table = pkv.pkv_rotary_table(torch.from_numpy(R.frequencies(rotary, 10000.0)).cuda(), 700)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    slots = torch.arange(tokens, device="cuda")
    caches = [torch.zeros((-(-tokens // B), 4, Q.record_bytes(d)), dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = pkv.pkv_append_rotary(q, k, v, pos, table, slots, caches[0], interleaved=interleaved)
    pkv.pkv_append_rotary(q, k, v, pos, table, slots, caches[1], interleaved=interleaved, q_out=q)
    assert torch.equal(q, want) and torch.equal(*caches)
    with pytest.raises(pkv.PkvError, match="PKV_ERR_OVERLAP"):
        pkv.pkv_append_rotary(q, k, v, pos, table, slots, caches[1], interleaved=interleaved, q_out=qkv[:, d:17 * d].view(tokens, 16, d))


def test_two_graphs_on_one_workspace(pkv):
    """Captured calls of different sizes that share a workspace, replayed in turn on one stream."""
    sizes = [([2000, 40], [1, 1]), ([700], [4]), ([500, 900], [90, 30])]
    cases = [make(6 + i, lens, news, 8, 2, 128, width=130) for i, (lens, news) in enumerate(sizes)]
    need = max(pkv.pkv_multiquery_q4_workspace_size(len(c["news"]), 8, 130, max(c["news"]), c["cache"]) for c in cases)
    work = torch.zeros(need, dtype=torch.uint8, device="cuda")
    wants = [reference(c) for c in cases]
    graphs, outs = [], []

    def call(c, out):
        return pkv.pkv_multiquery_attention_q4(c["q"], c["cache"], c["tables"], c["lens"], c["start"], c["scale"], max(c["news"]),
                                               out=out, workspace=work)
    for c in cases:
        out = torch.zeros_like(c["q"])
        call(c, out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(c, out)
        graphs.append(graph)
        outs.append(out)
    for order in ((0, 1, 2), (2, 0, 1), (1, 1, 2, 2, 0, 0)):
        for i in order:
            outs[i].zero_()
            graphs[i].replay()
        for out, want in zip(outs, wants):
            check(out, *want)
    for c, (want, bound) in zip(cases, wants):
        check(call(c, None), want, bound)


def test_every_call_on_another_stream(pkv):
    """Inputs that become ready on the stream late; outputs that the calls allocate are ready there, and usable on the
    caller's stream once it waits."""
    d, kv, heads, tokens, batch = 128, 2, 8, 600, 5
    g = torch.Generator(device="cuda").manual_seed(9)
    qkv = torch.randn((tokens, (heads + 2 * kv) * d), device="cuda", generator=g).to(torch.bfloat16)
    f = pkv.pkv_rotary_frequencies(d).cuda()
    lens0, held0 = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(2))
    new = torch.full((batch,), tokens // batch, dtype=torch.int32, device="cuda")
    free, left = torch.arange(60, dtype=torch.int32, device="cuda"), torch.tensor([60], dtype=torch.int32, device="cuda")

    def steps(rows, tables, cache, **kw):
        q, k, v = (x.view(tokens, -1, d) for x in (rows[:, :heads * d], rows[:, heads * d:(heads + kv) * d], rows[:, (heads + kv) * d:]))
        table = pkv.pkv_rotary_table(f, 200, **kw)
        slots, pos, start, lens, held, count, result = pkv.pkv_plan_step(lens0, new, held0, free, left, tables, tokens, **kw)
        turned = pkv.pkv_append_rotary(q, k, v, pos, table, slots, cache, **kw)
        out = pkv.pkv_multiquery_attention_q4(turned, cache, tables, lens, start, 0.1, tokens // batch, **kw)
        one = pkv.pkv_decode_attention_q4(turned[:batch], cache, tables, lens, 0.1, **kw)
        return [table, slots, pos, start, lens, held, count, result, turned, out, one, *pkv.pkv_gather_q4(cache, tables, lens, start, tokens, **kw)]

    fresh = lambda: (torch.full((batch, 10), -1, dtype=torch.int32, device="cuda"),  # noqa: E731
                     torch.zeros((60, kv, Q.record_bytes(d)), dtype=torch.uint8, device="cuda"))
    want = steps(qkv, *fresh())
    side = torch.cuda.Stream()
    late, tables_cache = torch.zeros_like(qkv), fresh()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            late.zero_()
            torch.cuda._sleep(2_000_000)
            late.copy_(qkv)
            tables_cache[0].fill_(-1)
            tables_cache[1].zero_()
        got = steps(late, *tables_cache, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        side.wait_stream(torch.cuda.current_stream())
