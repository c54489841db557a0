"""Appends of many rows into quantizing caches, where V's blocks are put together 16 tokens at a time: the same bytes as
the same rows appended in small calls (which tests/test_gpu_rotary.py and tests/test_gpu_q4.py hold to the oracle),
whatever the order and gaps of the slots."""

import numpy as np
import pytest
import torch

from oracle import quant4 as Q

pytestmark = pytest.mark.gpu
B = 16


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def slots_of(kind, tokens, blocks, seed):
    """Slots of `tokens` rows in `blocks` blocks (distinct, -1 among them in some kinds)."""
    rng = np.random.default_rng(seed)
    order = rng.permutation(blocks)
    place = lambda t: order[t // B] * B + t % B  # noqa: E731
    if kind == "aligned":
        return place(np.arange(tokens))
    if kind == "shifted":                                   # a prompt that goes on in the middle of a block
        return place(np.arange(tokens) + 5)
    if kind == "ragged":                                    # sequences of odd lengths, each from its block's first slot on or not
        out, at, block = [], 0, 0
        while at < tokens:
            n, first = int(rng.integers(1, 70)), int(rng.choice([0, 0, 3, 15]))
            n = min(n, tokens - at)
            out.append(place(block * B + first + np.arange(n)))
            block += -(-(first + n) // B)
            at += n
        return np.concatenate(out)
    if kind == "holes":                                     # padding inside runs
        s = place(np.arange(tokens))
        s[rng.random(tokens) < 0.02] = -1
        return s
    if kind == "backwards":
        return place(np.arange(tokens))[::-1].copy()
    if kind == "scattered":
        return rng.permutation(blocks * B)[:tokens]
    if kind == "swapped":                                   # runs of 16 in which two tokens have changed places
        s = place(np.arange(tokens))
        at = np.arange(0, tokens - B, 3 * B) + 4
        s[at], s[at + 7] = s[at + 7], s[at].copy()
        return s
    raise ValueError(kind)


def pools_of(cache, blocks, kv, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if cache == "q4":
        return [torch.randint(0, 256, (blocks, kv, Q.record_bytes(d)), dtype=torch.uint8, device="cuda", generator=g)]
    return [torch.randint(-128, 128, (blocks, kv, B, d), dtype=torch.int8, device="cuda", generator=g),
            torch.randint(-128, 128, (blocks, kv, d, B), dtype=torch.int8, device="cuda", generator=g),
            torch.rand((blocks, kv, 2, B), device="cuda", generator=g)]


@pytest.mark.parametrize("kind", ["aligned", "shifted", "ragged", "holes", "backwards", "scattered", "swapped"])
@pytest.mark.parametrize("cache", ["q4", "q8"])
@pytest.mark.parametrize("heads,kv,d,rotary,interleaved", [(16, 8, 128, 128, False), (8, 1, 128, 64, True), (6, 3, 64, 64, False)])
def test_same_bytes_as_small_calls(pkv, kind, cache, heads, kv, d, rotary, interleaved):
    tokens, small = 1333, 130                               # 13330 to 42656 rows at once, at most 4160 a small call
    blocks = 2 * tokens // B + 200
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((tokens, (heads + 2 * kv) * d), device="cuda", generator=g).to(torch.bfloat16)
    q, k, v = (x.view(tokens, -1, d) for x in (qkv[:, :heads * d], qkv[:, heads * d:(heads + kv) * d], qkv[:, (heads + kv) * d:]))
    slots = torch.from_numpy(np.ascontiguousarray(slots_of(kind, tokens, blocks, 2)).astype(np.int64)).cuda()
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda") % 900
    if kind == "holes":
        pos[slots < 0] = -1
    table = pkv.pkv_rotary_table(pkv.pkv_rotary_frequencies(rotary).cuda(), 900)
    whole, parts = pools_of(cache, blocks, kv, d, 3), pools_of(cache, blocks, kv, d, 3)
    out = pkv.pkv_append_rotary(q, k, v, pos, table, slots, *whole, interleaved=interleaved, q_out=torch.zeros_like(q).contiguous())
    for a in range(0, tokens, small):
        b = min(a + small, tokens)
        few = pkv.pkv_append_rotary(q[a:b], k[a:b], v[a:b], pos[a:b], table, slots[a:b], *parts, interleaved=interleaved,
                                    q_out=torch.zeros_like(q[a:b]).contiguous())
        assert torch.equal(out[a:b], few)
    for x, y in zip(whole, parts):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("kind", ["aligned", "ragged", "scattered"])
@pytest.mark.parametrize("kv,d", [(8, 128), (3, 64)])
def test_without_positions(pkv, kind, kv, d):
    tokens, small = 4000, 300
    blocks = 2 * tokens // B + 200
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn((tokens, kv, d), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    v[5::7] = 0                                             # rows of nothing
    slots = torch.from_numpy(np.ascontiguousarray(slots_of(kind, tokens, blocks, 5)).astype(np.int64)).cuda()
    whole, parts = pools_of("q4", blocks, kv, d, 6), pools_of("q4", blocks, kv, d, 6)
    pkv.pkv_append_q4(k, v, slots, *whole)
    for a in range(0, tokens, small):
        pkv.pkv_append_q4(k[a:a + small], v[a:a + small], slots[a:a + small], *parts)
    assert torch.equal(whole[0], parts[0])


@pytest.mark.parametrize("cache", ["q4", "q8"])
def test_bad_rows_in_the_middle_of_a_block(pkv, cache):
    """A slot past the pool, or a position past the table, inside a run of 16: that token alone is left out."""
    tokens, kv, d, heads = 1400, 2, 128, 8
    blocks = tokens // B + 1
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = (torch.randn((tokens, h, d), device="cuda", generator=g).to(torch.bfloat16) for h in (heads, kv, kv))
    slots, pos = torch.arange(tokens, device="cuda"), torch.arange(tokens, dtype=torch.int32, device="cuda")
    table = pkv.pkv_rotary_table(pkv.pkv_rotary_frequencies(d).cuda(), tokens)
    wrong = slots.clone()
    wrong[[7, 40]] = blocks * B + 3
    far = pos.clone()
    far[[100, 127]] = tokens
    got, want = pools_of(cache, blocks, kv, d, 8), pools_of(cache, blocks, kv, d, 8)
    pkv.pkv_append_rotary(q, k, v, far, table, wrong, *got)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
    keep = torch.ones(tokens, dtype=torch.bool, device="cuda")
    keep[[7, 40, 100, 127]] = False
    at = torch.nonzero(keep).flatten()
    for a in range(0, len(at), 400):
        i = at[a:a + 400]
        pkv.pkv_append_rotary(q[i], k[i], v[i], pos[i], table, slots[i], *want)
    for x, y in zip(got, want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("cache", ["q4", "q8"])
def test_checked_calls_refuse_a_slot_named_twice(pkv, cache):
    tokens, kv, d, heads = 1400, 2, 128, 8
    q, k, v = (torch.zeros((tokens, h, d), dtype=torch.bfloat16, device="cuda") for h in (heads, kv, kv))
    slots, pos = torch.arange(tokens, device="cuda"), torch.arange(tokens, dtype=torch.int32, device="cuda")
    table = pkv.pkv_rotary_table(pkv.pkv_rotary_frequencies(d).cuda(), tokens)
    pools, before = pools_of(cache, tokens // B + 1, kv, d, 9), pools_of(cache, tokens // B + 1, kv, d, 9)
    slots[1000] = 17
    with pytest.raises(pkv.PkvError, match="PKV_ERR_OVERLAP"):
        pkv.pkv_append_rotary(q, k, v, pos, table, slots, *pools, flags=pkv.PKV_FLAG_CHECKED)
    slots[1000] = 1000
    pos[999] = tokens
    with pytest.raises(pkv.PkvError, match="PKV_ERR_RANGE"):
        pkv.pkv_append_rotary(q, k, v, pos, table, slots, *pools, flags=pkv.PKV_FLAG_CHECKED)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(pools, before))
    pos[999] = 999
    pkv.pkv_append_rotary(q, k, v, pos, table, slots, *pools, flags=pkv.PKV_FLAG_CHECKED)


@pytest.mark.parametrize("cache", ["q4", "q8"])
def test_captured(pkv, cache):
    """A captured append of many rows, replayed on other values and slots."""
    tokens, kv, d, heads = 1500, 2, 128, 6
    blocks = 2 * tokens // B + 200
    g = torch.Generator(device="cuda").manual_seed(10)
    rows = torch.randn((tokens, (heads + 2 * kv) * d), device="cuda", generator=g).to(torch.bfloat16)
    q, k, v = (x.view(tokens, -1, d) for x in (rows[:, :heads * d], rows[:, heads * d:(heads + kv) * d], rows[:, (heads + kv) * d:]))
    slots = torch.from_numpy(slots_of("ragged", tokens, blocks, 11).astype(np.int64)).cuda()
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    table = pkv.pkv_rotary_table(pkv.pkv_rotary_frequencies(d).cuda(), tokens)
    captured, eager = pools_of(cache, blocks, kv, d, 12), pools_of(cache, blocks, kv, d, 12)
    out = torch.zeros((tokens, heads, d), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.pkv_append_rotary(q, k, v, pos, table, slots, *captured, q_out=out)
    for seed in (13, 14):
        rows.normal_()
        slots.copy_(torch.from_numpy(slots_of("ragged", tokens, blocks, seed).astype(np.int64)))
        graph.replay()
        want = pkv.pkv_append_rotary(q, k, v, pos, table, slots, *eager)
        assert torch.equal(out, want)
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(captured, eager))
