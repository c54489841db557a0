"""Rows that hold a NaN or an infinity in the quantizing appends: such a row's scale is NaN, so that it reads back as
nothing but NaN and spoils the attention rows that see it; every other row is what it is without them. Calls of few
rows and of many (where V's blocks are put together 16 tokens at a time) both."""

import math

import numpy as np
import pytest
import torch

from oracle import quant4 as Q
from oracle.quant import quantize_rows
from q4_cases import check, reference

pytestmark = pytest.mark.gpu
B = 16


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def spoil(k, v):
    """Some elements of some rows: in the lanes' first and last vectors, alone and beside larger numbers, whole rows.
    Returns which (token, head) rows of k and of v are spoilt."""
    tokens, kv, d = k.shape
    marks = [torch.zeros((tokens, kv), dtype=torch.bool) for _ in range(2)]
    bad = [math.nan, math.inf, -math.inf, -math.nan]
    for side, (x, mark) in enumerate(zip((k, v), marks)):
        for n, t in enumerate(range(1 + side, tokens, 7)):
            h = (n + side) % kv
            x[t, h, [0, d - 1, d // 2, 9][n % 4]] = bad[n % 4]
            if n % 3 == 0:
                x[t, h, 3] = 3e38
            if n % 5 == 0:
                x[t, h] = bad[(n // 5) % 4]
            mark[t, h] = True
    return marks


def pools_of(cache, blocks, kv, d):
    if cache == "q4":
        return [torch.full((blocks, kv, Q.record_bytes(d)), 0x35, dtype=torch.uint8, device="cuda")]
    return [torch.full((blocks, kv, B, d), 3, dtype=torch.int8, device="cuda"),
            torch.full((blocks, kv, d, B), 3, dtype=torch.int8, device="cuda"),
            torch.full((blocks, kv, 2, B), 0.5, device="cuda")]


def contents(cache, pools, kv, d):
    """(K codes, V codes, K scales, V scales), the slots of the pool one after another."""
    host = [p.cpu().numpy() for p in pools]
    flat = lambda x: np.moveaxis(x, 1, 2).reshape(-1, kv, *x.shape[3:])  # noqa: E731
    if cache == "q4":
        return [flat(x) for x in Q.unpack(host[0], d)]
    return [flat(host[0]), flat(host[1].swapaxes(2, 3)), flat(host[2][:, :, 0]), flat(host[2][:, :, 1])]


@pytest.mark.parametrize("cache", ["q4", "q8"])
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("tokens,kv,d", [(1, 1, 128), (20, 2, 64), (33, 3, 128), (2000, 4, 128), (3333, 3, 64)])
@pytest.mark.parametrize("step", [1, 3])
def test_codes_and_scales(pkv, cache, turned, tokens, kv, d, step):
    """`step` 1: slots that follow one another; 3: apart, so that V goes byte by byte."""
    g = torch.Generator().manual_seed(tokens)
    k, v = (torch.randn((tokens, kv, d), generator=g).to(torch.bfloat16) for _ in range(2))
    clean = k.clone(), v.clone()
    marks = spoil(k, v)
    if tokens == 1:
        k[0, 0, 5], marks[0][0, 0] = math.nan, True
        v[0, 0, 77], marks[1][0, 0] = math.inf, True
    blocks = tokens * step // B + 2
    slots = torch.arange(tokens, device="cuda") * step
    pools = pools_of(cache, blocks, kv, d)
    if turned:
        # position 0 turns nothing: c = 1, s = 0 (and infinity times 0 is not a number, in the other half of its pair)
        table = pkv.pkv_rotary_table(pkv.pkv_rotary_frequencies(d).cuda(), 4)
        pkv.pkv_append_rotary(None, k.cuda(), v.cuda(), torch.zeros(tokens, dtype=torch.int32, device="cuda"), table, slots, *pools)
    elif cache == "q4":
        pkv.pkv_append_q4(k.cuda(), v.cuda(), slots, *pools)
    else:
        pkv.pkv_append_q8(k.cuda(), v.cuda(), slots, *pools)
    found = contents(cache, pools, kv, d)
    at = slots.cpu().numpy()
    for side, (x, mark) in enumerate(zip(clean, marks)):
        codes, scales = (Q.quantize_rows4 if cache == "q4" else quantize_rows)(x.double().numpy())
        bad = mark.numpy()
        scales[bad] = np.nan
        assert np.array_equal(found[side][at][~bad], codes[~bad])
        assert np.array_equal(found[2 + side][at], scales, equal_nan=True)


def test_oracles_agree_with_the_statement():
    x = np.array([[1.0, -2.0, 0.5], [1.0, np.nan, 3.0], [np.inf, 1.0, 0.0], [0.0, 0.0, -np.inf]])
    for quantize, largest in ((Q.quantize_rows4, 7), (quantize_rows, 127)):
        codes, scales = quantize(x)
        assert np.abs(codes[0]).max() == largest and np.isfinite(scales[0])
        assert np.isnan(scales[1:]).all()


@pytest.mark.parametrize("cache", ["q4", "q8"])
@pytest.mark.parametrize("tokens", [40, 2000])
def test_reading_back(pkv, cache, tokens):
    kv, d = 2, 128
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((tokens, kv, d), generator=g).to(torch.bfloat16) for _ in range(2))
    marks = spoil(k, v)
    pools = pools_of(cache, tokens // B + 2, kv, d)
    slots = torch.arange(tokens, device="cuda")
    (pkv.pkv_append_q4 if cache == "q4" else pkv.pkv_append_q8)(k.cuda(), v.cuda(), slots, *pools)
    tables = torch.arange(tokens // B + 2, dtype=torch.int32, device="cuda")[None].contiguous()
    lens, start = (torch.tensor(n, dtype=torch.int32, device="cuda") for n in ([tokens], [0, tokens]))
    for dtype in (torch.bfloat16, torch.float32):
        read = (pkv.pkv_gather_q4 if cache == "q4" else pkv.pkv_gather_q8)(*pools, tables, lens, start, tokens, out_dtype=dtype)
        for x, mark in zip(read, marks):
            nan = x.isnan().cpu()
            assert torch.equal(nan.all(-1), mark) and torch.equal(nan.any(-1), mark) and x.cpu()[~mark].isfinite().all()


# rows of a KV head: 4 and 16 on the kernel that splits the cache, 160 in tiles
@pytest.mark.parametrize("new", [1, 4, 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("where", [3, 250, 298, 299])
def test_attention_over_the_4_bit_cache(pkv, new, d, side, bad, where):
    """One head's token is spoilt: the rows of that head that see it are no numbers, all others are as without it."""
    n, kv, heads = 300, 2, 8
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn((n, kv, d), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((new, heads, d), device="cuda", generator=g).to(torch.bfloat16)
    slots = torch.arange(n, device="cuda")
    tables = torch.arange(n // B + 1, dtype=torch.int32, device="cuda")[None].contiguous()
    lens, start = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([n], [0, new]))

    def append():
        cache = torch.zeros((n // B + 1, kv, Q.record_bytes(d)), dtype=torch.uint8, device="cuda")
        pkv.pkv_append_q4(k, v, slots, cache)
        return cache
    case = dict(cache=append(), tables=tables, lens=lens, start=start, q=q, scale=0.1, lens_list=[n], news=[new], d=d)
    want, bound = reference(case)
    (k if side == "k" else v)[where, 1, 17] = bad
    got = pkv.pkv_multiquery_attention_q4(q, append(), tables, lens, start, 0.1, new)
    sees = torch.zeros((new, heads), dtype=torch.bool, device="cuda")
    sees[max(0, where - (n - new)):, heads // 2:] = True
    assert got[sees].isnan().all()
    check(got[~sees], want[~sees], bound[~sees])


SIZES = [(1, 300), (4, 300), (8, 303), (4, 40000)]


@pytest.mark.parametrize("call,new,n", [("decode_q8", *s) for s in SIZES] + [("multiquery_q8", *s) for s in SIZES + [(40, 300)]])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("back", [1, 2, 50, 297])
def test_attention_over_int8_pools(pkv, call, new, n, side, bad, back):
    """The same over int8 pools, 40000 tokens on the kernel that splits the cache: a spoilt token `back` from the end."""
    kv, heads, d, where = 2, 8, 128, n - back
    g = torch.Generator(device="cuda").manual_seed(6)
    k, v = (torch.randn((n, kv, d), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((new, heads, d), device="cuda", generator=g).to(torch.bfloat16)
    slots = torch.arange(n, device="cuda")
    tables = torch.arange(n // B + 1, dtype=torch.int32, device="cuda")[None].contiguous()
    lens, start = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([n], [0, new]))

    def attend():
        pools = [torch.zeros((n // B + 1, kv, B, d), dtype=torch.int8, device="cuda"),
                 torch.zeros((n // B + 1, kv, d, B), dtype=torch.int8, device="cuda"), torch.zeros((n // B + 1, kv, 2, B), device="cuda")]
        pkv.pkv_append_q8(k, v, slots, *pools)
        if call == "decode_q8":
            return pkv.pkv_decode_attention_q8(q, *pools, tables, lens, 0.1, query_start=start, max_query_len=new)
        return pkv.pkv_multiquery_attention_q8(q, *pools, tables, lens, start, 0.1, new)
    want = attend()
    (k if side == "k" else v)[where, 1, 17] = bad
    got = attend()
    sees = torch.zeros((new, heads), dtype=torch.bool, device="cuda")
    sees[max(0, where - (n - new)):, heads // 2:] = True
    assert got[sees].isnan().all()
    # each is off by half a bf16 step and by its f16 weights, 2^-11 of an average of |v| (below 1 here): twice both
    assert ((got[~sees].double() - want[~sees].double()).abs() <= 2 * (want[~sees].double().abs() * 2.0 ** -8 + 4 * 2.0 ** -11)).all()
