"""The 4-bit cache on the GPU: append, copy and reading back bit for bit, attention
within derived bounds of float64 (tests/q4_cases.py)."""

import numpy as np
import pytest
import torch

from oracle import quant4 as Q
from q4_cases import B, check, fast_pack, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def test_fast_pack_is_pack():
    rng = np.random.default_rng(0)
    for d in (64, 128):
        kc, vc = rng.integers(-8, 8, (2, 2, 3, 16, d)).astype(np.int8)
        ks, vs = rng.random((2, 2, 3, 16)).astype(np.float32)
        assert np.array_equal(fast_pack(kc, vc, ks, vs), Q.pack(kc, vc, ks, vs))


def rows_bf16(seed, shape, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * size).to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", [1, 3, 8])
@pytest.mark.parametrize("tokens", [1, 5, 67])
@pytest.mark.parametrize("size", [1.0, 1e-37, 1e-30, 1e37])
def test_append_bit_exact(pkv, d, kv, tokens, size):
    blocks = 9
    rng = np.random.default_rng(tokens)
    before = rng.integers(0, 256, (blocks, kv, Q.record_bytes(d)), dtype=np.uint8)
    slots = rng.permutation(blocks * B)[:tokens].astype(np.int64)
    if tokens > 2:
        slots[1] = -1
    k, v = rows_bf16(1, (tokens, kv, d), size), rows_bf16(2, (tokens, kv, d), size)
    k[0, 0] = 0
    v[-1, -1] = 0
    v[-1, -1, 3] = -size
    cache = torch.from_numpy(before.copy()).cuda()
    pkv.pkv_append_q4(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), cache)
    want = before.copy()
    Q.append_tokens_q4(want, k.double().numpy(), v.double().numpy(), slots)
    assert np.array_equal(cache.cpu().numpy(), want)
    again = torch.from_numpy(before.copy()).cuda()
    pkv.pkv_append_q4(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), again, flags=pkv.PKV_FLAG_CHECKED)
    assert torch.equal(cache, again)


def test_append_borders(pkv):
    """Rows whose quotients lie on and next to every border: all codes by rational arithmetic."""
    d, rows = 128, 64
    base = torch.linspace(-1, 1, rows * d).reshape(rows, 1, d).to(torch.bfloat16)
    base[:, 0, 0] = 1.0
    for i in range(rows):                                   # values halfway between two codes, and their neighbours
        top = base[i, 0, 0].float()
        near = (torch.arange(-7, 7) + 0.5) * (top * torch.tensor(1.0) / 7 * (1 + i / 4096))
        base[i, 0, 1:15] = near.to(torch.bfloat16)
    cache = torch.zeros((4, 1, Q.record_bytes(d)), dtype=torch.uint8, device="cuda")
    pkv.pkv_append_q4(base.cuda(), base.cuda(), torch.arange(rows, device="cuda"), cache)
    kc, vc, ks, vs = Q.unpack(cache.cpu().numpy(), d)
    for t in range(rows):
        x = base[t, 0].float().numpy()
        want = [Q.code_exactly(e, ks[t // B, 0, t % B]) for e in x]
        assert kc[t // B, 0, t % B].tolist() == want and vc[t // B, 0, t % B].tolist() == want


def test_bad_slots(pkv):
    cache = torch.full((3, 2, Q.record_bytes(64)), 7, dtype=torch.uint8, device="cuda")
    k = rows_bf16(3, (3, 2, 64)).cuda()
    slots = torch.tensor([48, 5, 1 << 40], device="cuda")
    before = cache.clone()
    with pytest.raises(pkv.PkvError, match="PKV_ERR_RANGE"):
        pkv.pkv_append_q4(k, k, slots, cache, flags=pkv.PKV_FLAG_CHECKED)
    with pytest.raises(pkv.PkvError, match="PKV_ERR_OVERLAP"):
        pkv.pkv_append_q4(k, k, torch.tensor([4, 5, 4], device="cuda"), cache, flags=pkv.PKV_FLAG_CHECKED)
    assert torch.equal(cache, before)
    pkv.pkv_append_q4(k, k, slots, cache)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
    alone = before.clone()
    pkv.pkv_append_q4(k[1:2], k[1:2], slots[1:2], alone)
    assert torch.equal(cache, alone)


@pytest.mark.parametrize("d,kv", [(64, 1), (128, 8), (128, 3)])
def test_copy_blocks(pkv, d, kv):
    rng = np.random.default_rng(2)
    cache = torch.from_numpy(rng.integers(0, 256, (40, kv, Q.record_bytes(d)), dtype=np.uint8)).cuda()
    perm = rng.permutation(40)
    pairs = torch.from_numpy(np.stack([perm[:15], perm[15:30]], 1).astype(np.int64)).cuda()
    want = cache.clone()
    want[pairs[:, 1]] = cache[pairs[:, 0]]
    pkv.pkv_copy_blocks_q4(pairs, cache)
    assert torch.equal(cache, want)
    pkv.pkv_copy_blocks_q4(pairs[:0], cache)
    bad = torch.tensor([[0, 40], [int(perm[31]), int(perm[32])]], device="cuda")
    with pytest.raises(pkv.PkvError, match="PKV_ERR_RANGE"):
        pkv.pkv_copy_blocks_q4(bad, cache, flags=pkv.PKV_FLAG_CHECKED)
    assert torch.equal(cache, want)
    pkv.pkv_copy_blocks_q4(bad, cache)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
    want[perm[32]] = want[perm[31]]
    assert torch.equal(cache, want)


@pytest.mark.parametrize("d,kv", [(64, 2), (128, 1), (128, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gather(pkv, d, kv, dtype):
    lens, firsts = [0, 1, 16, 45, 100], [0, 0, 3, 17, 64]
    s = make(8, lens, [0] * 5, kv, kv, d)
    k, v = Q.values(s["cache"].cpu().numpy(), d)
    counts = [n - f for n, f in zip(lens, firsts)]
    start = np.concatenate([[0], np.cumsum(counts)])
    rows = int(start[-1]) + 2                               # two rows that no sequence names
    tables = s["tables"].cpu().numpy()
    for token_start in (firsts, None):
        outs = [torch.full((rows, kv, d), -3.0, dtype=dtype, device="cuda") for _ in range(2)]
        want = [torch.full((rows, kv, d), -3.0, dtype=dtype) for _ in range(2)]
        pkv.pkv_gather_q4(s["cache"], s["tables"], s["lens"], torch.from_numpy(start.astype(np.int32)).cuda(), rows,
                          token_start=None if token_start is None else torch.tensor(token_start, dtype=torch.int32, device="cuda"),
                          out_dtype=dtype, k_out=outs[0], v_out=outs[1])
        for i, n in enumerate(counts):
            for r in range(n):
                t = (firsts[i] if token_start is not None else 0) + r
                for side, pool in enumerate((k, v)):
                    want[side][start[i] + r] = torch.from_numpy(pool[tables[i, t // B], :, t % B].astype(np.float32)).to(dtype)
        for got, exp in zip(outs, want):
            assert torch.equal(got.cpu(), exp)


def run(pkv, s, decode=False, **kw):
    if decode:
        return pkv.pkv_decode_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["scale"], **kw)
    return pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["start"], s["scale"],
                                           max(1, max(s["news"])), **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (4, 4), (6, 2), (32, 8), (10, 2), (16, 2), (9, 1), (32, 1), (17, 1)])
def test_decode(pkv, d, q_heads, kv_heads):
    lens = [1, 2, 15, 16, 17, 31, 33, 200, 513]
    s = make(11, lens, [1] * 9, q_heads, kv_heads, d)
    check(run(pkv, s, decode=True), *reference(s, decode=True))


@pytest.mark.parametrize("d", [64, 128])
def test_decode_against_the_oracle(pkv, d):
    s = make(12, [0, 3, 40, 129], [1] * 4, 6, 2, d)
    got = run(pkv, s, decode=True)
    want = Q.attention_q4(s["q"].double().cpu().numpy(), s["cache"].cpu().numpy(), s["tables"].cpu().numpy(), s["lens_list"],
                          None, s["scale"])
    assert torch.equal(got[0], torch.zeros_like(got[0]))    # no tokens: a zero row
    _, bound = reference(s, decode=True)
    check(got, torch.from_numpy(want).cuda(), bound)
    with pytest.raises(pkv.PkvError, match="PKV_ERR_RANGE"):
        run(pkv, s, decode=True, flags=pkv.PKV_FLAG_CHECKED)


CHUNKS = [([1], [1]), ([40], [40]), ([17, 5, 300, 64], [3, 0, 2, 4]), ([33, 16, 500], [8, 16, 1]), ([260, 131], [200, 77]),
          ([0, 12, 0], [0, 12, 0]), ([700], [129])]


@pytest.mark.parametrize("lens,news", CHUNKS)
@pytest.mark.parametrize("q_heads,kv_heads,d", [(4, 1, 128), (6, 2, 64), (8, 8, 128), (24, 8, 128), (16, 2, 64), (33, 1, 128)])
def test_multiquery(pkv, lens, news, q_heads, kv_heads, d):
    s = make(13, lens, news, q_heads, kv_heads, d)
    out = torch.full((s["q"].shape[0], q_heads, d), 5.0, dtype=torch.bfloat16, device="cuda")
    check(run(pkv, s, out=out), *reference(s))
    if sum(news):
        checked = run(pkv, s, flags=pkv.PKV_FLAG_CHECKED)
        assert torch.equal(checked, out)


def test_rows_behind_the_last_sequence_stay(pkv):
    s = make(14, [50, 20], [3, 2], 8, 2, 128)
    q = torch.cat([s["q"], s["q"][:2]])
    out = torch.full_like(q, 9.0)
    pkv.pkv_multiquery_attention_q4(q, s["cache"], s["tables"], s["lens"], s["start"], s["scale"], 3, out=out)
    assert torch.equal(out[5:], torch.full_like(out[5:], 9.0))
    check(out[:5], *reference(s))


@pytest.mark.parametrize("news", [[1, 1], [3, 2], [90, 40]])
@pytest.mark.parametrize("d", [64, 128])
def test_absent_blocks(pkv, news, d):
    """A block whose id is out of range has no weight; a row without any token is zero."""
    s = make(15, [100, 41], news, 8, 2, d, garbage=False)
    tables = s["tables"].clone()
    tables[0, 2] = -1
    tables[1, :] = 1 << 30
    got = pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], tables, s["lens"], s["start"], s["scale"], max(news))
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
    want = torch.from_numpy(Q.attention_q4(s["q"].double().cpu().numpy(), s["cache"].cpu().numpy(), tables.cpu().numpy(),
                                           s["lens_list"], s["start"].cpu().numpy(), s["scale"])).cuda()
    assert torch.equal(got[news[0]:], torch.zeros_like(got[news[0]:]))
    _, bound = reference(s)
    check(got[:news[0]], want[:news[0]], bound[:news[0]] + want[:news[0]].abs() * 2.0 ** -8 + 0.02, mean=False)


@pytest.mark.parametrize("case", ["length", "rows", "negative", "many"])
def test_bad_lengths(pkv, case):
    s = make(16, [64, 30], [2, 2], 8, 2, 128, garbage=False)
    lens, start, out = s["lens"].clone(), s["start"].clone(), torch.full_like(s["q"], 4.0)
    if case == "length":
        lens[1] = 65
    elif case == "rows":
        start[2] = 1
    elif case == "negative":
        lens[1] = -5
    else:
        lens[1] = 1
    with pytest.raises(pkv.PkvError, match="PKV_ERR_RANGE"):
        pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], lens, start, s["scale"], 2, out=out,
                                        flags=pkv.PKV_FLAG_CHECKED)
    assert torch.equal(out, torch.full_like(out, 4.0))
    pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], lens, start, s["scale"], 2, out=out)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
    want, bound = reference(s)
    check(out[:2], want[:2], bound[:2])
