"""Rotary positions on the GPU: the table within its stated bound of float64, the turned
rows and what a quantizing cache makes of them bit for bit."""

import numpy as np
import pytest
import torch

from oracle import quant4 as Q
from oracle import rotary as R
from oracle.quant import quantize_rows

pytestmark = pytest.mark.gpu
B = 16


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("dim", [2, 6, 10, 32, 64, 128, 514])
@pytest.mark.parametrize("positions,first", [(1, 0), (7, 0), (1000, 0), (333, 1 << 20), (5, (1 << 31) - 6)])
def test_table(pkv, dim, positions, first):
    f = torch.from_numpy(R.frequencies(dim, 10000.0))
    f[0] = 2.5                                              # more than a radian a position
    if dim > 2:
        f[1] = -0.3
    got = pkv.pkv_rotary_table(f.cuda(), positions, first, 1.25).double().cpu().numpy()
    want = R.table(f.numpy(), np.arange(first, first + positions), 1.25)
    # 2^-22 of the factor, and float64's angle itself: p f and p (f / 2 pi) are each off by 2^-53 of themselves
    angle = np.arange(first, first + positions)[:, None] * np.abs(np.concatenate([f, f]))
    assert np.all(np.abs(got - want) <= 1.25 * (2.0 ** -22 + angle * 2.0 ** -51))


def test_table_rows_do_not_depend_on_the_call(pkv):
    f = torch.from_numpy(R.frequencies(96, 500000.0)).cuda()
    whole = pkv.pkv_rotary_table(f, 5000)
    assert torch.equal(pkv.pkv_rotary_table(f, 1234, 3000), whole[3000:4234])
    assert pkv.pkv_rotary_table(f, 0).shape == (0, 96)


def inputs(seed, tokens, heads, kv, d, dtype, size=1.0, positions=500):
    """q, k and v as parts of one product, positions (any order, the same twice) and slots."""
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((tokens, (heads + 2 * kv) * d + 8), generator=g) * size).to(dtype).cuda()
    part = lambda a, n: qkv[:, a * d:(a + n) * d].view(tokens, n, d)  # noqa: E731
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, positions, tokens).astype(np.int32)
    blocks = tokens // B + 3
    slots = rng.permutation(blocks * B)[:tokens].astype(np.int64)
    if tokens > 3:
        slots[2] = -1
        pos[1] = pos[0]
    return part(0, heads), part(heads, kv), part(heads + kv, kv), pos, slots, blocks


def bf16_of(x):
    return torch.from_numpy(np.ascontiguousarray(x)).float().to(torch.bfloat16)


SHAPES = [(32, 8, 128, 128), (3, 1, 128, 64), (4, 4, 64, 64), (5, 1, 64, 16), (0, 2, 128, 96), (2, 2, 128, 20), (2, 1, 64, 2),
          (6, 3, 128, 126)]


@pytest.mark.parametrize("heads,kv,d,R_", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens", [1, 37, 300])
@pytest.mark.parametrize("cache", ["bf16", "q8", "q4"])
def test_append_bit_exact(pkv, heads, kv, d, R_, interleaved, tokens, cache):
    q, k, v, pos, slots, blocks = inputs(tokens + R_, tokens, heads, kv, d, torch.bfloat16)
    table = pkv.pkv_rotary_table(torch.from_numpy(R.frequencies(R_, 10000.0)).cuda(), 500, factor=1.1)
    rows = table.double().cpu().numpy()[pos]
    turned = [bf16_of(R.turn(x.double().cpu().numpy(), rows, interleaved)) for x in (q, k)]
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    args = (q if heads else None, k, v, dev(pos), table, dev(slots))
    live = np.flatnonzero(slots >= 0)
    at = slots[live]
    if cache == "bf16":
        pools = [torch.full((blocks, kv, B, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        want = [p.clone().cpu() for p in pools]
        for p, x in zip(want, (turned[1], v.cpu())):
            p[at // B, :, at % B] = x[live]
    elif cache == "q8":
        pools = [torch.full((blocks, kv, B, d), 3, dtype=torch.int8, device="cuda"),
                 torch.full((blocks, kv, d, B), 3, dtype=torch.int8, device="cuda"),
                 torch.full((blocks, kv, 2, B), 0.5, device="cuda")]
        want = [p.clone().cpu() for p in pools]
        for side, x in enumerate((turned[1], v.cpu())):
            codes, scales = (torch.from_numpy(a) for a in quantize_rows(x.double().numpy()))
            (want[0] if side == 0 else want[1].transpose(2, 3))[at // B, :, at % B] = codes[live]
            want[2][at // B, :, side, at % B] = scales[live]
    else:
        rng = np.random.default_rng(1)
        before = rng.integers(0, 256, (blocks, kv, Q.record_bytes(d)), dtype=np.uint8)
        pools = [dev(before.copy())]
        Q.append_tokens_q4(before, turned[1].double().numpy(), v.double().cpu().numpy(), slots)
        want = [torch.from_numpy(before)]
    start = [p.clone() for p in pools]
    got = pkv.pkv_append_rotary(*args, *pools, interleaved=interleaved)
    for p, w in zip(pools, want):
        assert torch.equal(p.cpu(), w)
    if heads:
        assert torch.equal(got.cpu(), turned[0])
        # in place, into the product's own memory, checked
        again = pkv.pkv_append_rotary(*args, *start, interleaved=interleaved, q_out=q, flags=pkv.PKV_FLAG_CHECKED)
        assert again is q and torch.equal(q, got)
        for p, w in zip(start, pools):
            assert torch.equal(p, w)
    else:
        assert got is None


@pytest.mark.parametrize("heads,kv,d,R_", SHAPES[:6])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_f32(pkv, heads, kv, d, R_, interleaved):
    q, k, v, pos, slots, blocks = inputs(5, 53, heads, kv, d, torch.float32)
    table = pkv.pkv_rotary_table(torch.from_numpy(R.frequencies(R_, 10000.0)).cuda(), 500)
    rows = table.double().cpu().numpy()[pos]
    pools = [torch.zeros((blocks, kv, B, d), device="cuda") for _ in range(2)]
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    got = pkv.pkv_append_rotary(q if heads else None, k, v, dev(pos), table, dev(slots), *pools, interleaved=interleaved)
    live = np.flatnonzero(slots >= 0)
    at = torch.from_numpy(slots[live])
    out = [(pools[0].cpu()[at // B, :, at % B], k[live])] + ([(got.cpu(), q)] if heads else [])
    for y, x in out:
        x = x.double().cpu().numpy()
        use = rows if y.shape[0] == len(pos) else rows[live]
        want = R.turn(x, use, interleaved)
        size = R.turn(np.abs(x), np.concatenate([np.abs(use[:, :R_ // 2]), -np.abs(use[:, R_ // 2:])], 1), interleaved)
        other = R.turn(np.abs(x), np.abs(use), interleaved)  # |x_a c| + |x_b s|, whichever sign the pair takes
        assert np.all(np.abs(y.double().numpy() - want) <= 2.0 ** -23 * np.maximum(np.abs(size), np.abs(other)) + 1e-45)
    assert torch.equal(pools[1].cpu()[at // B, :, at % B], v[live].cpu())


@pytest.mark.parametrize("size", [1e-38, 1e-30, 3e37])
def test_sizes(pkv, size):
    """Values at the ends of the float range: rounded once, and quantized from there."""
    q, k, v, pos, slots, blocks = inputs(9, 40, 4, 2, 128, torch.bfloat16, size)
    table = pkv.pkv_rotary_table(torch.from_numpy(R.frequencies(128, 10000.0)).cuda(), 500)
    rows = table.double().cpu().numpy()[pos]
    cache = torch.zeros((blocks, 2, Q.record_bytes(128)), dtype=torch.uint8, device="cuda")
    got = pkv.pkv_append_rotary(q, k, v, torch.from_numpy(pos).cuda(), table, torch.from_numpy(slots).cuda(), cache)
    turned = [bf16_of(R.turn(x.double().cpu().numpy(), rows, False)) for x in (q, k)]
    assert torch.equal(got.cpu(), turned[0])
    want = np.zeros(cache.shape, np.uint8)
    Q.append_tokens_q4(want, turned[1].double().numpy(), v.double().cpu().numpy(), slots)
    assert np.array_equal(cache.cpu().numpy(), want)


def test_nan_and_infinity_stay_in_their_pair(pkv):
    q, k, v, pos, slots, blocks = inputs(10, 8, 2, 1, 64, torch.bfloat16)
    table = pkv.pkv_rotary_table(torch.from_numpy(R.frequencies(64, 10000.0)).cuda(), 500)
    pools = [torch.zeros((blocks, 1, B, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    clean = pkv.pkv_append_rotary(q, k, v, dev(pos), table, dev(slots), *pools)
    q = q.clone()
    q[3, 1, 5] = float("nan")
    q[4, 0, 40] = float("inf")
    got = pkv.pkv_append_rotary(q, k, v, dev(pos), table, dev(slots), *pools)
    assert got[3, 1, [5, 37]].isnan().all() and not got[4, 0, [8, 40]].isfinite().any()
    same = torch.ones_like(got, dtype=torch.bool)
    same[3, 1, [5, 37]] = False
    same[4, 0, [8, 40]] = False
    assert torch.equal(got[same], clean[same])


@pytest.mark.parametrize("cache", ["bf16", "q4"])
def test_bad_positions_and_padding(pkv, cache):
    q, k, v, pos, slots, blocks = inputs(11, 20, 4, 2, 64, torch.bfloat16)
    table = pkv.pkv_rotary_table(torch.from_numpy(R.frequencies(64, 10000.0)).cuda(), 500)
    make = (lambda: [torch.zeros((blocks, 2, Q.record_bytes(64)), dtype=torch.uint8, device="cuda")]) if cache == "q4" else \
        (lambda: [torch.zeros((blocks, 2, B, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)])
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    keep, whole = torch.full((20, 4, 64), 2.0, dtype=torch.bfloat16, device="cuda"), make()
    full = pkv.pkv_append_rotary(q, k, v, dev(pos), table, dev(slots), *whole)
    padded, pslots, pools = pos.copy(), slots.copy(), make()
    padded[15:] = -1
    pslots[15:] = -1
    pkv.pkv_append_rotary(q, k, v, dev(padded), table, dev(pslots), *pools, q_out=keep, flags=pkv.PKV_FLAG_CHECKED)
    assert torch.equal(keep[:15], full[:15]) and torch.equal(keep[15:], torch.full_like(keep[15:], 2.0))
    first = make()
    pkv.pkv_append_rotary(None, k[:15], v[:15], dev(pos[:15]), table, dev(slots[:15]), *first)
    assert all(torch.equal(a, b) for a, b in zip(pools, first))
    for p, s in ((500, 3), (-1, 3), (1 << 30, -1), (4, blocks * B)):
        bad, bslots, pools, out = pos.copy(), slots.copy(), make(), torch.full_like(keep, 2.0)
        bad[15:], bslots[15:] = p, -1
        bslots[15] = s
        before = [x.clone() for x in pools]
        with pytest.raises(pkv.PkvError, match="PKV_ERR_RANGE"):
            pkv.pkv_append_rotary(q, k, v, dev(bad), table, dev(bslots), *pools, q_out=out, flags=pkv.PKV_FLAG_CHECKED)
        assert torch.equal(out, torch.full_like(out, 2.0)) and all(torch.equal(a, b) for a, b in zip(pools, before))
        if p == -1:
            bslots[16:] = -1
        pkv.pkv_append_rotary(q, k, v, dev(bad), table, dev(bslots), *pools, q_out=out)
        assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
        assert torch.equal(out[:15], full[:15]) and all(torch.equal(a, b) for a, b in zip(pools, first))
        if p != 4:
            assert torch.equal(out[15:], torch.full_like(out[15:], 2.0))


def test_strides_and_refusals(pkv):
    q, k, v, pos, slots, blocks = inputs(12, 6, 4, 2, 64, torch.bfloat16)
    table = pkv.pkv_rotary_table(torch.from_numpy(R.frequencies(64, 10000.0)).cuda(), 500)
    pools = [torch.zeros((blocks, 2, B, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    want = pkv.pkv_append_rotary(q, k, v, dev(pos), table, dev(slots), *pools)
    wide = torch.zeros((6, 9, 64), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_append_rotary(q.contiguous(), k.contiguous(), v, dev(pos), table, dev(slots), *pools, q_out=wide[:, 3:7])
    assert torch.equal(wide[:, 3:7], want) and not wide[:, :3].any() and not wide[:, 7:].any()
    back = q.flip(0)                                        # (a copy: torch has no negative strides)
    with pytest.raises(ValueError):
        pkv.pkv_append_rotary(back.transpose(1, 2).contiguous().transpose(1, 2), k, v, dev(pos), table, dev(slots), *pools)
    with pytest.raises(ValueError):
        pkv.pkv_append_rotary(q.float(), k, v, dev(pos), table, dev(slots), *pools)
    with pytest.raises(ValueError):
        pkv.pkv_append_rotary(q, k, v, dev(pos)[:5], table, dev(slots), *pools)
    with pytest.raises(ValueError):
        pkv.pkv_append_rotary(q, k, v, dev(pos), table.double(), dev(slots), *pools)
    with pytest.raises(pkv.PkvError, match="PKV_ERR_SHAPE"):
        pkv.pkv_append_rotary(q, k, v, dev(pos), torch.zeros((500, 66), device="cuda"), dev(slots), *pools)
    with pytest.raises(pkv.PkvError, match="PKV_ERR_ALIGN"):
        odd = torch.zeros((6, 4 * 64 + 3), dtype=torch.bfloat16, device="cuda")[:, :256].view(6, 4, 64)
        pkv.pkv_append_rotary(odd, k, v, dev(pos), table, dev(slots), *pools)
    none = pkv.pkv_append_rotary(q[:0], k[:0], v[:0], dev(pos)[:0], table, dev(slots)[:0], *pools)
    assert none.shape == (0, 4, 64)
