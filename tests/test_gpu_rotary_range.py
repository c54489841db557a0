"""Rotary appends at the end of the float range and past it: infinities, and products that leave the range although the
turned value does not (tables with a factor above 1)."""

import numpy as np
import pytest
import torch

from oracle import rotary as R

pytestmark = pytest.mark.gpu
B = 16
# d, R and the order of pairs: halves, neighbours, and dimensions one by one
SHAPES = [(128, 128, False), (128, 64, True), (64, 64, False), (64, 16, True), (128, 20, False), (64, 6, True)]


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def rows(seed, shape, size, infinite):
    g = torch.Generator().manual_seed(seed)
    x = (torch.rand(shape, generator=g, dtype=torch.float64) * 2 - 1) * size
    if infinite:
        at = torch.rand(shape, generator=g)
        x[at < 0.03] = float("inf")
        x[at > 0.97] = float("-inf")
        x[(at > 0.5) & (at < 0.51)] = float("nan")
        x[(at > 0.6) & (at < 0.65)] = 0.0
    return x


def call(pkv, q, k, v, pos, table, interleaved, dtype):
    tokens, kv, d = k.shape
    pools = [torch.zeros((-(-tokens // B), kv, B, d), dtype=dtype, device="cuda") for _ in range(2)]
    slots = torch.arange(tokens, device="cuda")
    out = pkv.pkv_append_rotary(q, k, v, pos, table, slots, *pools, interleaved=interleaved)
    k_out = pools[0].transpose(1, 2).reshape(-1, kv, d)[:tokens]
    v_out = pools[1].transpose(1, 2).reshape(-1, kv, d)[:tokens]
    assert torch.equal(v_out.nan_to_num(7.0, 8.0, 9.0), v.nan_to_num(7.0, 8.0, 9.0))
    return out.cpu(), k_out.cpu()


@pytest.mark.parametrize("d,rotary,interleaved", SHAPES)
@pytest.mark.parametrize("factor", [1.0, 1.5, 100.0])
@pytest.mark.parametrize("tokens", [5, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size,infinite", [(3.3e38, False), (1.0, True), (3e37, True)])
def test_against_float64(pkv, d, rotary, interleaved, factor, tokens, dtype, size, infinite):
    q, k, v = (rows(seed, (tokens, h, d), size, infinite).float().to(dtype) for seed, h in ((1, 4), (2, 2), (3, 2)))
    table = pkv.pkv_rotary_table(pkv.pkv_rotary_frequencies(rotary).cuda(), 300, factor=factor)
    pos = torch.arange(tokens, dtype=torch.int32) * 7 % 300
    got = call(pkv, q.cuda(), k.cuda(), v.cuda(), pos.cuda(), table, interleaved, dtype)
    angles = table.double().cpu().numpy()[pos.numpy()]
    half = rotary // 2
    for x, y in zip((q, k), got):
        with np.errstate(all="ignore"):
            x64 = x.double().numpy()
            want = torch.from_numpy(R.turn(x64, angles, interleaved))       # (products and differences are exact but for one rounding)
            mass = np.zeros(x64.shape)                                      # |x_a c_i| + |x_b s_i|
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                c, s = np.abs(angles[:, None, i]), np.abs(angles[:, None, half + i])
                mass[..., a] = np.abs(x64[..., a]) * c + np.abs(x64[..., b]) * s
                mass[..., b] = np.abs(x64[..., b]) * c + np.abs(x64[..., a]) * s
        rounded = want.float()
        if dtype == torch.bfloat16:
            # bit for bit; a pair that holds no number, or an infinity, gives two that are not finite
            bad = ~np.isfinite(mass) & ~np.isfinite(want.numpy())
            assert not y[torch.from_numpy(bad)].isfinite().any()
            keep = torch.from_numpy(~bad)
            assert torch.equal(y[keep].isnan(), rounded[keep].isnan())      # (a NaN past the R-th dimension stays one)
            keep &= ~rounded.isnan()
            assert torch.equal(y[keep], rounded.to(torch.bfloat16)[keep])
            continue
        assert torch.equal(y.isnan(), rounded.isnan())
        # finite where the definition is (but within the stated bound of the range's end), infinite where it is
        bound = torch.from_numpy(mass) * 2.0 ** -23 + 1e-45
        top = float(torch.finfo(torch.float32).max)
        border = torch.isfinite(want) & ((want.abs() - top).abs() <= bound)
        sure = ~border & ~rounded.isnan()
        assert torch.equal(y.isinf()[sure], rounded.isinf()[sure])
        assert torch.equal(y[sure & rounded.isinf()], rounded[sure & rounded.isinf()])
        near = sure & rounded.isfinite()
        assert ((y.double() - want).abs()[near] <= bound[near]).all()
