"""Scales that are NaN or infinite in 4-bit records and int8 pools, from wherever they come: a row that sees such a token
is not finite, however little weight the token has, and every other row is right."""

import math

import numpy as np
import pytest
import torch

from oracle import quant4 as Q
from q4_cases import B, check, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


# rows of a KV head: 4, 32 (split), 160 (tiles)
@pytest.mark.parametrize("new", [1, 8, 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [300, 320])
@pytest.mark.parametrize("back", [1, 30, 250])
@pytest.mark.parametrize("what", ["k_nan", "k_inf", "k_minus_inf", "v_nan", "v_inf", "v_minus_inf"])
@pytest.mark.parametrize("weight", [-400.0, 40.0])
def test_scales(pkv, new, d, n, back, what, weight):
    """`weight`: the token's score above the others', in nats."""
    s = make(21, [n, 77], [new, 2], 8, 2, d)
    q = s["q"].float() * 0.25
    q[..., 0] = 8
    s["q"] = q.to(torch.bfloat16)
    kc, vc, ks, vs = Q.unpack(s["cache"].cpu().numpy(), d)
    kc[..., 0] = 0
    block, t = s["tables"][0, (n - back) // B].item(), (n - back) % B
    kc[block, 1, t] = 0
    kc[block, 1, t, 0] = 7 if weight >= 0 else -7
    ks[block, 1, t] = abs(weight) / (8 * s["scale"] * 7)
    s["cache"] = torch.from_numpy(Q.pack(kc, vc, ks, vs)).cuda()
    want, bound = reference(s)
    side, value = (ks if what[0] == "k" else vs), what.split("_", 1)[1]
    side[block, 1, t] = {"nan": math.nan, "inf": math.inf, "minus_inf": -math.inf}[value]
    if what[0] == "k":
        kc[block, 1, t] = -7 if weight < 0 else 7
    s["cache"] = torch.from_numpy(Q.pack(kc, vc, ks, vs)).cuda()
    got = pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["start"], s["scale"], max(new, 2))
    sees = torch.zeros(got.shape[:2], dtype=torch.bool, device="cuda")
    sees[max(0, new - back):new, 4:] = True
    assert not got[sees].isfinite().any()
    check(got[~sees], want[~sees], bound[~sees], mean=False)
    if new == 1:
        one = pkv.pkv_decode_attention_q4(s["q"][:1], s["cache"], s["tables"][:1], s["lens"][:1], s["scale"])
        assert not one[0, 4:].isfinite().any() and one[0, :4].isfinite().all()


@pytest.mark.parametrize("what", ["k_nan", "k_inf", "v_nan", "v_inf"])
@pytest.mark.parametrize("back", [1, 30, 250])
@pytest.mark.parametrize("sign", [-1, 1])
def test_int8_tiles(pkv, what, back, sign):
    n, new, kv, heads, d = 300, 40, 2, 8, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    blocks = n // B + 1
    kc = torch.randint(-127, 128, (blocks, kv, B, d), dtype=torch.int8, device="cuda", generator=g)
    vc = torch.randint(-127, 128, (blocks, kv, d, B), dtype=torch.int8, device="cuda", generator=g)
    scales = torch.full((blocks, kv, 2, B), 0.01, device="cuda")
    q = torch.randn((new, heads, d), device="cuda", generator=g).to(torch.bfloat16).abs()
    at = n - back
    kc[at // B, 1, at % B] = 127 * sign                     # every query's score of it far above, or below, all others
    scales[at // B, 1, 0, at % B] = 0.1
    tables = torch.arange(blocks, dtype=torch.int32, device="cuda")[None].contiguous()
    lens, start = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([n], [0, new]))
    attend = lambda: pkv.pkv_multiquery_attention_q8(q, kc, vc, scales, tables, lens, start, 0.1, new)  # noqa: E731
    want = attend()
    scales[at // B, 1, 0 if what[0] == "k" else 1, at % B] = math.nan if what.endswith("nan") else math.inf
    got = attend()
    sees = torch.zeros((new, heads), dtype=torch.bool, device="cuda")
    sees[max(0, new - back):, 4:] = True
    assert not got[sees].isfinite().any()
    # each is off by half a bf16 step and by f16 roundings, 4 2^-11 of an average of |v| (1.27 at most): twice both
    assert ((got[~sees].double() - want[~sees].double()).abs() <= 2 * (want[~sees].double().abs() * 2.0 ** -8 + 1.27 * 4 * 2.0 ** -11)).all()
