"""The 4-bit attention's sums over long contexts where a warp sums thousands of tokens: so many sequences that a CTA takes
whole ones, all of them over the same blocks. Dimensions in which the tokens that have the weight hold the code 0 (and so
add nothing) show what the sums over code + 8 lose, against the bound that include/pkv.h states for a context of n tokens:
(n / 4 + 368) 2^-23 of the sum of the weights times their V scales.

From where the bound comes: a warp sums every 4th stage of 32 tokens of a context that one CTA takes (every 2nd where two
warps share a block), 16 products at a time. With A the sum of weight times scale before a window of 256 tokens and S that
of the window, the running sum is at most 7 A + 15 S and 8 S is summed beside it; the tensor cores round each by at most
2^-23 of it, 16 times a window: 16 2^-23 (7 A + 23 S). Over the n / 512 windows of the busier case A <= the whole sum and
the S add up to it: (16 7 n / 512 + 368) 2^-23, and 112 / 512 is below a quarter."""

import numpy as np
import pytest
import torch

from oracle import quant4 as Q
from q4_cases import B, fast_pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [1400, 16384, 131072])
@pytest.mark.parametrize("rows,d", [(4, 128), (16, 128), (32, 64)])
@pytest.mark.parametrize("kind", ["even", "few", "zeros"])
def test_bound(pkv, n, rows, d, kind):
    rng = np.random.default_rng(n + rows)
    blocks, many = n // B + 1, 480
    kc = rng.integers(-7, 8, (blocks, 1, B, d)).astype(np.int8)
    vc = rng.integers(-7, 8, (blocks, 1, B, d)).astype(np.int8)
    ks, vs = np.full((blocks, 1, B), 0.02, np.float32), np.full((blocks, 1, B), 0.3, np.float32)
    if kind == "zeros":                                     # codes of 0 but for a little: what is left is the sums' own error
        vc[..., :d // 2] = 0
        vc[::7, :, 3, :d // 2] = 1
    elif kind == "few":                                     # a tenth of the tokens has nearly all of the weight, and code 0 there
        heavy = rng.random((blocks, 1, B)) < 0.1
        kc[..., 0] = np.where(heavy, 7, -7)
        vc[heavy] = np.where(np.arange(d) < d // 2, 0, vc[heavy])
    cache = torch.from_numpy(fast_pack(kc, vc, ks, vs)).cuda()
    new = max(1, rows // 8)
    heads = rows // new
    g = torch.Generator().manual_seed(n)
    q = torch.randn((new, heads, d), generator=g)
    if kind == "few":
        q[..., 0] = 20
    q = q.to(torch.bfloat16).cuda()
    tables = torch.arange(blocks, dtype=torch.int32, device="cuda").expand(many, -1).contiguous()
    lens = torch.full((many,), n, dtype=torch.int32, device="cuda")
    start = torch.arange(0, many * new + 1, new, dtype=torch.int32, device="cuda")
    got = pkv.pkv_multiquery_attention_q4(q.repeat(many, 1, 1), cache, tables, lens, start, 1.0, new).view(many, new, heads, d)
    k, v = (torch.from_numpy(x[:, 0].reshape(-1, d)[:n]).cuda().double() for x in Q.values(cache.cpu().numpy(), d))
    x = q.double()
    seen = torch.arange(n, device="cuda") <= torch.arange(n - new, n, device="cuda")[:, None]
    w = torch.softmax((x @ k.T).masked_fill(~seen[:, None], -torch.inf), -1)
    want, mass = w @ v, w @ v.abs()
    weight = 0.3 * w.sum(-1, keepdim=True)                  # of weights times their V scales: 0.3
    # the score is summed to 2^-15 |scale| (K scale) sum|q|, which moves the weights by factors within e^+-that, numerator and
    # denominator; a weight times its scale is rounded to f16 once, 2^-12 of it, or 2^-32 of the largest one; one bf16 step
    delta = 2.0 ** -15 * 0.02 * x.abs().sum(-1, keepdim=True)
    bound = want.abs() * 2.0 ** -8 + mass * (2.0 ** -11 + 4 * delta) + 8 * n * 2.0 ** -32 * 0.3 * w.amax(-1, keepdim=True) + \
        (n / 4 + 368) * 2.0 ** -23 * weight
    # (480 sequences on some 304 to 456 CTAs: where they are cut differs, and so do the sums, by less)
    worst = max(((x.double() - want).abs() / bound).max().item() for x in got)
    assert worst <= 1, f"{worst} times the bound"
