"""pkv_multiquery_attention_q8 with up to 16 query rows per (sequence, KV head) on
wide tables, where the kernel that splits the cache takes the call: scales of any
size and spread, and anything on tokens that a row may not see.

Tolerance: that of tests/test_gpu_chunk_q8.py, which this kernel's roundings stay
within. K's codes and q are exact here; a score is 32-bit products and sums, with
K's code bias (at most 2^-16 of the largest score; there 2^-11 for K's rounding); the
weight times the V scale is rounded to f16 once (there three roundings). Below f16's
normal range that product loses at most 2^-25, where the largest one of the row's
tokens is at least 2^8, or was before the base moved on: 2^-33 max_p w_p vs_p per
token, times a code of at most 2^7: n 2^-26 sum_p softmax_p vs_p together, less than
the 2^-11 sum_p softmax_p vs_p there up to 2^15 tokens.
"""

import numpy as np
import pytest
import torch

import test_gpu_chunk_q8 as T
from test_gpu_chunk_q8 import pkv  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def wide(c):
    """The case with table entries that no sequence uses: enough of them for the splitting kernel
    (524288 (token, KV head) pairs)."""
    batch, width = c["tables"].shape
    more = 524288 // (16 * c["kv_heads"] * batch) + 2
    return dict(c, tables=np.pad(c["tables"], ((0, 0), (0, more)), constant_values=-1))


def both(pkv, c, want=None):  # noqa: F811
    want = want or T.reference(c)
    T.check(T.call(pkv, wide(c)), c, want)
    T.check(T.call(pkv, c), c, want)
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("kscale,vscale", [(1.0, 1.0), (1e-3, 1e-3), (1.0, 1e-6), (1.0, 1e-8), (1.0, 1e-12),
                                           (1.0, 1e-20), (1.0, 1e-33), (8.0, 1e3), (1e-4, 1e8), (1.0, 1e30)])
@pytest.mark.parametrize("nqs,hq", [([4, 1, 2, 0], 8), ([3, 4, 4, 1], 2), ([1, 1, 1, 1], 32)])
def test_value_ranges(pkv, nqs, hq, kscale, vscale):  # noqa: F811
    both(pkv, T.make(21 + hq, [400, 130, 65, 7], nqs, hq, 2, 128, kscale, vscale))


@pytest.mark.parametrize("factor", [1e-30, 1e-9, 1e-4, 1e2, 1e5, 1e20])
def test_v_rows_of_another_size_than_the_others(pkv, factor):  # noqa: F811
    """A fifth of the V rows larger or smaller by a factor that leaves f16, first seen at
    the beginning of a context, in its middle or only at its end."""
    c = T.make(22, [600, 500, 700, 90], [4, 3, 1, 2], 8, 2, 128)
    rng = np.random.default_rng(9)
    for i, (a, b) in enumerate([(0, 600), (300, 500), (690, 700), (0, 90)]):
        for t in range(a, b):
            if rng.random() < 0.2 or t == b - 1:
                c["vs"][c["tables"][i, t // 16], :, t % 16] *= np.float32(factor)
    both(pkv, c)


@pytest.mark.parametrize("vscale", [1e-12, 1.0, 1e8])
def test_zero_rows(pkv, vscale):  # noqa: F811
    """Zero rows have scale 1, whatever the size of the others."""
    c = T.make(23, [300, 200, 50], [4, 2, 1], 8, 2, 128, 1.0, vscale)
    rng = np.random.default_rng(8)
    for pool, scales in ((c["kc"], c["ks"]), (c["vc"], c["vs"])):
        zero = rng.random(scales.shape) < 0.1
        pool[zero] = 0
        scales[zero] = 1.0
    both(pkv, c)


def test_all_values_zero(pkv):  # noqa: F811
    """Zero V codes under any scale, and a scale of zero under any codes, give zeros."""
    c = T.make(24, [90, 40], [4, 1], 8, 2, 128)
    for vs, vc in ((1.0, 0), (1e-30, 0), (1e30, 0), (0.0, 1)):
        d = dict(c, vs=np.full_like(c["vs"], vs), vc=c["vc"] * np.int8(vc))
        assert bool((T.call(pkv, wide(d)) == 0).all())


@pytest.mark.parametrize("k,v", [(np.nan, np.inf), (1.0, np.inf), (1.0, np.nan), (np.inf, 1e38)])
def test_later_drafts_hold_anything(pkv, k, v):  # noqa: F811
    """The last draft's scales are no numbers or immense: the rows before it are right."""
    c = T.make(25, [140, 300, 33], [4, 3, 2], 8, 2, 128)
    want = T.reference(c)
    for i, n in enumerate(c["lens"]):
        b, s = c["tables"][i, (n - 1) // 16], (n - 1) % 16
        c["ks"][b, :, s], c["vs"][b, :, s] = k, v
    keep = [0, 1, 2, 4, 5, 7]
    for c in (wide(c), c):
        T.check(T.call(pkv, c)[keep], c, (want[0][keep], want[1][keep]))


@pytest.mark.parametrize("e", [-110, -60, -20, -10, 20, 100])
def test_sizes_of_q_and_k_that_cancel(pkv, e):  # noqa: F811
    """q times 2^e and K's scales times 2^-e: the scores, and so the result, stay."""
    c = T.make(26, [300, 90, 40], [4, 3, 1], 8, 2, 128)
    want = T.reference(c)
    c["q"] = (c["q"].double() * 2.0 ** e).to(torch.bfloat16)
    c["ks"] = (c["ks"].astype(np.float64) * 2.0 ** -e).astype(np.float32)
    both(pkv, c, want)


@pytest.mark.parametrize("seed", range(8))
def test_random_scales(pkv, seed):  # noqa: F811
    rng = np.random.default_rng(800 + seed)
    hkv, group = int(rng.choice([1, 2, 4])), int(rng.choice([1, 2, 4]))
    lens = [int(n) for n in np.exp(rng.uniform(0, np.log(2500), rng.integers(1, 7)))]
    nqs = [int(rng.integers(0, min(n, 4) + 1)) for n in lens]
    c = T.make(seed, lens, nqs, group * hkv, hkv, 128, 2.0 ** rng.integers(-6, 2), 2.0 ** rng.integers(-60, 60))
    odd = rng.random(c["ks"].shape) < 0.01
    c["ks"][odd] *= np.float32(2.0) ** np.float32(-20)
    odd = rng.random(c["vs"].shape) < 0.01
    c["vs"][odd] *= np.float32(2.0) ** rng.choice([-40, 26], odd.sum()).astype(np.float32)
    both(pkv, T.poison(c))
