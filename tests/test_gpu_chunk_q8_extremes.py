"""pkv_multiquery_attention_q8 at the ends of the float range: q and K of sizes that
cancel, scores far apart under V scales far apart, V scales of zero. Tolerances are those
of tests/test_gpu_chunk_q8.py (and of tests/test_gpu_chunk_q8_few_rows.py)."""

import numpy as np
import pytest
import torch

import test_gpu_chunk_q8 as T
from test_gpu_chunk_q8 import pkv  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def wide(c):
    """With table entries that no sequence uses: few rows then run on the kernel that splits the cache."""
    batch = c["tables"].shape[0]
    more = 524288 // (16 * c["kv_heads"] * batch) + 2
    return dict(c, tables=np.pad(c["tables"], ((0, 0), (0, more)), constant_values=-1))


@pytest.mark.parametrize("e,peaked", [(-130, False), (-128, True), (-125, False), (-125, True), (-110, False), (-110, True),
                                      (-60, False), (-60, True), (60, False), (60, True), (110, False), (110, True)])
@pytest.mark.parametrize("nqs,d", [([60, 33], 64), ([60, 33], 128), ([4, 2], 128)])
def test_sizes_of_q_and_k_that_cancel(pkv, nqs, d, e, peaked):  # noqa: F811
    """q times 2^e (down to rows of numbers below the normal range) and K's scales times 2^-e."""
    c = T.make(51, [500, 90], nqs, 8, 2, d)
    c["q"] = (c["q"].double() * 2.0 ** e).to(torch.bfloat16)
    ramp = np.linspace(0.5, 15, 500) if peaked else np.ones(500)      # later tokens far above earlier ones
    c["ks"] = c["ks"].astype(np.float64) * 2.0 ** -e
    for i, n in enumerate(c["lens"]):
        for t in range(int(n)):
            c["ks"][c["tables"][i, t // 16], :, t % 16] *= ramp[t]
    c["ks"] = c["ks"].astype(np.float32)
    T.check(T.call(pkv, wide(c)), c)
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("nqs,d", [([60, 33], 64), ([60, 33], 128), ([4, 2], 128)])
def test_v_scales_of_zero(pkv, nqs, d):  # noqa: F811
    """All of them, and those of some tokens (the first block's among them)."""
    c = T.make(52, [500, 90], nqs, 8, 2, d)
    some = dict(c, vs=c["vs"].copy())
    c["vs"][:] = 0
    assert bool((T.call(pkv, wide(c)) == 0).all())
    some["vs"][np.random.default_rng(52).random(some["vs"].shape) < 0.3] = 0
    some["vs"][some["tables"][0, 0]] = 0
    T.check(T.call(pkv, wide(some)), some)


@pytest.mark.parametrize("vs", [0.0, 1e-45, 1e-38, 1e-30])
@pytest.mark.parametrize("nq,d", [(40, 64), (40, 128), (4, 128)])
def test_scores_and_v_scales_far_apart(pkv, nq, d, vs):  # noqa: F811
    """Token 200 stands 139 above the others with a V scale of (next to) nothing, token 5000,
    in another piece of the context, 416 above: the rows are its value."""
    c = T.make(53, [6000], [nq], 4, 1, d, 1.0, 1e6)
    q = c["q"].clone()
    q[..., 0] = 16
    c["q"] = q
    c["kc"][..., 0] = 0
    for t, nats in ((200, 139.0), (5000, 416.0)):
        b, s = c["tables"][0, t // 16], t % 16
        c["kc"][b, :, s], c["kc"][b, :, s, 0] = 0, 127
        c["ks"][b, :, s] = nats / (16 * 127 * c["scale"])
    b, s = c["tables"][0, 200 // 16], 200 % 16
    c["vs"][b, :, s] = vs
    b, s = c["tables"][0, 5000 // 16], 5000 % 16
    v = (c["vc"][b, 0, s].astype(np.float64) * c["vs"][b, 0, s])
    for c in (wide(c), c):
        out = T.call(pkv, c).double().cpu().numpy()
        assert np.abs(out - v).max() <= 2.0 ** -8 * np.abs(v).max() + 3 * 2.0 ** -11 * np.abs(v).max()


@pytest.mark.parametrize("nq,d", [(40, 64), (40, 128), (4, 128)])
def test_a_row_of_small_v_before_large_ones(pkv, nq, d):  # noqa: F811
    """A prompt whose first token has a V row 2^90 smaller than the next ones: its own row is that value."""
    c = T.make(54, [nq], [nq], 4, 1, d)
    b = c["tables"][0, 0]
    c["vs"][b, :, 0] *= np.float32(2.0 ** -90)
    T.check(T.call(pkv, wide(c)), c)
    out = T.call(pkv, c)[0].double().cpu().numpy()
    v = c["vc"][b, 0, 0].astype(np.float64) * c["vs"][b, 0, 0]
    assert (np.abs(out - v) <= (2.0 ** -8 + 3 * 2.0 ** -11) * np.abs(v)).all()


@pytest.mark.parametrize("first,rest", [(0.0, 1e8), (1e-38, 1e8), (1e-30, 1.0), (1e30, 1e-4), (1e12, 1e-12)])
@pytest.mark.parametrize("nqs,d", [([60, 33], 64), ([60, 33], 128), ([4, 2], 128)])
def test_a_first_block_of_another_size(pkv, nqs, d, first, rest):  # noqa: F811
    c = T.make(55, [500, 90], nqs, 8, 2, d)
    head = c["tables"][:, 0]
    size = np.full(c["vs"].shape, rest)
    size[head] = first
    c["vs"] = (c["vs"] * size).astype(np.float32)
    T.check(T.call(pkv, wide(c)), c)


@pytest.mark.parametrize("factor", [1.0, 1e12])
@pytest.mark.parametrize("nqs,d", [([60, 33], 64), ([60, 33], 128), ([4, 2], 128)])
def test_negative_scales(pkv, nqs, d, factor):  # noqa: F811
    """A value is its code times its scale, whatever the signs; some V scales leave the others' range."""
    c = T.make(56, [500, 90], nqs, 8, 2, d)
    rng = np.random.default_rng(56)
    for scales in (c["ks"], c["vs"]):
        scales[rng.random(scales.shape) < 0.3] *= -1
    c["vs"][rng.random(c["vs"].shape) < 0.1] *= np.float32(factor)
    T.check(T.call(pkv, wide(c)), c)
