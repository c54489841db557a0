"""pkv_multiquery_attention_q8 at the ends of the float range: q and K of sizes that
cancel. Tolerances are those of tests/test_gpu_chunk_q8.py (and of
tests/test_gpu_chunk_q8_few_rows.py)."""

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
