"""pkv_multiquery_attention_q8 over contexts so long that one CTA works on a unit for
about a second. The table names two blocks again and again."""

import pytest
import torch

from test_gpu_chunk_q8 import pkv  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def test_units_of_a_quarter_million_steps(pkv):  # noqa: F811
    """One query of 304 heads on 2^25 tokens: two units a CTA or so, whole ones among them,
    each one row, so that one half of the rows' warps waits for all of a unit. K is zero
    (every weight 1), V too but for the last 128 tokens: the mean, 128 / 2^25 of V's code
    times its scale, is exact at every step (no sum needs more than 24 bits)."""
    n, heads, d = 1 << 25, 304, 64
    kc = torch.zeros((2, heads, 16, d), dtype=torch.int8, device="cuda")
    vc = torch.zeros((2, heads, d, 16), dtype=torch.int8, device="cuda")
    codes = torch.arange(d, device="cuda") - d // 2
    vc[1] = codes.to(torch.int8)[:, None]
    sc = torch.ones((2, heads, 2, 16), device="cuda")
    sc[1, :, 1] = 16
    tables = torch.zeros((1, n // 16), dtype=torch.int32, device="cuda")
    tables[:, -8:] = 1
    q = torch.ones((1, heads, d), dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out = pkv.pkv_multiquery_attention_q8(q, kc, vc, sc, tables, lens, start, 0.125, 1)
    torch.cuda.synchronize()
    assert pkv.pkv_device_status(clear=True) == 0
    assert torch.equal(out.double(), (codes.double() * 16 * 128 / n).expand(1, heads, d))
