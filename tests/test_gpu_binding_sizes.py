"""Sizes past 32 bits, which tensors without elements may have, are refused by the native binding and not cut to 32 bits."""

import pytest
import torch

pytestmark = pytest.mark.gpu
LARGE = (1 << 32) + 2


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def test_tables_and_heads(pkv):
    cache = torch.zeros((4, 2, 16 * 64 + 128), dtype=torch.uint8, device="cuda")
    work = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    rows = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros((0, LARGE, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="32-bit"):
        pkv.pkv_decode_attention_q4(rows, cache, ints(LARGE, 0), ints(2), 0.1, workspace=work)
    with pytest.raises(ValueError, match="32-bit"):
        pkv.pkv_gather_q4(cache, ints(LARGE, 0), ints(2), ints(3), 0)
    with pytest.raises(ValueError, match="32-bit"):
        pkv.pkv_plan_step(ints(2), ints(2), ints(2), ints(1), ints(1), ints(LARGE, 0), 0)
    with pytest.raises(ValueError, match="q is"):
        pkv.pkv_multiquery_attention_q4(wide, cache, ints(1, 1), ints(1), ints(2), 0.1, 1, workspace=work)
    with pytest.raises(ValueError, match="q is"):
        pkv.pkv_append_rotary(wide, rows[:0], rows[:0], ints(0), torch.zeros((3, 64), device="cuda"),
                              torch.zeros(0, dtype=torch.int64, device="cuda"), cache)
