"""More sequences than one launch of the 4-bit calls takes (1024): decode, drafts, chunks and reading back, with ragged
lengths and sequences without tokens or queries among them."""

import random

import pytest
import torch

from q4_cases import B, check, make, reference, values64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def lengths(batch, seed, most=70):
    rng = random.Random(seed)
    return [0 if i in (0, 1023, 1024, batch - 1) or rng.random() < 0.05 else rng.randrange(1, most) for i in range(batch)]


@pytest.mark.parametrize("batch", [1024, 1025, 2500])
def test_decode(pkv, batch):
    lens = lengths(batch, batch)
    s = make(51, lens, [1] * batch, 6, 2, 64)
    got = pkv.pkv_decode_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["scale"])
    check(got, *reference(s, decode=True))
    assert not got[[i for i, n in enumerate(lens) if n == 0]].any()


@pytest.mark.parametrize("batch", [1025, 2500])
@pytest.mark.parametrize("most", [3, 20])
def test_multiquery(pkv, batch, most):
    lens = lengths(batch, batch + most)
    rng = random.Random(most)
    news = [min(n, rng.randrange(0, most + 1)) for n in lens]
    news[3] = lens[3] = most
    s = make(52, lens, news, 4, 1, 128)
    got = torch.full_like(s["q"], 7.0)
    pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["start"], s["scale"], most, out=got)
    check(got, *reference(s))


@pytest.mark.parametrize("batch", [1024, 1025, 2500])
def test_gather(pkv, batch):
    lens = lengths(batch, batch + 7)
    s = make(53, lens, [0] * batch, 2, 2, 64)
    rows = sum(lens)
    start = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    k, v = pkv.pkv_gather_q4(s["cache"], s["tables"], s["lens"], start, rows, out_dtype=torch.float32)
    seq = torch.repeat_interleave(torch.arange(batch, device="cuda"), torch.tensor(lens, device="cuda"))
    t = torch.arange(rows, device="cuda") - start[seq].long()
    block = s["tables"][seq, t // B].long()
    for got, pool in zip((k, v), values64(s)):
        assert torch.equal(got, pool[block, :, t % B].float())
