"""Blocks whose ids are out of range, anywhere in a context: their tokens carry no weight and all others do, held to the
bounds of attention over exactly the tokens that are there."""

import numpy as np
import pytest
import torch

from q4_cases import B, check, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def without(s, seq, gone):
    """The reference and its bounds of sequence `seq` with some of its blocks' tokens taken out, query by query: each
    query as the last token of a context of what it sees."""
    n, new = s["lens_list"][seq], s["news"][seq]
    row0 = sum(s["news"][:seq])
    there = np.array([t // B not in gone for t in range(n)])
    out, bound = torch.zeros_like(s["q"][row0:row0 + new]).double(), torch.zeros_like(s["q"][row0:row0 + new]).double()
    table, cache = s["tables"][seq].cpu().numpy(), s["cache"].cpu().numpy()
    from oracle import quant4 as Q
    parts = [p[table[:-(-n // B)]] for p in Q.unpack(cache, s["d"])]        # blocks in order
    flat = [np.moveaxis(p, 1, 2).reshape(-1, p.shape[1], *p.shape[3:])[:n] for p in parts]
    from q4_cases import fast_pack
    for i in range(new):
        seen = np.flatnonzero(there & (np.arange(n) <= n - new + i))
        m = len(seen)
        if m == 0:
            continue
        fill = -(-m // B) * B
        rows = []
        for p in flat:
            x = np.zeros((fill, *p.shape[1:]), p.dtype)
            x[:m] = p[seen]
            rows.append(np.moveaxis(x.reshape(-1, B, *p.shape[1:]), 1, 2))
        packed = torch.from_numpy(fast_pack(*rows)).cuda()
        one = dict(s, cache=packed, tables=torch.arange(fill // B, device="cuda")[None], lens_list=[m], news=[1],
                   q=s["q"][row0 + i:row0 + i + 1])
        out[i:i + 1], bound[i:i + 1] = reference(one)
    return out, bound


# a stage is 32 tokens, two blocks: the first of one, the second, both, the last whole, the last partly filled, all
GONE = [[0], [1], [2], [3], [2, 3], [5], [6], [5, 6], [0, 1, 3, 6], list(range(7))]


@pytest.mark.parametrize("gone", GONE)
@pytest.mark.parametrize("new", [1, 4, 8, 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [97, 112, 104])
@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_absent_blocks(pkv, gone, new, d, n, bad):
    s = make(31, [n, 500], [new, 1], 8, 2, d)
    whole = reference(s)
    tables = s["tables"].clone()
    tables[0, gone] = bad
    got = pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], tables, s["lens"], s["start"], s["scale"], new)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
    check(got[:new], *without(s, 0, gone), mean=False)
    check(got[new:], whole[0][new:], whole[1][new:], mean=False)
    if new == 1:
        one = pkv.pkv_decode_attention_q4(s["q"], s["cache"], tables, s["lens"], s["scale"])
        assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
        check(one[:1], *without(s, 0, gone), mean=False)
