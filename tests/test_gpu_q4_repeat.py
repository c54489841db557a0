"""The 4-bit attention gives the same bits every time, eagerly, in place and replayed: its sums have a fixed order. And each
call is right where its output is q itself."""

import pytest
import torch

from q4_cases import check, make, reference

pytestmark = pytest.mark.gpu
CASES = {
    "one": ([1000], [1], 32, 8, 128), "ragged": ([5, 700, 8000, 1, 3000, 64, 2049] * 9, [1] * 63, 24, 8, 128),
    "drafts": ([4000, 100, 2500, 17] * 4, [4, 4, 3, 1] * 4, 32, 8, 128), "rows32": ([900, 3000], [8, 7], 16, 4, 64),
    "chunks": ([2000, 300, 1500], [512, 300, 77], 16, 4, 128),
}


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("name", sorted(CASES))
def test_same_bits(pkv, name):
    lens, news, q_heads, kv_heads, d = CASES[name]
    s = make(41, lens, news, q_heads, kv_heads, d, garbage=False)
    most = max(news)
    work = torch.zeros(pkv.pkv_multiquery_q4_workspace_size(len(lens), q_heads, s["tables"].shape[1], most, s["cache"]),
                       dtype=torch.uint8, device="cuda")

    def call(q, out=None):
        return pkv.pkv_multiquery_attention_q4(q, s["cache"], s["tables"], s["lens"], s["start"], s["scale"], most, out=out,
                                               workspace=work)
    first = call(s["q"])
    check(first, *reference(s))
    for _ in range(20):
        assert torch.equal(call(s["q"]), first)
    same = s["q"].clone()
    assert call(same, out=same) is same and torch.equal(same, first)
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(first)
    with torch.cuda.graph(graph):
        call(s["q"], out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    if most == 1:
        decode = pkv.pkv_decode_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["scale"], workspace=work)
        assert torch.equal(decode, first)
        same = s["q"].clone()
        pkv.pkv_decode_attention_q4(same, s["cache"], s["tables"], s["lens"], s["scale"], out=same, workspace=work)
        assert torch.equal(same, first)
