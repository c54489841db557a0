"""Attention calls with the caller's own buffers, from a host thread that has made no CUDA call before (a serving loop's
worker): the same result as from the main thread."""

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
KV, HEADS, BATCH, WIDTH = 2, 8, 3, 8


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def inputs(head_dim, new):
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *shape: torch.randn(shape, device="cuda", generator=g)  # noqa: E731
    pools = [randn(40, KV, 16, head_dim).to(torch.bfloat16) for _ in range(2)]
    k8 = torch.randint(-127, 128, (40, KV, 16, head_dim), dtype=torch.int8, device="cuda", generator=g)
    v8 = torch.randint(-127, 128, (40, KV, head_dim, 16), dtype=torch.int8, device="cuda", generator=g)
    scales = torch.rand((40, KV, 2, 16), device="cuda", generator=g) * 0.01
    q4 = torch.randint(0, 256, (40, KV, 16 * head_dim + 128), dtype=torch.uint8, device="cuda", generator=g)
    q4[..., 16 * head_dim:] = torch.full((40, KV, 32), 0.1, device="cuda").view(torch.uint8)
    tables = torch.randperm(40, device="cuda", generator=g)[:BATCH * WIDTH].view(BATCH, WIDTH).to(torch.int32)
    lens = torch.tensor([100, 128, 77], dtype=torch.int32, device="cuda")
    start = torch.arange(0, BATCH * new + 1, new, dtype=torch.int32, device="cuda")
    q = randn(BATCH * new, HEADS, head_dim).to(torch.bfloat16)
    return pools, (k8, v8, scales), q4, tables, lens, start, q


@pytest.mark.parametrize("name,head_dim,new", [
    ("decode", 128, 1), ("decode", 64, 1), ("prefixed", 128, 1), ("prefixed", 64, 1), ("multiquery", 128, 3),
    ("multiquery", 64, 40), ("multiquery", 128, 40), ("decode_q8", 128, 1), ("multiquery_q8", 128, 3), ("multiquery_q8", 128, 60),
    ("multiquery_q4", 128, 3), ("multiquery_q4", 64, 40)])
def test_first_call_of_a_thread(pkv, name, head_dim, new):
    pools, q8, q4, tables, lens, start, q = inputs(head_dim, new)
    out = torch.zeros_like(q)
    zeros = lambda n: torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")  # noqa: E731
    here = torch.cuda.current_stream().cuda_stream
    how = dict(out=out, stream=here)
    if name == "decode":
        how["workspace"] = zeros(pkv.pkv_decode_workspace_size(BATCH, HEADS, WIDTH, pools[0]))
        call = lambda: pkv.pkv_decode_attention(q, *pools, tables, lens, 0.1, **how)  # noqa: E731
    elif name == "prefixed":
        tables[:, :3] = tables[0, :3].clone()
        group = torch.zeros(BATCH, dtype=torch.int32, device="cuda")
        shared = torch.tensor([3], dtype=torch.int32, device="cuda")
        how["workspace"] = zeros(pkv.pkv_decode_prefixed_workspace_size(BATCH, HEADS, WIDTH, 1, 3, pools[0]))
        call = lambda: pkv.pkv_decode_attention_prefixed(q, *pools, tables, lens, 0.1, group, shared, 3, **how)  # noqa: E731
    elif name == "multiquery":
        how["workspace"] = zeros(pkv.pkv_multiquery_workspace_size(BATCH, HEADS, WIDTH, new, pools[0]))
        call = lambda: pkv.pkv_multiquery_attention(q, *pools, tables, lens, start, 0.1, new, **how)  # noqa: E731
    elif name == "decode_q8":
        how["workspace"] = zeros(pkv.pkv_decode_q8_workspace_size(BATCH, HEADS, WIDTH, q8[0]))
        call = lambda: pkv.pkv_decode_attention_q8(q, *q8, tables, lens, 0.1, **how)  # noqa: E731
    elif name == "multiquery_q8":
        how["workspace"] = zeros(pkv.pkv_multiquery_q8_workspace_size(BATCH, HEADS, WIDTH, new, q8[0]))
        call = lambda: pkv.pkv_multiquery_attention_q8(q, *q8, tables, lens, start, 0.1, new, **how)  # noqa: E731
    else:
        how["workspace"] = zeros(pkv.pkv_multiquery_q4_workspace_size(BATCH, HEADS, WIDTH, new, q4))
        call = lambda: pkv.pkv_multiquery_attention_q4(q, q4, tables, lens, start, 0.1, new, **how)  # noqa: E731
    call()
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    raised = []

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            raised.append(e)
    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not raised and torch.equal(out, want) and out.any()
