"""pkv_gather and pkv_gather_q8: the rows of a plain index loop, bit for bit
(the int8 value is code * scale rounded once to float32, then to bf16)."""

import numpy as np
import pytest
import torch

import cases

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_209_gb300 import pkv as P
    P.load_library()
    P.pkv_device_status(clear=True)
    return P


def pools(seed, lens, heads, d, form):
    """A paged case whose unused slots hold NaN (bf16, f32) or NaN scales (int8)."""
    c = cases.random_case(seed, lens, heads, heads, d, torch.bfloat16 if form == "bf16" else torch.float32,
                          poison=form != "q8")
    if form == "q8":
        rng = np.random.default_rng(seed)
        nb = c["k_pool"].shape[0]
        live = np.zeros((nb, 16), dtype=bool)
        for i, n in enumerate(c["lens"]):
            for t in range(int(n)):
                live[c["tables"][i, t // 16], t % 16] = True
        c["k_pool"] = torch.from_numpy(rng.integers(-128, 128, (nb, heads, 16, d)).astype(np.int8))
        c["v_pool"] = torch.from_numpy(rng.integers(-128, 128, (nb, heads, d, 16)).astype(np.int8))
        sc = rng.uniform(1e-4, 3.0, (nb, heads, 2, 16)).astype(np.float32)
        sc.transpose(0, 3, 1, 2)[~live] = np.nan
        c["scales"] = torch.from_numpy(sc)
    return c


def plain(c, first, counts, dtype):
    """Rows in order, from host loops over (sequence, token)."""
    k, v = [], []
    for i, n in enumerate(counts):
        for t in range(int(first[i]), int(first[i]) + int(n)):
            b, s = int(c["tables"][i, t // 16]), t % 16
            if "scales" in c:
                k.append((c["k_pool"][b, :, s].float() * c["scales"][b, :, 0, s, None]).to(dtype))
                v.append((c["v_pool"][b, :, :, s].float() * c["scales"][b, :, 1, s, None]).to(dtype))
            else:
                k.append(c["k_pool"][b, :, s])
                v.append(c["v_pool"][b, :, s])
    return torch.stack(k), torch.stack(v)


def call(pkv, c, first, start, rows, dtype=torch.bfloat16, **kw):
    dev = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
    args = (dev(c["tables"]), dev(c["lens"]), dev(start), rows)
    kw.setdefault("token_start", None if first is None else dev(first))
    if "scales" in c:
        return pkv.pkv_gather_q8(c["k_pool"].cuda(), c["v_pool"].cuda(), c["scales"].cuda(), *args, out_dtype=dtype, **kw)
    return pkv.pkv_gather(c["k_pool"].cuda(), c["v_pool"].cuda(), *args, **kw)


def same(a, b):
    bits = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.cpu().view(bits), b.cpu().view(bits))


FORMS = [("bf16", torch.bfloat16), ("f32", torch.float32), ("q8", torch.bfloat16), ("q8", torch.float32)]


@pytest.mark.parametrize("form,dtype", FORMS)
@pytest.mark.parametrize("heads,d", [(8, 128), (2, 64), (1, 128), (3, 64)])
def test_ranges_match_a_plain_loop(pkv, form, dtype, heads, d):
    lens = [1, 16, 17, 0, 333, 64, 5, 31]
    c = pools(heads * d, lens, heads, d, form)
    rng = np.random.default_rng(heads)
    first = np.array([rng.integers(0, n + 1) for n in lens])
    counts = np.array([rng.integers(0, n - f + 1) for n, f in zip(lens, first)])
    for f, n in ((np.zeros(8, int), np.array(lens)), (first, counts), (np.array([0, 15, 16, 0, 320, 1, 4, 0]),
                                                                      np.array([1, 1, 1, 0, 13, 62, 1, 16]))):
        start = np.concatenate([[0], np.cumsum(n)])
        k, v = call(pkv, c, f, start, int(start[-1]), dtype)
        wk, wv = plain(c, f, n, dtype)
        assert same(k, wk) and same(v, wv)
    k2, v2 = call(pkv, c, None, np.concatenate([[0], np.cumsum(lens)]), sum(lens), dtype)
    wk, wv = plain(c, np.zeros(8, int), np.array(lens), dtype)
    assert same(k2, wk) and same(v2, wv)
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("form,dtype", FORMS)
def test_rows_no_sequence_names_stay(pkv, form, dtype):
    """Gaps between the sequences' rows, and rows behind the last."""
    lens = [40, 7]
    c = pools(3, lens, 2, 128, form)
    k = torch.full((70, 2, 128), 3.0, dtype=dtype, device="cuda")
    v = torch.full((70, 2, 128), 4.0, dtype=dtype, device="cuda")
    # sequence 1's rows lie before sequence 0's: offsets need only be right pairwise for the used ones
    call(pkv, c, [2, 1], [5, 35, 41], 70, dtype, k_out=k, v_out=v)
    wk, wv = plain(c, [2, 1], [30, 6], dtype)
    assert same(k[5:41], wk) and same(v[5:41], wv)
    assert bool((k[:5] == 3).all()) and bool((k[41:] == 3).all())
    assert bool((v[:5] == 4).all()) and bool((v[41:] == 4).all())
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("form,dtype", FORMS)
def test_malformed_ranges_and_checked_mode(pkv, form, dtype):
    lens = [40, 70, 33]
    c = pools(4, lens, 2, 64, form)
    wk, _ = plain(c, [0, 0, 0], lens, dtype)
    start = np.array([0, 40, 110, 143])
    bads = []
    for tables, ln, first, st in (
            (None, lens, [0, 1, 0], start),                              # token_start + rows past the context
            (None, lens, [0, -1, 0], start),                             # before it
            (None, [40, 10 ** 6, 33], [0, 0, 0], start),                 # a context past its table
            ((1, 2), lens, [0, 0, 0], start)):                           # a block id outside the pool
        b = dict(c, tables=c["tables"].copy(), lens=np.array(ln))
        if tables:
            b["tables"][tables] = c["k_pool"].shape[0] + 3
        bads.append((b, first, st))
    for b, first, st in bads:
        k = torch.full((143, 2, 64), 3.0, dtype=dtype, device="cuda")
        v = torch.full_like(k, 3.0)
        call(pkv, b, first, st, 143, dtype, k_out=k, v_out=v)
        assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
        assert same(k[:40], wk[:40]) and same(k[110:], wk[110:])         # the other sequences are right
        assert bool((k[72:88] == 3).all())                              # at least the bad block's rows stay
        k.fill_(3.0)
        with pytest.raises(pkv.PkvError) as e:
            call(pkv, b, first, st, 143, dtype, k_out=k, v_out=v, flags=pkv.PKV_FLAG_CHECKED)
        assert e.value.name == "PKV_ERR_RANGE" and bool((k == 3).all())
    # rows past the outputs: sequence 2 would end at row 143 of 142
    k = torch.full((142, 2, 64), 3.0, dtype=dtype, device="cuda")
    v = torch.full_like(k, 3.0)
    call(pkv, c, None, start, 142, dtype, k_out=k, v_out=v)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
    assert same(k[:110], wk[:110]) and bool((k[110:] == 3).all())
    # offsets that fall: skipped, never a negative count
    call(pkv, c, None, [0, 40, 30, 63], 142, dtype, k_out=k, v_out=v)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
    call(pkv, c, None, start, 143, dtype, flags=pkv.PKV_FLAG_CHECKED)
    assert pkv.pkv_device_status(clear=True) == 0


def test_append_then_gather_is_the_identity(pkv):
    """What pkv_append wrote comes back bit for bit, every bit pattern included."""
    rng = np.random.default_rng(5)
    c = cases.random_case(5, [100, 37], 4, 4, 128, torch.bfloat16)
    rows = torch.from_numpy(rng.integers(0, 65536, (137, 4, 128)).astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    slots = np.concatenate([c["tables"][i, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
                            for i, n in enumerate(c["lens"])])
    kp, vp = c["k_pool"].cuda(), c["v_pool"].cuda()
    pkv.pkv_append(rows.cuda(), rows.flip(0).cuda(), torch.from_numpy(slots).cuda(), kp, vp)
    dev = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
    k, v = pkv.pkv_gather(kp, vp, dev(c["tables"]), dev(c["lens"]), dev([0, 100, 137]), 137)
    assert same(k, rows) and same(v, rows.flip(0))


def test_many_sequences_and_many_heads(pkv):
    lens = np.random.default_rng(8).integers(0, 20, 1500)
    c = pools(8, lens, 1, 64, "q8")
    start = np.concatenate([[0], np.cumsum(lens)])
    k, v = call(pkv, c, None, start, int(start[-1]))
    wk, wv = plain(c, np.zeros(1500, int), lens, torch.bfloat16)
    assert same(k, wk) and same(v, wv)
    # more KV heads than a grid dimension holds
    heads = 66000
    kp = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, heads, 16, 64), dtype=torch.int32, device="cuda").view(torch.float32)
    t = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    n = torch.tensor([20], dtype=torch.int32, device="cuda")
    st = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    k, v = pkv.pkv_gather(kp, kp, t, n, st, 20)
    want = torch.cat([kp[1].transpose(0, 1), kp[0, :, :4].transpose(0, 1)])
    assert torch.equal(k.view(torch.int32), want.contiguous().view(torch.int32)) and same(v, k)
    assert pkv.pkv_device_status(clear=True) == 0


def test_captured_and_replayed(pkv):
    c = pools(9, [50, 80], 2, 128, "q8")
    d = {k: c[k].cuda() for k in ("k_pool", "v_pool", "scales")}
    dev = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
    t, n, st, first = dev(c["tables"]), dev(c["lens"]), dev([0, 20, 60]), dev([0, 0])
    run = lambda: pkv.pkv_gather_q8(d["k_pool"], d["v_pool"], d["scales"], t, n, st, 60, token_start=first)  # noqa: E731
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k, v = run()
    for f in ([30, 40], [3, 0]):
        first.copy_(dev(f))
        graph.replay()
        torch.cuda.synchronize()
        wk, wv = plain(c, f, [20, 40], torch.bfloat16)
        assert same(k, wk) and same(v, wv)


def test_rows_past_32_bits(pkv):
    """Pools and outputs of more than 2^32 bytes each, the tokens at their far ends."""
    nb, rows, heads, d = 140_000, 2_200_000, 8, 128
    k, v = (torch.empty((nb, heads, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = torch.tensor([nb - 1, 0, nb - 2], device="cuda")
    k[ids], v[ids] = torch.randn(2, 3, heads, 16, d, device="cuda").to(torch.bfloat16)
    ko, vo = (torch.zeros((rows, heads, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    pkv.pkv_gather(k, v, ids.to(torch.int32)[None], torch.tensor([45], **i32), torch.tensor([rows - 40, rows], **i32), rows,
                   token_start=torch.tensor([5], **i32), k_out=ko, v_out=vo)
    for out, pool in ((ko, k), (vo, v)):
        want = pool[ids].permute(0, 2, 1, 3).reshape(48, heads, d)[5:45]
        assert torch.equal(out[-40:], want) and not out[:-40].any()
    assert pkv.pkv_device_status(clear=True) == 0
