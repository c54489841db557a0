"""pkv_verify_drafts against the float64 oracle: every output is a whole number
and must be equal. Random inputs are multiples of 2^-30 below one, so that
every sum of a row is exact in 64 bits and no draw can lie between two
roundings of a border."""

import numpy as np
import pytest
import torch

from oracle import verify as OV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_209_gb300 import pkv as P
    P.load_library()
    P.pkv_device_status(clear=True)
    return P


def case(seed, drafts, vocab, dtype=torch.float32, accept=0.7, peak=3.0):
    """Drafts per sequence (None: an idle one) -> inputs on the host."""
    rng = np.random.default_rng(seed)
    ks = [0 if k is None else k for k in drafts]
    ts = [0 if k is None else k + 1 for k in drafts]
    qs = np.concatenate([[0], np.cumsum(ts)]).astype(np.int32)
    ds = np.concatenate([[0], np.cumsum(ks)]).astype(np.int32)

    def rows(n):
        x = np.exp(peak * rng.standard_normal((n, vocab)))
        x /= x.sum(-1, keepdims=True)
        return x
    q, p = rows(int(ds[-1])), rows(int(qs[-1]))
    for i, k in enumerate(ks):
        p[qs[i]:qs[i] + k] = (1 - accept) * p[qs[i]:qs[i] + k] + accept * q[ds[i]:ds[i + 1]]
    # dtype's grid, and multiples of 2^-30
    grid = lambda x: torch.from_numpy(np.round(x * 2.0 ** 30) / 2.0 ** 30).to(dtype)  # noqa: E731
    tokens = np.array([rng.choice(vocab, p=r / r.sum()) for r in q], dtype=np.int32)
    return dict(p=grid(p), q=grid(q), tokens=tokens, accept=rng.random(len(tokens)).astype(np.float32),
                sample=rng.random(len(drafts)).astype(np.float32), qs=qs, ds=ds, most=max(ks + [0]),
                lens=(100 + rng.integers(0, 50, len(drafts))).astype(np.int32))


def oracle(c, certain=False):
    q = None if certain else c["q"].float().numpy()
    out, kept, rej = OV.verify_batch(c["p"].float().numpy(), q, c["tokens"], c["accept"], c["sample"], c["qs"],
                                     c["ds"], c["most"])
    return out, kept, c["lens"] - rej


def device(c):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(v)).cuda())
            for k, v in c.items() if k != "most"}


def call(pkv, c, certain=False, **kw):
    d = device(c)
    return pkv.pkv_verify_drafts(d["p"], None if certain else d["q"], d["tokens"], d["accept"], d["sample"], d["qs"],
                                 d["ds"], c["most"], context_lens=d["lens"], **kw)


def check(pkv, c, certain=False, **kw):
    got = call(pkv, c, certain, **kw)
    for g, w in zip(got, oracle(c, certain)):
        assert np.array_equal(g.cpu().numpy(), w)
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1, 2, 31, 1023, 1024, 1025, 5001, 32000])
@pytest.mark.parametrize("certain", [False, True])
def test_matches_oracle(pkv, dtype, vocab, certain):
    check(pkv, case(vocab + certain, [4, 0, 1, None, 7, 3, 2, 8, 5], vocab, dtype), certain)


@pytest.mark.parametrize("accept", [0.0, 0.5, 1.0])
def test_acceptance_rates_and_long_drafts(pkv, accept):
    c = case(5, [40, 33, 64, 1], 300, accept=accept)          # more drafts than one warp looks at together
    check(pkv, c)


def test_large_vocabulary(pkv):
    check(pkv, case(6, [3, 2, 0], 262147))


def test_many_sequences(pkv):
    check(pkv, case(7, list(np.random.default_rng(1).integers(0, 4, 1500)), 97))


def test_the_largest_vocabulary_and_one_past_it(pkv):
    c = case(8, [1], 1 << 20, peak=1.0)
    check(pkv, c)
    p = torch.zeros((1, (1 << 20) + 1), device="cuda")
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_verify_drafts(p, None, z[:0], p[0, :0], p[0, :1], z, z, 0)
    assert e.value.name == "PKV_ERR_SHAPE"


def test_draws_at_the_borders(pkv):
    """w = 0 and the largest float32 below one, masses only at the first and
    last index, and a border hit exactly."""
    v = 3001
    rows = np.zeros((6, v), dtype=np.float32)
    rows[0, [0, v - 1]] = 0.5, 0.5
    rows[1, [5, v - 1]] = 0.25, 0.75
    rows[2, 1500] = 1.0
    rows[3, [1023, 1024]] = 0.5, 0.5
    rows[4, [1023, 1024]] = 0.5, 0.5
    rows[5, [0, v - 1]] = 0.5, 0.5
    below = float(np.nextafter(np.float32(1), np.float32(0)))
    c = dict(p=torch.from_numpy(rows), q=torch.zeros((0, v)), tokens=np.zeros(0, np.int32),
             accept=np.zeros(0, np.float32), sample=np.array([0, 0.25, below, 0.5, 0.49, below], np.float32),
             qs=np.arange(7, dtype=np.int32), ds=np.zeros(7, np.int32), most=0, lens=np.full(6, 9, np.int32))
    assert oracle(c)[0][:, 0].tolist() == [0, v - 1, 1500, 1024, 1023, v - 1]
    check(pkv, c)


def test_rows_without_mass_nan_and_infinities(pkv):
    """Entries that are no finite number above zero carry nothing; a row of
    nothing gives token -1; max(p - q, 0) of nothing falls back to p."""
    v = 2050
    rng = np.random.default_rng(3)
    p = rng.random((6, v)).astype(np.float32)
    p = np.round(p * 2 ** 12).astype(np.float32) / 2 ** 20
    q = p[[0, 2]].copy()
    p[1, ::3], p[1, 1::3] = np.nan, np.inf
    p[3] = 0
    p[4, 7], p[4, 8] = -1.0, np.nan
    q[0] *= 2                                                  # p < q everywhere, the draft rejected
    q[1, 100:] = np.nan                                        # NaN differences carry nothing
    c = dict(p=torch.from_numpy(p), q=torch.from_numpy(q), tokens=np.array([3, 5], np.int32),
             accept=np.array([0.99, 0.0], np.float32), sample=np.array([0.3, 0.9, 0.5, 0.6, 0.1], np.float32)[:4],
             qs=np.array([0, 2, 4, 5, 6], np.int32), ds=np.array([0, 1, 2, 2, 2], np.int32), most=1,
             lens=np.full(4, 50, np.int32))
    c["q"][1, 5] = 1e9                                         # rejected although u = 0 keeps any p > 0: p is zero
    c["p"][2, 5] = 0
    check(pkv, c)
    c["p"][2:4] = 0                                            # no mass anywhere: -1
    assert oracle(c)[0][1, 0] == -1
    check(pkv, c)


def test_strided_rows_and_unaligned_bases(pkv):
    """Rows padded to another stride, starting off the 16-byte grid."""
    c = case(9, [4, 2, 0, 3], 1001)
    want = oracle(c)
    for dtype, off, pad in ((torch.float32, 1, 3), (torch.float32, 0, 0), (torch.bfloat16, 3, 6)):
        c2 = dict(c, p=c["p"].to(dtype), q=c["q"].to(dtype))
        want = oracle(c2)
        d = device(c2)

        def spread(t):
            rows, v = t.shape
            flat = torch.full((rows * (v + pad) + off + 8,), 7.0, dtype=dtype, device="cuda")
            view = flat[off:off + rows * (v + pad)].view(rows, v + pad)[:, :v]
            view.copy_(t)
            return view
        got = pkv.pkv_verify_drafts(spread(d["p"]), spread(d["q"]), d["tokens"], d["accept"], d["sample"], d["qs"],
                                    d["ds"], c["most"])
        assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
        assert got[2] is None
    assert pkv.pkv_device_status(clear=True) == 0


def test_lengths_in_place(pkv):
    c = case(10, [4, None, 2], 50)
    d = device(c)
    pkv.pkv_verify_drafts(d["p"], d["q"], d["tokens"], d["accept"], d["sample"], d["qs"], d["ds"], c["most"],
                          context_lens=d["lens"], new_context_lens=d["lens"])
    assert np.array_equal(d["lens"].cpu().numpy(), oracle(c)[2])


def test_malformed_sequences_and_checked_mode(pkv):
    """Offsets that leave the arrays or disagree, a token outside the vocabulary:
    reported, the other sequences right; checked mode writes nothing."""
    c = case(11, [2, 3, 1, 2], 300)
    want = oracle(c)
    bad = dict(c, qs=c["qs"].copy(), tokens=c["tokens"].copy())
    bad["qs"][4] = 99                                          # sequence 3: more rows than there are
    got = call(pkv, bad)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
    assert np.array_equal(got[0].cpu().numpy()[:3], want[0][:3])
    assert got[0][3].tolist() == [-1] * 4 and got[1][3] == -1 and got[2][3] == int(c["lens"][3])
    bad = dict(c, ds=c["ds"].copy())
    bad["ds"][0] = -5
    got = call(pkv, bad)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE and got[1][0] == -1
    assert np.array_equal(got[0].cpu().numpy()[1:], want[0][1:])
    for token in (300, -1, 2 ** 31 - 1):
        bad = dict(c, tokens=c["tokens"].copy())
        bad["tokens"][2] = token                               # sequence 1's first draft: rejected
        got = call(pkv, bad)
        assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
        assert np.array_equal(got[0].cpu().numpy(), oracle(bad)[0]) and got[1][1] == 0
        out = torch.full((4, 4), 77, dtype=torch.int32, device="cuda")
        with pytest.raises(pkv.PkvError) as e:
            call(pkv, bad, out_tokens=out, flags=pkv.PKV_FLAG_CHECKED)
        assert e.value.name == "PKV_ERR_RANGE" and bool((out == 77).all())
    check(pkv, c, flags=pkv.PKV_FLAG_CHECKED)


def test_captured_and_replayed_and_another_stream(pkv):
    """A captured call replayed on new probabilities; a call on a side stream."""
    a, b = case(12, [3, 1, 4], 2000), case(13, [3, 1, 4], 2000)
    d = device(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run = lambda: pkv.pkv_verify_drafts(d["p"], d["q"], d["tokens"], d["accept"], d["sample"], d["qs"], d["ds"],  # noqa: E731
                                        a["most"], context_lens=d["lens"])
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.synchronize()
    assert np.array_equal(got[0].cpu().numpy(), oracle(a)[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for c in (b, a, b):
        for key, v in device(c).items():
            d[key].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(out, oracle(c)):
            assert np.array_equal(g.cpu().numpy(), w)


def test_rows_past_32_bits(pkv):
    """The last rows of 4.4 billion probabilities."""
    c = case(12, [4], 262144, torch.bfloat16)
    rows = 17_000
    d = device(c)
    p = torch.empty((rows, 262144), dtype=torch.bfloat16, device="cuda")
    p[-5:] = d["p"]
    got = pkv.pkv_verify_drafts(p, d["q"], d["tokens"], d["accept"], d["sample"], d["qs"] + (rows - 5), d["ds"], c["most"],
                                context_lens=d["lens"])
    for g, w in zip(got, oracle(c)):
        assert np.array_equal(g.cpu().numpy(), w)
    assert pkv.pkv_device_status(clear=True) == 0


def test_sums_past_float32_still_name_a_token(pkv):
    """Rows that are no probabilities at all: some index or -1, and nothing left unwritten."""
    v = 5000
    p = torch.full((2, v), 3e38, device="cuda")
    z = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.full((2, 1), 12345, dtype=torch.int32, device="cuda")
    pkv.pkv_verify_drafts(p, None, none[:0], p[0, :0], torch.tensor([0.5, 0.0], device="cuda"), z, none, 0, out_tokens=out)
    assert ((out >= -1) & (out < v)).all()
