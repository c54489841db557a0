"""Attention over the 4-bit cache where numbers leave their usual range: scales of any size and spread, zero rows,
peaked and far scores, attention sinks, huge and tiny queries, NaN and infinity where a row may not see them.

Bounds: that of tests/q4_cases.py (roundings relative to sum_p w_p |v_p| and to the scores), and three terms for what is
absolute in it.
Scores: the tensor cores sum (code + 8) q, and 8 sum(q) is taken off. A product of 16 terms is summed to 2^-22 of its
largest term or sum at worst, D / 16 <= 8 of them, so a score is off by at most |scale| ks 8 2^-22 15 sum|q|, less than
2^-15 |scale| ks sum|q|; weights move by twice that, taken twice for the second order.
Weights: one times its V scale is held in f16, whose smallest step is 2^-24, where the row's largest such product is
2^8 or more: n tokens lose at most n 2^-25 2^-8 max_p(w_p vs_p) times a code of at most 8. In the tiles a weight alone is
held so, the largest (behind a sink, otherwise 2^9 less) at 2^9: n 2^-34 max_p|v_p| (n 2^-32 is allowed).
Values, where the cache is split: with P'_p = w_p vs_p (over the row's sum), A their sum before a window of 256 tokens and S
that in it, O is sum (code + 8) P' over the window and sum code P' before it, at most 7 A + 15 S, and 8 S is summed beside
it and taken off at its end. The tensor cores round each of these sums by at most 2^-23 of it, 16 products a window: 16
2^-23 (7 A + 23 S) a window. Over all windows the S add up to sum_p w_p vs_p, and A <= that: (7 n / 16 + 368) 2^-23 sum_p w_p
vs_p, which is less than 2^-13 of it up to 1400 tokens. It shows where the tokens that have a row's weight have a code of 0.
"""

import math

import numpy as np
import pytest
import torch

from oracle import quant4 as Q
from q4_cases import B, check, make, values64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def attend(s, q, k, v, i, row, new, h, group):
    """One (sequence, KV head) in float64: out, sum w|v|, max w vs, max|v|, the score's sizes."""
    kv, d = k.shape[1], s["d"]
    n = s["lens_list"][i]
    blocks = s["tables"][i, :-(-n // B)].long()
    kk = k[blocks].transpose(0, 1).reshape(kv, -1, d)[h, :n]
    vv = v[blocks].transpose(0, 1).reshape(kv, -1, d)[h, :n]
    x = q[row:row + new, h * group:(h + 1) * group]
    seen = torch.arange(n, device="cuda") <= torch.arange(n - new, n, device="cuda")[:, None]
    z = (s["scale"] * (x @ kk.T)).masked_fill(~seen[:, None], -math.inf)
    w = torch.softmax(z, -1)
    return seen, x, kk, vv, w


def reference(s):
    k, v = values64(s)
    k, v = torch.nan_to_num(k, 0, 0, 0), torch.nan_to_num(v, 0, 0, 0)   # (only where no row that is looked at sees them)
    scales = torch.from_numpy(np.ascontiguousarray(s["cache"].cpu().numpy()[..., 16 * s["d"]:]).view(np.float32)).cuda().double()
    scales = torch.nan_to_num(scales.abs(), 0, 0, 0)
    q = s["q"].double()
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    kv = k.shape[1]
    group = q.shape[1] // kv
    row = 0
    for i, n in enumerate(s["lens_list"]):
        new = s["news"][i]
        for h in range(kv):
            seen, x, kk, vv, w = attend(s, q, k, v, i, row, new, h, group)
            ks, vs = (scales[s["tables"][i, :-(-n // B)].long(), h, a:a + B].reshape(-1)[:n] for a in (0, B))
            o, mass = w @ vv, w @ vv.abs()
            delta = abs(s["scale"]) * 2.0 ** -11 * (x.abs() @ kk.abs().T).masked_fill(~seen[:, None], 0).amax(-1, keepdim=True)
            delta += abs(s["scale"]) * 2.0 ** -15 * x.abs().sum(-1, keepdim=True) * ks.max()
            lost = n * 2.0 ** -30 * (w * vs).amax(-1, keepdim=True) + n * 2.0 ** -32 * vv.abs().max() * (new * group > 32)
            if new * group <= 32:
                assert n <= 1400
                lost = lost + 2.0 ** -13 * (w * vs).sum(-1, keepdim=True)
            out[row:row + new, h * group:(h + 1) * group] = o
            bound[row:row + new, h * group:(h + 1) * group] = o.abs() * 2.0 ** -8 + mass * (4 * 2.0 ** -11 + 4 * delta) + lost
        row += new
    return out, bound


def call(pkv, s):
    decode = all(n == 1 for n in s["news"])
    if decode:
        return pkv.pkv_decode_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["scale"])
    return pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["start"], s["scale"],
                                           max_query_len=max(s["news"]))


def scales_of(s):
    """A writable view of every record's scales on the host, and what puts them back."""
    host = s["cache"].cpu().numpy()
    view = np.ascontiguousarray(host[..., 16 * s["d"]:]).view(np.float32)

    def put():
        host[..., 16 * s["d"]:] = view.view(np.uint8).reshape(host[..., 16 * s["d"]:].shape)
        s["cache"].copy_(torch.from_numpy(host))
    return view, put


# rows of a KV head: 4, 16, 32 (split), 160 and more (tiles)
NEWS = [[1, 1], [4, 3], [8, 8], [40, 150]]


@pytest.mark.parametrize("news", NEWS)
@pytest.mark.parametrize("d", [64, 128])
def test_wide_scales_and_zero_rows(pkv, news, d):
    def sizes(low, high):
        return lambda rng, shape: np.where(rng.random(shape) < 0.1, 0.0, rng.uniform(low, high, shape))
    s = make(1, [300, 900], news, 8, 2, d, k_sizes=sizes(1e-3, 3), v_sizes=sizes(1e-2, 1e2))
    check(call(pkv, s), *reference(s), mean=False)


@pytest.mark.parametrize("news", NEWS)
@pytest.mark.parametrize("k_size,q_size", [(1e-30, 1e30), (1e30, 1e-30), (1e-3, 3e5), (1e4, 1e-4)])
def test_sizes_of_k_and_q(pkv, news, k_size, q_size):
    s = make(2, [200, 333], news, 8, 2, 128, spread=q_size, k_sizes=lambda rng, shape: np.full(shape, k_size))
    s["scale"] /= k_size * q_size
    check(call(pkv, s), *reference(s))


@pytest.mark.parametrize("news", NEWS)
@pytest.mark.parametrize("size", [1e-25, 1e-10, 1e10, 1e35])
def test_sizes_of_v(pkv, news, size):
    s = make(3, [200, 333], news, 8, 2, 128, v_sizes=lambda rng, shape: np.full(shape, size))
    want, bound = reference(s)
    got = call(pkv, s).double()
    assert torch.isfinite(got).all() and ((got - want).abs() <= bound).all()


@pytest.mark.parametrize("news", NEWS)
@pytest.mark.parametrize("d", [64, 128])
def test_v_rows_far_apart(pkv, news, d):
    """V rows from 2^-40 to 2^40, and the first block of the sequence the smallest, or the largest."""
    s = make(4, [500, 400], news, 8, 2, d, v_sizes=lambda rng, shape: np.exp2(rng.uniform(-40, 40, shape)))
    view, put = scales_of(s)
    view[s["tables"][0, 0].item(), :, B:] = 1e-13
    view[s["tables"][1, 0].item(), :, B:] = 1e13
    put()
    want, bound = reference(s)
    got = call(pkv, s).double()
    assert torch.isfinite(got).all() and ((got - want).abs() <= bound).all()


@pytest.mark.parametrize("news", NEWS)
@pytest.mark.parametrize("d", [64, 128])
def test_scores_far_apart(pkv, news, d):
    """Scores of standard deviation 6, and a ramp: later tokens far above earlier ones."""
    s = make(5, [700, 260], news, 8, 2, d, spread=6.0)
    check(call(pkv, s), *reference(s), mean=False)
    s = make(6, [700, 260], news, 8, 2, d)
    view, put = scales_of(s)
    ramp = np.linspace(0.5, 30, 700).astype(np.float32)
    tables = s["tables"].cpu().numpy()
    for i, n in enumerate(s["lens_list"]):
        for t in range(n):
            view[tables[i, t // B], :, t % B] *= ramp[t]
    put()
    check(call(pkv, s), *reference(s), mean=False)


@pytest.mark.parametrize("news", NEWS)
@pytest.mark.parametrize("nats", [10.0, 18.0, 30.0])
@pytest.mark.parametrize("where", [0, 100])
def test_sink_of_zero_value(pkv, news, nats, where):
    """One token takes nearly all of a row's weight and its value is nothing."""
    d = 128
    s = make(7, [1200, 300], news, 8, 2, d)
    q = s["q"].float() * 0.5
    q[..., 0] = 16
    s["q"] = q.to(torch.bfloat16)
    host, tables = s["cache"].cpu().numpy(), s["tables"].cpu().numpy()
    kc, vc, ks, vs = Q.unpack(host, d)
    kc[..., 0] = 0
    for i in range(2):
        b, o = tables[i, where // B], where % B
        kc[b, :, o] = 0
        kc[b, :, o, 0] = 7
        ks[b, :, o] = nats / (16 * s["scale"]) / 7
        vc[b, :, o] = 0
        vs[b, :, o] = 0
    s["cache"] = torch.from_numpy(Q.pack(kc, vc, ks, vs)).cuda()
    check(call(pkv, s), *reference(s), mean=False)


@pytest.mark.parametrize("news", NEWS)
def test_nothing_but_zero_rows(pkv, news):
    s = make(8, [100, 333], news, 8, 2, 128, v_sizes=lambda rng, shape: np.zeros(shape))
    assert (call(pkv, s) == 0).all()
    s = make(9, [100, 333], news, 8, 2, 128, k_sizes=lambda rng, shape: np.zeros(shape))
    check(call(pkv, s), *reference(s))
    s["q"].zero_()
    check(call(pkv, s), *reference(s))


@pytest.mark.parametrize("news", NEWS[1:])
@pytest.mark.parametrize("d", [64, 128])
def test_hidden_tokens_hold_anything(pkv, news, d):
    """Each sequence's last token has a NaN K scale and an infinite V scale: the rows before it are right, its own
    rows are not numbers."""
    s = make(10, [300, 170], news, 8, 2, d)
    want, bound = reference(s)
    view, put = scales_of(s)
    for i, n in enumerate(s["lens_list"]):
        b, o = s["tables"][i, (n - 1) // B].item(), (n - 1) % B
        view[b, :, o], view[b, :, B + o] = np.nan, np.inf
    put()
    got = call(pkv, s)
    last = [news[0] - 1, sum(news) - 1]
    keep = [r for r in range(sum(news)) if r not in last]
    check(got[keep], want[keep], bound[keep])
    assert torch.isnan(got[last].float()).all()


@pytest.mark.parametrize("news", NEWS)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_queries_that_are_not_numbers_stay_alone(pkv, news, bad):
    s = make(11, [300, 170], news, 8, 2, 128)
    want, bound = reference(s)
    s["q"][0, 1, 5] = bad
    s["q"][-1, 7, 127] = bad
    got = call(pkv, s)
    spoilt = torch.zeros(got.shape[:2], dtype=torch.bool, device="cuda")
    spoilt[0, 1] = spoilt[-1, 7] = True
    check(got[~spoilt], want[~spoilt], bound[~spoilt])
    assert not torch.isfinite(got[spoilt].float()).any()


@pytest.mark.parametrize("news", NEWS)
def test_negative_scale(pkv, news):
    s = make(12, [300, 170], news, 8, 2, 128)
    s["scale"] = -0.2
    check(call(pkv, s), *reference(s))
