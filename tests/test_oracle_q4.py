"""Pins of the 4-bit cache's, the rotary and the planning oracles (CPU)."""

import math

import numpy as np
import pytest

from oracle import plan as plan_oracle
from oracle import quant4 as Q
from oracle import rotary as R
from oracle.paged_pool import PagedKVPool


@pytest.mark.parametrize("d", [64, 128])
def test_places_cover_the_record_once(d):
    seen = set()
    for t in range(16):
        for e in range(d):
            seen |= {Q.k_place(d, t, e), Q.v_place(d, t, e)}
    assert seen == {(b, s) for b in range(16 * d) for s in (0, 4)}
    assert Q.record_bytes(d) == 16 * d + 128


@pytest.mark.parametrize("d", [64, 128])
def test_a_byte_holds_one_token(d):
    """Tokens of a block are written without reading what is there."""
    for place in (Q.k_place, Q.v_place):
        owner = {}
        for t in range(16):
            for e in range(d):
                assert owner.setdefault(place(d, t, e)[0], t) == t


@pytest.mark.parametrize("d", [64, 128])
def test_pack_unpack_and_append_agree(d):
    rng = np.random.default_rng(3)
    x, y = rng.standard_normal((2, 3, 16, d)).astype(np.float32).astype(np.float64), rng.standard_normal((2, 3, 16, d))
    y = y.astype(np.float32).astype(np.float64)
    kc, ks = Q.quantize_rows4(x)
    vc, vs = Q.quantize_rows4(y)
    packed = Q.pack(kc, vc, ks, vs)
    for a, b in zip(Q.unpack(packed, d), (kc, vc, ks, vs)):
        assert np.array_equal(a, b)
    cache = np.full_like(packed, 0xA5)
    slots = np.arange(32)
    Q.append_tokens_q4(cache, x.transpose(0, 2, 1, 3).reshape(32, 3, d), y.transpose(0, 2, 1, 3).reshape(32, 3, d), slots)
    assert np.array_equal(cache, packed)
    before = cache.copy()
    Q.append_tokens_q4(cache, x.reshape(-1, 3, d)[:2], y.reshape(-1, 3, d)[:2], [-1, -7])
    assert np.array_equal(cache, before)


def test_codes_are_the_exact_quotients():
    rng = np.random.default_rng(4)
    for size in (1.0, 1e-30, 3e4, 1e30):
        x = (rng.standard_normal((64, 16)) * size).astype(np.float32).view(np.uint32)
        x = (x & 0xffff0000).view(np.float32).astype(np.float64)          # bf16 values: borders are met often
        codes, scales = Q.quantize_rows4(x)
        for r in range(64):
            assert [Q.code_exactly(v, scales[r]) for v in x[r]] == codes[r].tolist()
        assert np.abs(codes).max() == 7
        assert np.all(np.abs(codes * scales.astype(np.float64)[:, None] - x) <= scales[:, None] * (0.5 + 2.0 ** -20))


def test_zero_row_and_scale():
    codes, scales = Q.quantize_rows4(np.zeros((2, 64)))
    assert not codes.any() and not scales.any()
    codes, scales = Q.quantize_rows4(np.array([[7.0, -3.5, 0.4, 0.0]]))
    assert scales[0] == np.float32(7) * (np.float32(1) / np.float32(7)) and codes[0, 0] == 7


def test_attention_against_contiguous_values():
    rng = np.random.default_rng(5)
    d, kv, heads, n, new = 64, 2, 6, 37, 3
    kc, ks = Q.quantize_rows4(rng.standard_normal((5, kv, 16, d)))
    vc, vs = Q.quantize_rows4(rng.standard_normal((5, kv, 16, d)))
    cache, table = Q.pack(kc, vc, ks, vs), np.array([[4, 0, 2]])
    q = rng.standard_normal((new, heads, d))
    got = Q.attention_q4(q, cache, table, [n], [0, new], 0.2)
    k, v = (a * s[..., None].astype(np.float64) for a, s in ((kc, ks), (vc, vs)))
    for t in range(new):
        for h in range(heads):
            keys = np.concatenate([k[b, h // 3] for b in table[0]])[:n - new + 1 + t]
            vals = np.concatenate([v[b, h // 3] for b in table[0]])[:n - new + 1 + t]
            w = np.exp(0.2 * keys @ q[t, h])
            assert np.allclose(got[t, h], w @ vals / w.sum(), rtol=1e-12)
    one = Q.attention_q4(q[-1:], cache, table, [n], None, 0.2)
    assert np.allclose(one[0], got[-1])
    absent = Q.attention_q4(q[-1:], cache, np.array([[4, 77, 2]]), [n], None, 0.2)
    short = Q.attention_q4(q[-1:], cache, np.array([[4, 2]]), [n - 16], None, 0.2)
    assert np.allclose(absent, short)


def test_turning_is_a_rotation_and_depends_on_the_distance():
    rng = np.random.default_rng(6)
    f = R.frequencies(32, 10000.0)
    x, y = rng.standard_normal((2, 1, 1, 64))
    for interleaved in (False, True):
        at = lambda z, p: R.turn(z, R.table(f, [p]), interleaved)[0, 0]  # noqa: E731
        assert np.allclose(at(x, 0), x[0, 0])
        assert math.isclose(np.linalg.norm(at(x, 77)), np.linalg.norm(x))
        assert np.array_equal(at(x, 5)[32:], x[0, 0, 32:])
        assert math.isclose(at(x, 17) @ at(y, 12), at(x, 1005) @ at(y, 1000), rel_tol=1e-9)
    assert np.allclose(R.turn(np.eye(1, 64).reshape(1, 1, 64), R.table(f, [1]), False)[0, 0][[0, 16]], [math.cos(1), math.sin(1)])
    assert np.allclose(R.turn(np.eye(1, 64).reshape(1, 1, 64), R.table(f, [1]), True)[0, 0][[0, 1]], [math.cos(1), math.sin(1)])


@pytest.mark.parametrize("kind,more", [("plain", {}), ("linear", dict(stretch=4.0)), ("base", dict(stretch=8.0)),
                                       ("turns", dict(stretch=8.0, original_context=8192, low_turns=1, high_turns=4)),
                                       ("ramp", dict(stretch=4.0, original_context=4096, low_turns=1, high_turns=32)),
                                       ("ramp", dict(stretch=2.0, original_context=7, low_turns=1, high_turns=32))])
@pytest.mark.parametrize("dim,base", [(128, 500000.0), (64, 10000.0), (6, 100.0)])
def test_frequencies_of_the_library(kind, more, dim, base):
    from paged_kv_cache_209_gb300 import pkv
    got = pkv.pkv_rotary_frequencies(dim, base, kind, **more).numpy()
    assert np.allclose(got, R.frequencies(dim, base, kind, **more), rtol=1e-13, atol=0)
    plain = R.frequencies(dim, base)
    assert np.all(got <= plain * (1 + 1e-13)) and np.all(got >= plain / more.get("stretch", 1.0) * (1 - 1e-12))


@pytest.mark.parametrize("bad", [dict(rotary_dim=3), dict(rotary_dim=0), dict(base=1.0), dict(base=float("nan")),
                                 dict(kind="linear", stretch=0.5), dict(kind="linear", stretch=float("inf")),
                                 dict(kind="base", rotary_dim=2, stretch=2.0), dict(kind="turns", stretch=2.0),
                                 dict(kind="ramp", stretch=2.0, original_context=8, low_turns=4, high_turns=2)])
def test_frequencies_refused(bad):
    from paged_kv_cache_209_gb300 import pkv
    with pytest.raises(pkv.PkvError, match="PKV_ERR_SHAPE"):
        pkv.pkv_rotary_frequencies(**{**dict(rotary_dim=64), **bad})
    with pytest.raises(ValueError):
        pkv.pkv_rotary_frequencies(64, kind="other")


def test_plan_follows_the_page_pool():
    """The pool's own appends, sequence by sequence, give the plan's slots and tables."""
    rng = np.random.default_rng(7)
    pool = PagedKVPool(60, 16, pop_order=rng.permutation(60))
    lens = [0, 5, 16, 31, 64, 1]
    for i, n in enumerate(lens):
        pool.create(i)
        pool.append(i, n)
    order = []
    probe = PagedKVPool(60, 16, pop_order=np.random.default_rng(7).permutation(60))
    probe.create("all")
    probe.append("all", 60 * 16)
    order = [int(b) for b in probe.page_table("all")]
    used = sum(-(-n // 16) for n in lens)
    free = order[used:][::-1]                               # the next one handed out lies last
    tables = np.full((6, 8), -1, np.int32)
    for i in range(6):
        t = pool.page_table(i)
        tables[i, :len(t)] = t
    new = [1, 12, 0, 33, 1, 15]
    got = plan_oracle.plan(lens, new, [-(-n // 16) for n in lens], free, len(free), tables, 70)
    want = []
    for i, m in enumerate(new):
        n = pool.sequence_length(i)
        pool.append(i, m)
        want += pool.slots(i, n, m)
    assert got["slots"][:62].tolist() == [int(s) for s in want] and set(got["slots"][62:]) == {-1}
    for i in range(6):
        t = [int(b) for b in pool.page_table(i)]
        assert got["tables"][i, :len(t)].tolist() == t
    assert not got["bad"] and got["result"] == [62, 0]
    assert plan_oracle.plan(lens, new, [-(-n // 16) for n in lens], free, 2, tables, 70)["result"][1] == 3
