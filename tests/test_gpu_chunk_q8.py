"""pkv_multiquery_attention_q8 against the float64 oracle over the values the
cached rows stand for.

Tolerance, per element, with A = sum_p softmax_p |V_p| of its row and B the
largest scale * |q||K_p| its scores can reach (Cauchy-Schwarz):
  * the output's rounding to bf16: 2^-8 |ref| (half a step, eps / 2);
  * three roundings to f16 (the weight, the V scale, code * scale): 3 * 2^-11 A;
  * K's rounding to f16, half a step 2^-11 of each value: at most 2^-11 B in the score,
    counted twice (numerator and denominator); below f16's normal range half its
    smallest step, 2^-25 2^F <= 2^-11 ks (scales in plain steps are at least
    2^(F - 14)), at most 2^-11 scale |q|_1 ks;
  * the score: D + 2 float32 operations on products that sum to at most B in
    size, 2^-22 each (a truncating adder loses a whole step), a relative change
    of the weight, counted twice (numerator and denominator): 2 (D + 2) 2^-22 B A;
  * exp2 and the running sums: 2^-20 A and n 2^-23 A;
  * f16's smallest step, 2^-24, half of which a weight below the normal range may
    lose: the largest weight of a row is at least 1 (the maximum that is
    subtracted is never above it) and the sum with it, so the n seen tokens lose
    at most n 2^-25 max|V_p[d]| together;
  * the same for a scaled V value, 2^-25 2^E: a step keeps the scaled values only
    if its V scales are at least 2^(E - 14), so that is at most 2^-11 vs_p, in
    the weighted mean 2^-11 sum_p softmax_p vs_p.
"""

import math

import numpy as np
import pytest
import torch

import cases
from oracle import attention as OA
from oracle import multiquery as OM
from oracle import quant as OQ
from paged_kv_cache_209_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_209_gb300 import pkv as P
    P.load_library()
    P.pkv_device_status(clear=True)
    return P


def make(seed, lens, nqs, q_heads, kv_heads, d, kscale=1.0, vscale=1.0):
    c = cases.multiquery_case(seed, lens, nqs, q_heads, kv_heads, d, torch.bfloat16)
    c["kc"], c["ks"] = OQ.quantize_rows(OA.bf16_bits_to_f64(cases.host_view(c["k_pool"])) * kscale)
    c["vc"], c["vs"] = OQ.quantize_rows(OA.bf16_bits_to_f64(cases.host_view(c["v_pool"])) * vscale)
    c["scale"] = float(np.float32(c["scale"]))
    return c


def live_slots(c):
    live = np.zeros((c["kc"].shape[0], 16), dtype=bool)
    for i, n in enumerate(c["lens"]):
        for t in range(int(n)):
            live[c["tables"][i, t // 16], t % 16] = True
    return live


def poison(c):
    """Slots no sequence holds: NaN K scales, infinite V scales."""
    live = live_slots(c)
    c["ks"].transpose(0, 2, 1)[~live] = np.nan
    c["vs"].transpose(0, 2, 1)[~live] = np.inf
    return c


def device(c):
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    return dict(q=c["q"].cuda(), kc=dev(c["kc"]), vc=dev(c["vc"].transpose(0, 1, 3, 2)),
                sc=dev(np.stack([c["ks"], c["vs"]], axis=2)), tables=dev(c["tables"]), lens=dev(c["lens"]),
                start=dev(c["query_start"]))


def call(pkv, c, d=None, **kw):
    d = d or device(c)
    most = kw.pop("most", max(1, int(np.diff(c["query_start"]).max())))
    return pkv.pkv_multiquery_attention_q8(d["q"], d["kc"], d["vc"], d["sc"], d["tables"], d["lens"], d["start"],
                                           c["scale"], most, **kw)


def score_error(scale, q, k_norm, k_scale):
    """How far a score of each row may be off: f16 K values, float32 sums."""
    d = q.shape[-1]
    b = abs(scale) * np.linalg.norm(q, axis=-1) * k_norm
    return b * (2.0 ** -11 + (d + 2) * 2.0 ** -22) + 2.0 ** -11 * abs(scale) * np.abs(q).sum(-1) * k_scale


def reference(c):
    """(output, tolerance) in float64."""
    with np.errstate(invalid="ignore"):
        kd, vd = OQ.dequantize_rows(c["kc"], c["ks"]), OQ.dequantize_rows(c["vc"], c["vs"])
    dead = ~live_slots(c)
    kd.transpose(0, 2, 1, 3)[dead] = 0
    vd.transpose(0, 2, 1, 3)[dead] = 0
    qf = OA.bf16_bits_to_f64(cases.host_view(c["q"]))
    attend = lambda v: OM.multiquery_attention(qf, kd, v, c["tables"], c["lens"], c["query_start"], c["scale"],  # noqa: E731
                                               c["kv_heads"], "f64")
    ref, size = attend(vd), attend(np.abs(vd))
    d, n = qf.shape[2], int(max(c["lens"]))
    alive = lambda x: np.where(dead.reshape(-1, 1, 16), 0.0, np.abs(x.astype(np.float64)))  # noqa: E731
    b = score_error(c["scale"], qf, np.linalg.norm(kd, axis=-1).max(initial=0), alive(c["ks"]).max(initial=0))[..., None]
    tol = 2.0 ** -8 * np.abs(ref) + size * (3 * 2.0 ** -11 + 2 * b + 2.0 ** -20 + n * 2.0 ** -23)
    scales = alive(c["vs"])
    tol += 2.0 ** -11 * attend(np.broadcast_to(scales[..., None], vd.shape))
    group = qf.shape[1] // c["kv_heads"]
    for i, n in enumerate(c["lens"]):                          # the largest |V| among the tokens each row sees
        q0, q1 = c["query_start"][i], c["query_start"][i + 1]
        pos = np.arange(int(n))
        rows = np.abs(vd[c["tables"][i, pos // 16], :, pos % 16])
        top = np.maximum.accumulate(rows, axis=0)[int(n) - (q1 - q0):] if n else rows
        tol[q0:q1] += n * 2.0 ** -25 * np.repeat(top, group, axis=1)
    return ref, tol


def check(out, c, want=None):
    ref, tol = want or reference(c)
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - ref)[bad][:5], tol[bad][:5])


SHAPES = [
    # several sequences: a whole prompt, an empty one, one query, chunks behind a cached prefix
    ([40, 200, 0, 1, 129, 700], [40, 33, 0, 1, 0, 70], 32, 8, 128),
    ([40, 200, 0, 1, 129, 700], [40, 33, 0, 1, 0, 70], 16, 2, 64),
    # around the kernel's steps of 128 tokens and tiles of 128 and 256 rows
    ([127, 128, 129, 255, 256, 257], [127, 128, 129, 64, 65, 63], 8, 2, 128),
    ([127, 128, 129, 255, 256, 257], [127, 128, 129, 255, 256, 257], 2, 2, 64),
    ([300, 310, 640], [256, 257, 255], 1, 1, 128),
    # group sizes that do not divide a tile
    ([500, 77, 260], [90, 77, 201], 24, 8, 128),
    ([500, 77, 260], [90, 77, 201], 10, 2, 64),
    ([333, 90], [33, 19], 7, 1, 128),
    ([200, 50, 18], [9, 5, 1], 128, 1, 128),
    ([150, 40], [3, 2], 1024, 2, 64),
    # single tokens and short drafts at head_dim 64 (no other int8 attention takes them)
    ([1, 16, 17, 300, 1000, 64], [1, 1, 1, 1, 1, 1], 32, 8, 64),
    ([30, 16, 170, 300], [4, 3, 0, 2], 8, 8, 64),
    # few rows on long contexts (the context is split)
    ([5000, 3000], [9, 12], 32, 8, 128),
    ([4500], [70], 8, 8, 128),
    ([700, 40, 129, 9], [8, 3, 0, 5], 32, 8, 128),
]


@pytest.mark.parametrize("nqs,hq", [([1, 1, 1, 1, 1], 32), ([4, 3, 0, 2, 4], 32), ([2, 1, 2, 2, 0], 64)])
def test_few_rows_and_wide_tables(pkv, nqs, hq):
    """Up to 16 rows: the kernel that splits the cache where the tables are wide, tiles where they are not."""
    c = make(hq + nqs[0], [700, 40, 129, 9, 3000], nqs, hq, 8, 128)
    want = reference(c)
    narrow = call(pkv, c)
    c["tables"] = np.pad(c["tables"], ((0, 0), (0, 1200)), constant_values=-1)      # entries no sequence uses
    wide = call(pkv, c)
    check(narrow, c, want)
    check(wide, c, want)
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("lens,nqs,hq,hkv,d", SHAPES)
def test_matches_oracle(pkv, lens, nqs, hq, hkv, d):
    c = poison(make(sum(lens) + hq + d, lens, nqs, hq, hkv, d))
    check(call(pkv, c), c)
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_attention_scales(pkv, d, scale):
    c = make(3, [300, 65], [60, 65], 8, 2, d)
    c["scale"] = scale
    check(call(pkv, c), c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kscale,vscale", [(1e-3, 1e-3), (1.0, 1e-6), (8.0, 1e3), (1e-4, 1e8)])
def test_value_ranges(pkv, d, kscale, vscale):
    c = make(5, [400, 130], [70, 130], 8, 2, d, kscale, vscale)
    check(call(pkv, c), c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("factor", [1e2, 1e5, 1e20])
def test_v_rows_far_larger_than_the_others(pkv, d, factor):
    """A fifth of the V rows larger by a factor that leaves f16, first seen at the
    beginning of a context, in its middle or only at its end."""
    c = make(6, [600, 500, 700, 90], [60, 90, 40, 90], 8, 2, d)
    rng = np.random.default_rng(9)
    for i, (a, b) in enumerate([(0, 600), (300, 500), (690, 700), (0, 90)]):
        for t in range(a, b):
            if rng.random() < 0.2 or t == b - 1:
                c["vs"][c["tables"][i, t // 16], :, t % 16] *= np.float32(factor)
    check(call(pkv, c), c)


def test_zero_rows_and_wide_scales(pkv):
    """Zero rows have scale 1; other rows' scales span four orders of magnitude."""
    c = make(7, [300, 200], [80, 200], 8, 2, 128)
    rng = np.random.default_rng(8)
    c["ks"] = (c["ks"] * rng.uniform(1e-3, 3, c["ks"].shape)).astype(np.float32)
    c["vs"] = (c["vs"] * rng.uniform(1e-2, 1e2, c["vs"].shape)).astype(np.float32)
    for pool, scales in ((c["kc"], c["ks"]), (c["vc"], c["vs"])):
        zero = rng.random(scales.shape) < 0.1
        pool[zero] = 0
        scales[zero] = 1.0
    check(call(pkv, c), c)


@pytest.mark.parametrize("d", [64, 128])
def test_large_scores(pkv, d):
    """Peaked rows: scores in the hundreds, later tokens far above earlier ones."""
    c = make(8, [500, 260], [50, 260], 8, 2, d)
    ramp = np.linspace(0.5, 30, 500)
    for i, n in enumerate(c["lens"]):
        for t in range(int(n)):
            c["ks"][c["tables"][i, t // 16], :, t % 16] *= np.float32(ramp[t])
    check(call(pkv, c), c)


@pytest.mark.parametrize("d", [64, 128])
def test_tokens_a_row_may_not_see_hold_anything(pkv, d):
    """The chunk's last token has an infinite V scale and a NaN K scale: the rows
    before it are right (its own row is not a number)."""
    c = make(9, [140, 300], [140, 40], 8, 2, d)
    want = reference(c)
    for i, n in enumerate(c["lens"]):
        b, s = c["tables"][i, (n - 1) // 16], (n - 1) % 16
        c["ks"][b, :, s], c["vs"][b, :, s] = np.nan, np.inf
    out = call(pkv, c)
    keep = [r for r in range(180) if r not in (139, 179)]
    check(out[keep], c, (want[0][keep], want[1][keep]))
    assert bool(torch.isnan(out[[139, 179]].float()).all())


@pytest.mark.parametrize("d", [64, 128])
def test_blocks_outside_the_pool_are_absent(pkv, d):
    """A bad block's tokens have no weight, the call reports it; a sequence whose
    every block is bad gives zero rows."""
    c = make(10, [300, 200, 60], [70, 50, 40], 8, 2, d)
    nb = c["kc"].shape[0]
    good = dict(c, tables=c["tables"].copy())
    c["tables"][0, 3], c["tables"][1, 12], c["tables"][2, :4] = nb, -1, 2 ** 31 - 1
    out = call(pkv, c)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
    ref, tol = np.zeros((160, 8, d)), np.zeros((160, 8, d))
    for i, bad in ((0, 3), (1, 12)):
        # the same rows with the bad block's tokens cut out of the context
        n, nq, q0 = int(c["lens"][i]), int(np.diff(c["query_start"])[i]), int(c["query_start"][i])
        for t in range(nq):
            seen = [p for p in range(n - nq + t + 1) if p // 16 != bad]
            blocks = good["tables"][i, np.array(seen) // 16]
            slots = np.array(seen) % 16
            k = c["kc"][blocks, :, slots].astype(np.float64) * c["ks"][blocks, :, slots][..., None]
            v = c["vc"][blocks, :, slots].astype(np.float64) * c["vs"][blocks, :, slots][..., None]
            q = OA.bf16_bits_to_f64(cases.host_view(c["q"]))[q0 + t]
            for h in range(8):
                x = c["scale"] * k[:, h // 4] @ q[h]
                w = np.exp(x - x.max())
                w /= w.sum()
                ref[q0 + t, h], size = w @ v[:, h // 4], w @ np.abs(v[:, h // 4])
                b = score_error(c["scale"], q[h], np.linalg.norm(k[:, h // 4], axis=1).max(), float(c["ks"].max()))
                tol[q0 + t, h] = 2.0 ** -8 * np.abs(ref[q0 + t, h]) + size * (
                    3 * 2.0 ** -11 + 2 * b + 2.0 ** -20 + 300 * 2.0 ** -23)
                tol[q0 + t, h] += 300 * 2.0 ** -25 * np.abs(v[:, h // 4]).max() + 2.0 ** -11 * float(c["vs"].max())
    check(out, c, (ref, tol))
    assert bool((out[120:] == 0).all())
    buf = torch.full_like(out, 5.0)
    with pytest.raises(pkv.PkvError) as e:
        call(pkv, c, out=buf, flags=pkv.PKV_FLAG_CHECKED)
    assert e.value.name == "PKV_ERR_RANGE" and bool((buf == 5.0).all())
    assert pkv.pkv_device_status(clear=True) == 0


def test_malformed_query_ranges(pkv):
    """More queries than tokens or than max_query_len, a negative range, a context
    past its table: no rows for that sequence, the others right."""
    c = make(11, [90, 60, 200], [40, 60, 50], 8, 2, 128)
    ref, tol = reference(c)
    rows = [slice(0, 40), slice(40, 100), slice(100, 150)]
    for change in ("tokens", "most", "past"):
        b = dict(c, lens=c["lens"].copy())
        kw = {}
        if change == "tokens":
            b["lens"][1] = 59
        if change == "past":
            b["lens"][1] = 16 * c["tables"].shape[1] + 1
        if change == "most":
            kw["most"] = 59
        buf = torch.full((150, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        call(pkv, b, out=buf, **kw)
        assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE
        assert bool((buf[rows[1]] == 5.0).all())
        for r in (rows[0], rows[2]):
            check(buf[r], c, (ref[r], tol[r]))
        buf.fill_(5.0)
        with pytest.raises(pkv.PkvError) as e:
            call(pkv, b, out=buf, flags=pkv.PKV_FLAG_CHECKED, **kw)
        assert e.value.name == "PKV_ERR_RANGE" and bool((buf == 5.0).all())
    b = dict(c, query_start=np.array([0, 40, 20, 70], dtype=np.int32))
    call(pkv, b, most=60)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVERR_RANGE


def test_rows_no_sequence_names_stay(pkv):
    """Rows before the first and behind the last sequence keep their bytes; a
    checked call is right."""
    c = make(12, [90, 200], [40, 51], 8, 2, 128)
    ref, tol = reference(c)
    d = device(c)
    d["q"] = torch.cat([d["q"][:7], d["q"], d["q"][:9]])
    d["start"] = d["start"] + 7
    buf = torch.full_like(d["q"], 5.0)
    call(pkv, c, d, out=buf, flags=pkv.PKV_FLAG_CHECKED)
    assert bool((buf[:7] == 5.0).all()) and bool((buf[98:] == 5.0).all())
    check(buf[7:98], c, (ref, tol))


def test_batch_above_one_launch(pkv):
    rng = np.random.default_rng(13)
    lens = rng.integers(0, 60, 1100)
    nqs = np.minimum(lens, rng.integers(0, 40, 1100))
    lens[1050], nqs[1050] = 900, 100
    c = make(13, lens, nqs, 2, 1, 64)
    check(call(pkv, c), c)


def test_one_workspace_many_calls(pkv):
    """One workspace, never cleared again, over calls of other shapes."""
    first = make(14, [3000, 1500], [40, 70], 8, 2, 128)
    second = make(15, [200, 1000, 64], [150, 20, 64], 8, 2, 128)
    need = max(pkv.pkv_multiquery_q8_workspace_size(len(c["lens"]), 8, c["tables"].shape[1], 150, device(c)["kc"])
               for c in (first, second))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    wants = {id(c): reference(c) for c in (first, second)}
    for c in (first, second, first, second, second):
        check(call(pkv, c, workspace=ws), c, wants[id(c)])
    with pytest.raises(pkv.PkvError) as e:
        call(pkv, first, workspace=ws[:128])
    assert e.value.name == "PKV_ERR_WORKSPACE"


def test_same_call_same_bytes(pkv):
    c = make(16, [2500, 900, 10], [60, 300, 10], 24, 8, 128)
    d = device(c)
    a = call(pkv, c, d)
    for _ in range(3):
        assert torch.equal(call(pkv, c, d).view(torch.int16), a.view(torch.int16))


def test_captured_and_replayed_and_two_streams(pkv):
    """A captured call replayed on other lengths and offsets; two calls at once on
    two streams, each on its own workspace."""
    a, b = make(17, [400, 300], [50, 64], 8, 2, 128), make(18, [399, 290], [64, 50], 8, 2, 128)
    d, wa, wb = device(a), reference(a), reference(b)
    ws = torch.zeros(pkv.pkv_multiquery_q8_workspace_size(2, 8, a["tables"].shape[1], 64, d["kc"]), dtype=torch.uint8,
                     device="cuda")
    call(pkv, a, d, most=64, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(pkv, a, d, most=64, workspace=ws)
    for c, want in ((b, wb), (a, wa), (b, wb)):
        for key, v in device(c).items():
            d[key].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        check(out, c, want)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    da, db = device(a), device(b)
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        for s, c, dd in ((streams[0], a, da), (streams[1], b, db)):
            with torch.cuda.stream(s):
                outs.append(call(pkv, c, dd))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        check(o, a if i % 2 == 0 else b, wa if i % 2 == 0 else wb)


def test_prefill512_layer_sampled(pkv):
    """The chunked-prefill workload over an int8 cache, every row of sampled heads
    and queries (float64 on the device)."""
    cfg = W.CONFIGS["prefill512"]
    tables, lens, nb = W.workload_index("prefill512")
    g = torch.Generator(device="cuda").manual_seed(19)
    codes = lambda shape, s: W.int8_codes(shape, s, "cuda")  # noqa: E731
    kc, vc = codes((nb, 8, 16, 128), 1), codes((nb, 8, 128, 16), 2)
    sc = torch.rand((nb, 8, 2, 16), generator=g, device="cuda") * 0.01 + 0.02
    q = torch.randn((8 * 512, 32, 128), generator=g, device="cuda").to(torch.bfloat16)
    start = torch.arange(0, 8 * 512 + 1, 512, dtype=torch.int32, device="cuda")
    t = torch.from_numpy(tables).cuda()
    scale = 1 / math.sqrt(128)
    out = pkv.pkv_multiquery_attention_q8(q, kc, vc, sc, t, torch.from_numpy(lens.astype(np.int32)).cuda(), start,
                                          scale, cfg["queries"])
    for i, h in ((0, 0), (3, 13), (7, 31)):
        blk = t[i].long()
        k = (kc[blk, h // 4].double() * sc[blk, h // 4, 0, :, None].double()).reshape(-1, 128)
        v = (vc[blk, h // 4].double() * sc[blk, h // 4, 1, None].double()).transpose(1, 2).reshape(-1, 128)
        qq = q[512 * i:512 * (i + 1), h].double()
        x = scale * qq @ k.T
        x = x.masked_fill(torch.arange(8192, device="cuda") > torch.arange(7680, 8192, device="cuda")[:, None], -math.inf)
        w = torch.softmax(x, -1)
        ref, size = w @ v, w @ v.abs()
        b = torch.from_numpy(score_error(scale, qq.cpu().numpy(), float(k.norm(dim=1).max()), 0.03)).cuda()[:, None]
        tol = 2.0 ** -8 * ref.abs() + size * (3 * 2.0 ** -11 + 2 * b + 2.0 ** -20 + 8192 * 2.0 ** -23)
        tol = tol + 8192 * 2.0 ** -25 * v.abs().max() + 2.0 ** -11 * 0.03
        assert bool(((out[512 * i:512 * (i + 1), h].double() - ref).abs() <= tol).all())
    assert pkv.pkv_device_status(clear=True) == 0


def test_one_workspace_for_calls_of_all_sizes_on_both_kernels(pkv):
    """The size for the largest call serves every smaller one, in any order: each
    result is the one a workspace of its own gives, bit for bit."""
    mixes = [([700, 900, 65], [300, 40, 65]), ([2000, 77, 31, 5000, 900], [2, 1, 2, 2, 1]), ([300] * 70, [2] * 70),
             ([900, 2500], [8, 8]), ([40, 3000], [40, 100])]
    built = [make(90 + i, lens, nqs, 16, 4, 128) for i, (lens, nqs) in enumerate(mixes)]
    on = [device(c) for c in built]
    need = pkv.pkv_multiquery_q8_workspace_size(70, 16, 313, 300, on[0]["kc"])
    shared = torch.zeros(need, dtype=torch.uint8, device="cuda")
    want = [call(pkv, c, d) for c, d in zip(built, on)]
    for i in [0, 1, 2, 1, 3, 0, 2, 4, 3, 2, 1]:
        size = pkv.pkv_multiquery_q8_workspace_size(len(built[i]["lens"]), 16, on[i]["tables"].shape[1],
                                                    int(np.diff(built[i]["query_start"]).max()), on[i]["kc"])
        assert size <= need
        got = call(pkv, built[i], on[i], workspace=shared)
        assert torch.equal(got, want[i]), i
    assert pkv.pkv_device_status(clear=True) == 0


def test_pools_past_32_bits(pkv):
    """Blocks more than 2^32 bytes into the pools: the result of the same rows in a small pool."""
    c = make(99, [700, 40, 300], [90, 3, 300], 8, 8, 128)
    d = device(c)
    want = call(pkv, c, d)
    few = d["kc"].shape[0]
    nb = 300_000                                             # 4.9 GB of codes in each pool
    big = {"kc": torch.empty((nb, 8, 16, 128), dtype=torch.int8, device="cuda"),
           "vc": torch.empty((nb, 8, 128, 16), dtype=torch.int8, device="cuda"),
           "sc": torch.empty((nb, 8, 2, 16), device="cuda")}
    at = torch.cat([torch.arange(few // 2), torch.arange(nb - few + few // 2, nb)]).cuda()    # some first, some last
    for name, pool in big.items():
        pool[at] = d[name]
    d.update(big, tables=at.to(torch.int32)[d["tables"].long().clamp_(min=0)])
    assert torch.equal(call(pkv, c, d), want)
    start = torch.tensor([0, 700, 740, 1040], dtype=torch.int32, device="cuda")
    read = lambda d: pkv.pkv_gather_q8(d["kc"], d["vc"], d["sc"], d["tables"], d["lens"], start, 1040)  # noqa: E731
    assert all(torch.equal(a, b) for a, b in zip(read(d), read(device(c))))
    assert pkv.pkv_device_status(clear=True) == 0


def test_many_more_units_than_ctas(pkv):
    """Some 5000 units: every round of whole units is in use; sampled sequences against the oracle."""
    rng = np.random.default_rng(6)
    nqs = rng.integers(200, 700, 250)
    lens = nqs + rng.integers(0, 200, 250)
    c = make(6, [int(n) for n in lens], [int(n) for n in nqs], 8, 8, 64)
    out = call(pkv, c)
    some = [0, 97, 151, 249]
    start = c["query_start"]
    rows = np.concatenate([np.arange(start[i], start[i + 1]) for i in some])
    part = dict(c, tables=c["tables"][some], lens=c["lens"][some], q=c["q"][rows],
                query_start=np.concatenate([[0], np.cumsum(nqs[some])]).astype(np.int32))
    check(out[torch.from_numpy(rows).cuda()], part)
    assert torch.isfinite(out).all()
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(pkv, seed):
    """Lengths, chunks, groups and the size of the cached rows drawn at random, some rows far larger or smaller."""
    rng = np.random.default_rng(700 + seed)
    hkv, d = int(rng.choice([1, 2, 4])), int(rng.choice([64, 128]))
    group = int(rng.choice([1, 2, 3, 4, 5, 8, 12]))
    lens = [int(n) for n in np.exp(rng.uniform(0, np.log(2500), rng.integers(1, 7)))]
    nqs = [int(rng.integers(0, min(n, 300) + 1)) for n in lens]
    c = make(seed, lens, nqs, group * hkv, hkv, d, kscale=2.0 ** rng.integers(-6, 2), vscale=2.0 ** rng.integers(-20, 20))
    if seed % 2:                                             # tokens whose scales leave the range of the others
        odd = rng.random(c["ks"].shape) < 0.01
        c["ks"][odd] *= np.float32(2.0) ** np.float32(-20)
        odd = rng.random(c["vs"].shape) < 0.01
        c["vs"][odd] *= np.float32(2.0) ** rng.choice([-26, 12], odd.sum()).astype(np.float32)
    check(call(pkv, poison(c)), c)
    assert pkv.pkv_device_status(clear=True) == 0
