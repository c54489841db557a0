"""The 4-bit cache's calls as a serving loop makes them: plan -> rotary append ->
attention -> verification -> plan, on the device alone, eager and as a captured graph; calls
on other streams and of all sizes on one workspace."""

import numpy as np
import pytest
import torch

from oracle import plan as P
from oracle import quant4 as Q
from oracle import rotary as R
from oracle.verify import verify_batch
from q4_cases import check, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


HEADS, KV, D, VOCAB, BATCH, WIDTH, BLOCKS = 8, 2, 128, 97, 5, 12, 60


def model(step, rows):
    """What a model would put out for the step's rows: q, k, v, and the target's probabilities."""
    g = torch.Generator().manual_seed(1000 + step)
    qkv = torch.randn((rows, (HEADS + 2 * KV) * D), generator=g).to(torch.bfloat16).cuda()
    probs = torch.softmax(2 * torch.randn((rows, VOCAB), generator=g), -1).cuda()
    return qkv, probs


def parts(qkv):
    rows = qkv.shape[0]
    return (qkv[:, :HEADS * D].view(rows, HEADS, D), qkv[:, HEADS * D:(HEADS + KV) * D].view(rows, KV, D),
            qkv[:, (HEADS + KV) * D:].view(rows, KV, D))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_loop_without_the_host(pkv):
    """Prompts, then steps of three drafts each; every step against the oracles run beside it."""
    rng = np.random.default_rng(0)
    prompts, drafts = [17, 1, 48, 5, 33], 3
    free = rng.permutation(BLOCKS).astype(np.int32)
    table = pkv.pkv_rotary_table(pkv.pkv_rotary_frequencies(D).cuda(), WIDTH * 16)
    cache = torch.randint(0, 256, (BLOCKS, KV, Q.record_bytes(D)), dtype=torch.uint8, device="cuda")
    mirror = cache.cpu().numpy().copy()
    state = dict(lens=i32([0] * BATCH), held=i32([0] * BATCH), left=i32([BLOCKS]), tables=torch.full((BATCH, WIDTH), -1,
                 dtype=torch.int32, device="cuda"))
    host = dict(lens=np.zeros(BATCH, np.int32), held=np.zeros(BATCH, np.int32), left=BLOCKS, tables=np.full((BATCH, WIDTH), -1, np.int32))
    need = pkv.pkv_multiquery_q4_workspace_size(BATCH, HEADS, WIDTH, max(prompts), cache)
    work = torch.zeros(need, dtype=torch.uint8, device="cuda")
    dstart = i32([drafts * i for i in range(BATCH + 1)])
    for step in range(6):
        new = prompts if step == 0 else [drafts + 1] * BATCH
        rows = sum(new)
        room = rows + 3                                      # as a captured step would be padded
        slots, pos, start, lens, held, left, result = pkv.pkv_plan_step(
            state["lens"], i32(new), state["held"], torch.from_numpy(free).cuda(), state["left"], state["tables"], room, BLOCKS)
        want = P.plan(host["lens"], new, host["held"], free, host["left"], host["tables"], room, BLOCKS)
        assert np.array_equal(slots.cpu().numpy(), want["slots"]) and np.array_equal(state["tables"].cpu().numpy(), want["tables"])
        assert result.tolist() == [rows, 0] and np.array_equal(start.cpu().numpy(), want["start"])
        qkv, probs = model(step, room)
        q, k, v = parts(qkv)
        turned = pkv.pkv_append_rotary(q, k, v, pos, table, slots, cache, q_out=torch.zeros_like(q).contiguous())
        angles = table.double().cpu().numpy()[want["positions"][:rows]]
        bf16 = lambda x: torch.from_numpy(x).float().to(torch.bfloat16)  # noqa: E731
        kt = bf16(R.turn(k[:rows].double().cpu().numpy(), angles, False)).double().numpy()
        qt = bf16(R.turn(q[:rows].double().cpu().numpy(), angles, False))
        assert torch.equal(turned[:rows].cpu(), qt) and not turned[rows:].any()
        Q.append_tokens_q4(mirror, kt, v[:rows].double().cpu().numpy(), want["slots"][:rows])
        assert np.array_equal(cache.cpu().numpy(), mirror)
        out = pkv.pkv_multiquery_attention_q4(turned, cache, state["tables"], lens, start, 0.09, max(new), workspace=work)
        exp = Q.attention_q4(qt.double().numpy(), mirror, want["tables"], want["lens"], want["start"], 0.09)
        got = out[:rows].double().cpu().numpy()
        assert np.linalg.norm(got - exp) <= 2.5e-3 * np.linalg.norm(exp)
        host.update(lens=want["lens"], held=want["held"], left=want["left"], tables=want["tables"])
        if step:
            # drafts that are likely, or not: some are kept
            g = torch.Generator().manual_seed(step)
            tokens = torch.randint(0, VOCAB, (BATCH * drafts,), generator=g).to(torch.int32).cuda()
            u, w = torch.rand(BATCH * drafts, generator=g).cuda() * 0.02, torch.rand(BATCH, generator=g).cuda()
            toks, kept, lens = pkv.pkv_verify_drafts(probs[:rows].contiguous(), None, tokens, u, w, start, dstart, drafts,
                                                     context_lens=lens)
            wt, wk, _ = verify_batch(probs[:rows].cpu().numpy(), None, tokens.cpu().numpy(), u.cpu().numpy(), w.cpu().numpy(),
                                  want["start"], dstart.cpu().numpy(), drafts)
            wl = want["lens"] - (drafts - np.array(wk))
            assert toks.tolist() == np.asarray(wt).tolist() and kept.tolist() == list(wk) and lens.tolist() == list(wl)
            host["lens"] = np.array(wl, np.int32)
        state.update(lens=lens, held=held, left=left)
    assert 0 < int(host["left"]) < BLOCKS


def test_captured_step(pkv):
    """A decode step captured once and replayed: two plans in turn, so that lengths go from one buffer to the other."""
    lens, news = [40, 3, 100, 16], [1] * 4
    s = make(3, lens, news, HEADS, KV, D, width=10)
    blocks = s["cache"].shape[0]
    grown = torch.cat([s["cache"], torch.zeros((8, KV, Q.record_bytes(D)), dtype=torch.uint8, device="cuda")])
    free = torch.arange(blocks, blocks + 8, dtype=torch.int32, device="cuda")
    table = pkv.pkv_rotary_table(pkv.pkv_rotary_frequencies(D).cuda(), 200)
    qkv = torch.randn((4, (HEADS + 2 * KV) * D), device="cuda").to(torch.bfloat16)
    work = torch.zeros(pkv.pkv_multiquery_q4_workspace_size(4, HEADS, 10, 1, grown), dtype=torch.uint8, device="cuda")
    ones = torch.ones(4, dtype=torch.int32, device="cuda")

    def fresh():
        return dict(cache=grown.clone(), tables=s["tables"].clone(), lens=s["lens"].clone(), held=i32([-(-n // 16) for n in lens]),
                    left=i32([8]))

    def two(st):
        now, outs = (st["lens"], st["held"], st["left"]), []
        for _ in range(2):
            slots, pos, start, *now, result = pkv.pkv_plan_step(now[0], ones, now[1], free, now[2], st["tables"], 6)
            q, k, v = parts(torch.cat([qkv, qkv[:2]]))
            turned = pkv.pkv_append_rotary(q, k, v, pos, table, slots, st["cache"], q_out=torch.zeros_like(q).contiguous())
            outs.append(pkv.pkv_decode_attention_q4(turned[:4], st["cache"], st["tables"], now[0], 0.1, workspace=work))
        for name, x in zip(("lens", "held", "left"), now):
            st[name].copy_(x)
        return outs
    eager, captured = fresh(), fresh()
    two(fresh())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        outs = two(captured)
    for _ in range(3):
        want = two(eager)
        graph.replay()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        for name in eager:
            assert torch.equal(eager[name], captured[name]), name
    assert eager["lens"].tolist() == [46, 9, 106, 22]


SIZES = [([900, 30], [1, 1], 8, 2), ([5], [5], 8, 2), ([300, 2, 700], [70, 1, 200], 4, 2), ([2000], [1], 16, 2),
         ([64] * 40, [2] * 40, 8, 2), ([1500, 40], [6, 4], 8, 2)]


def test_one_workspace_for_calls_of_all_sizes(pkv):
    cases = [make(20 + i, lens, news, h, kv, D, width=130) for i, (lens, news, h, kv) in enumerate(SIZES)]
    need = max(pkv.pkv_multiquery_q4_workspace_size(len(c["news"]), c["q"].shape[1], 130, max(c["news"]), c["cache"]) for c in cases)
    work = torch.zeros(need, dtype=torch.uint8, device="cuda")
    wants = [reference(c) for c in cases]
    for turn in range(2):
        for c, (want, bound) in list(zip(cases, wants))[::1 if turn else -1]:
            got = pkv.pkv_multiquery_attention_q4(c["q"], c["cache"], c["tables"], c["lens"], c["start"], c["scale"], max(c["news"]),
                                                  workspace=work)
            check(got, want, bound)
            if max(c["news"]) == 1:
                check(pkv.pkv_decode_attention_q4(c["q"], c["cache"], c["tables"], c["lens"], c["scale"], workspace=work), want, bound)


def test_other_streams(pkv):
    """Two calls at once, each on its stream with its own workspace; outputs that the call allocates belong to it."""
    cases = [make(30 + i, lens, news, 8, 2, D) for i, (lens, news) in enumerate((([3000, 40], [1, 1]), ([500], [200])))]
    wants = [reference(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [pkv.pkv_multiquery_attention_q4(c["q"], c["cache"], c["tables"], c["lens"], c["start"], c["scale"], max(c["news"]), stream=st)
               for c, st in zip(cases, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, wants):
            check(g, *w)


def test_repeated_calls_give_the_same_bytes(pkv):
    for lens, news in (([2500, 7, 900], [1, 1, 1]), ([1200, 800], [4, 3]), ([900, 600], [150, 90])):
        s = make(40, lens, news, 16, 4, D)
        first = pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["start"], s["scale"], max(news))
        for _ in range(5):
            again = pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["start"], s["scale"], max(news))
            assert torch.equal(first, again)


def test_more_sequences_than_a_launch_holds(pkv):
    lens = [1 + i % 40 for i in range(1500)]
    s = make(50, lens, [1] * 1500, 4, 2, 64)
    want, bound = reference(s, decode=True)
    check(pkv.pkv_decode_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["scale"]), want, bound)
    check(pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["start"], s["scale"], 1), want, bound)


def test_refusals_of_the_binding(pkv):
    s = make(60, [20, 9], [1, 1], 8, 2, D)
    call = lambda **kw: pkv.pkv_decode_attention_q4(  # noqa: E731
        kw.get("q", s["q"]), kw.get("c", s["cache"]), kw.get("t", s["tables"]), kw.get("l", s["lens"]), 0.1, out=kw.get("o"),
        workspace=kw.get("w"))
    for bad in (dict(q=s["q"].float()), dict(q=s["q"][:, :, :64]), dict(q=s["q"][:1]), dict(q=s["q"].transpose(0, 1)), dict(c=s["cache"].to(torch.int8)),
                dict(c=s["cache"][:, :, :2000]), dict(c=s["cache"][:, :1].expand(-1, 2, -1)), dict(t=s["tables"].long()),
                dict(t=s["tables"][0]), dict(l=s["lens"][:1]), dict(l=s["lens"].cpu()), dict(q=s["q"].cpu()), dict(o=s["q"].float())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(pkv.PkvError, match="PKV_ERR_WORKSPACE"):
        call(w=torch.zeros(128, dtype=torch.uint8, device="cuda"))
    assert call(q=s["q"][:0], t=s["tables"][:0], l=s["lens"][:0]).shape == (0, 8, D)


@pytest.mark.parametrize("lens,news,kv", [([700] * 14, [1] * 14, 8), ([700] * 9, [4] * 9, 8), ([1000], [1], 8), ([300] * 8, [1] * 8, 3),
                                          ([0] * 3 + [320] * 5, [0] * 3 + [2] * 5, 2), ([1024], [8], 8), ([4000], [1], 8),
                                          ([16] * 30, [1] * 30, 8), ([641, 650, 656], [1] * 3, 8)])
def test_few_contexts_of_one_length(pkv, lens, news, kv):
    """(Fewer CTAs than fit, a whole number for each (sequence, KV head).)"""
    s = make(70, lens, news, 4 * kv, kv, D)
    check(pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["start"], s["scale"], max(news)), *reference(s))
