"""Speculative serving over an int8 cache, the calls in the order a serving loop
makes them: quantizing append, attention of each sequence's new tokens, a small
output layer, verification of the drafts, and the verified lengths straight into
the next append (which overwrites the rejected tokens' slots); at the end the
sequences are read back out of the cache. Every step is checked against the
oracle; the same loop, one step captured into a CUDA graph, has to give the
same tokens and the same cache.

Tolerances: tokens, lengths, cache contents and rows read back are exact (the
probabilities are multiples of 2^-30, so every sum of a row is exact in 64 bits);
attention as derived in test_gpu_chunk_q8, and as the other tests of the kernel
that splits the cache have it.
"""

import numpy as np
import pytest
import torch

import cases
from oracle import attention as OA
from oracle import quant as OQ
from oracle import verify as OV
from test_gpu_chunk_q8 import reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_209_gb300 import pkv as P
    P.load_library()
    P.pkv_device_status(clear=True)
    return P


class Server:
    """Sequences with blocks of their own and a one-layer model with random weights."""

    def __init__(self, pkv, prompts, drafts, q_heads, kv_heads, d, steps, least_width=0, vocab=211):
        self.pkv, self.k, self.hq, self.hkv, self.d, self.vocab = pkv, drafts, q_heads, kv_heads, d, vocab
        self.batch, self.steps = len(prompts), steps
        gen = torch.Generator().manual_seed(17 * drafts + d)
        rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        bf = lambda x: x.to(torch.bfloat16).cuda()  # noqa: E731
        self.eq, self.ek, self.ev = bf(rand(vocab, q_heads, d)), bf(rand(vocab, kv_heads, d)), bf(rand(vocab, kv_heads, d))
        self.pos = bf(rand(64, kv_heads, d))
        self.head = (rand(q_heads * d, vocab) * (3.0 / (q_heads * d) ** 0.5)).cuda()
        self.draft_logits = (2 * rand(vocab, vocab)).cuda()
        self.prompts = [torch.randint(0, vocab, (n,), generator=gen) for n in prompts]
        width = max(least_width, (max(prompts) + (steps + 1) * (drafts + 1) + 15) // 16)
        blocks = self.batch * width + 3
        self.tables = torch.randperm(blocks, generator=gen)[:self.batch * width].reshape(self.batch, width).to(torch.int32).cuda()
        self.kc = torch.zeros((blocks, kv_heads, 16, d), dtype=torch.int8, device="cuda")
        self.vc = torch.zeros((blocks, kv_heads, d, 16), dtype=torch.int8, device="cuda")
        self.sc = torch.zeros((blocks, kv_heads, 2, 16), device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.qs = torch.arange(self.batch + 1, **i32) * (drafts + 1)
        self.ds = torch.arange(self.batch + 1, **i32) * drafts
        self.uniform = torch.rand(steps, self.batch, drafts + 1, generator=gen).cuda()
        self.choice = torch.rand(steps, self.batch * drafts, generator=gen).cuda()
        # the loop's state: tokens in the cache, the last token of each sequence (not yet in it)
        self.lens = torch.tensor([n - 1 for n in prompts], **i32)
        self.last = torch.tensor([int(p[-1]) for p in self.prompts], **i32)
        most = max(drafts + 1, max(prompts))
        self.workspace = torch.zeros(max(256, pkv.pkv_multiquery_q8_workspace_size(self.batch, q_heads, width, most, self.kc)),
                                     dtype=torch.uint8, device="cuda")

    def append(self, tokens, seq, at):
        """K and V of ``tokens`` into positions ``at`` of sequences ``seq``; returns what was appended."""
        slots = self.tables[seq, at // 16].long() * 16 + at % 16
        k, v = self.ek[tokens] + self.pos[at % 64], self.ev[tokens]
        self.pkv.pkv_append_q8(k, v, slots, self.kc, self.vc, self.sc)
        return k, v, slots

    def attend(self, tokens, lens, start, most):
        return self.pkv.pkv_multiquery_attention_q8(self.eq[tokens], self.kc, self.vc, self.sc, self.tables, lens, start,
                                                    self.d ** -0.5, most, workspace=self.workspace)

    def prefill(self):
        """The prompts but their last tokens, as one batch of chunks (a prompt of one token: none)."""
        lens = [len(p) - 1 for p in self.prompts]
        tokens = torch.cat([p[:-1] for p in self.prompts]).cuda()
        seq = torch.repeat_interleave(torch.arange(self.batch), torch.tensor(lens)).cuda()
        at = torch.cat([torch.arange(n) for n in lens]).cuda()
        start = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        moved = self.append(tokens, seq, at)
        return dict(moved=moved, q=self.eq[tokens], lens=self.lens.clone(), start=start,
                    out=self.attend(tokens, self.lens, start, max(lens)))

    def step(self, uniform, choice):
        """Draft, append, attend, verify; moves the state on."""
        t = self.k + 1
        rows, drafted = [], [self.last.long()]
        for j in range(self.k):                              # draft tokens from the draft model's rows
            p = self.grid(torch.softmax(self.draft_logits[drafted[-1]], -1))
            rows.append(p)
            u = choice.view(self.batch, self.k)[:, j:j + 1]
            drafted.append((p.cumsum(-1) <= u * p.sum(-1, keepdim=True)).sum(-1).clamp_(max=self.vocab - 1))
        tokens = torch.stack(drafted, 1)                     # [batch][k + 1]
        draft_probs = torch.stack(rows, 1).reshape(self.batch * self.k, self.vocab) if rows else None
        at = (self.lens.long()[:, None] + torch.arange(t, device="cuda")).reshape(-1)
        seq = torch.arange(self.batch, device="cuda").repeat_interleave(t)
        moved = self.append(tokens.reshape(-1), seq, at)
        lens = self.lens + t
        out = self.attend(tokens.reshape(-1), lens, self.qs, t)
        probs = self.grid(torch.softmax(out.float().reshape(len(at), -1) @ self.head, -1))
        accept = uniform[:, :self.k].contiguous().view(-1)
        sample = uniform[:, self.k].contiguous()
        new, kept, new_lens = self.pkv.pkv_verify_drafts(
            probs, draft_probs, tokens[:, 1:].reshape(-1).to(torch.int32), accept, sample, self.qs, self.ds, self.k,
            context_lens=lens)
        self.lens.copy_(new_lens)
        self.last.copy_(new.gather(1, kept.long()[:, None])[:, 0])
        return dict(moved=moved, q=self.eq[tokens.reshape(-1)], lens=lens, start=self.qs, out=out, probs=probs,
                    draft_probs=draft_probs, tokens=tokens, accept=accept, sample=sample, new=new, kept=kept,
                    new_lens=new_lens)

    @staticmethod
    def grid(p):
        return torch.round(p * 2.0 ** 30) / 2.0 ** 30

    def read_back(self):
        start = torch.zeros(self.batch + 1, dtype=torch.int32, device="cuda")
        start[1:] = self.lens.cumsum(0)
        return self.pkv.pkv_gather_q8(self.kc, self.vc, self.sc, self.tables, self.lens, start, int(start[-1]))


class Mirror:
    """The cache as the oracle has it."""

    def __init__(self, s):
        nb = s.kc.shape[0]
        self.s = s
        self.kc, self.vc = (np.zeros((nb, s.hkv, 16, s.d), np.int8) for _ in range(2))
        self.ks, self.vs = (np.zeros((nb, s.hkv, 16), np.float32) for _ in range(2))

    def check(self, r):
        s = self.s
        k, v, slots = r["moved"]
        wide = lambda x: OA.bf16_bits_to_f64(cases.host_view(x.cpu()))  # noqa: E731
        OQ.append_tokens_q8(self.kc, self.vc, self.ks, self.vs, wide(k), wide(v), slots.cpu().numpy())
        assert np.array_equal(s.kc.cpu().numpy(), self.kc)
        assert np.array_equal(s.vc.cpu().numpy().transpose(0, 1, 3, 2), self.vc)
        assert np.array_equal(s.sc.cpu().numpy(), np.stack([self.ks, self.vs], axis=2))
        c = dict(kc=self.kc, vc=self.vc, ks=self.ks, vs=self.vs, q=r["q"].cpu(), tables=s.tables.cpu().numpy(),
                 lens=r["lens"].cpu().numpy(), query_start=r["start"].cpu().numpy(), kv_heads=s.hkv,
                 scale=float(np.float32(s.d ** -0.5)))
        ref, tol = reference(c)
        got = r["out"].float().cpu().numpy().astype(np.float64)
        if s.d == 128 and np.diff(c["query_start"]).max() * s.hq // s.hkv <= 16:
            ma, rl = cases.attention_errors(r["out"], ref)
            assert ma <= 1e-2 and rl <= 2e-3
        else:
            assert (np.abs(got - ref) <= tol).all()

    def check_verified(self, r):
        s = self.s
        host = lambda x: None if x is None else x.cpu().numpy()  # noqa: E731
        out, kept, rejected = OV.verify_batch(host(r["probs"]), host(r["draft_probs"]), host(r["tokens"][:, 1:]).reshape(-1),
                                              host(r["accept"]), host(r["sample"]), host(s.qs), host(s.ds), s.k)
        assert np.array_equal(host(r["new"]), out) and np.array_equal(host(r["kept"]), kept)
        assert np.array_equal(host(r["new_lens"]), host(r["lens"]) - rejected)
        assert np.array_equal(host(s.lens), host(r["new_lens"]))
        return int(kept.sum()), int(rejected.sum())


SHAPES = [  # prompts, drafts, query heads, KV heads, head_dim, least table width
    ([38, 1, 131, 16, 2], 1, 8, 2, 128, 512),    # 8 rows per KV head, wide tables: the kernel that splits the cache
    ([38, 1, 131, 16, 2], 1, 8, 2, 128, 0),      # the same on tiles
    ([38, 1, 131, 16, 2], 9, 8, 2, 128, 0),      # 40 rows
    ([5, 200, 17], 3, 6, 2, 64, 0),
    ([300, 1], 0, 4, 4, 64, 0),                  # no drafts: each step samples one token
]


@pytest.mark.parametrize("prompts,drafts,hq,hkv,d,width", SHAPES)
def test_loop_against_the_oracle(pkv, prompts, drafts, hq, hkv, d, width):
    s = Server(pkv, prompts, drafts, hq, hkv, d, steps=6, least_width=width)
    m = Mirror(s)
    m.check(s.prefill())
    kept = rejected = 0
    for i in range(s.steps):
        r = s.step(s.uniform[i], s.choice[i])
        m.check(r)
        a, b = m.check_verified(r)
        kept, rejected = kept + a, rejected + b
    assert drafts == 0 or (kept > 0 and rejected > 0)        # both happen, or the loop shows nothing
    k, v = s.read_back()
    tables = s.tables.cpu().numpy()
    for got, codes, scales in ((k, m.kc, m.ks), (v, m.vc, m.vs)):
        rows = np.concatenate([(codes[b, :, t].astype(np.float32) * scales[b, :, t, None])[None]
                               for i, n in enumerate(s.lens.tolist()) for t0 in range(n)
                               for b, t in [(tables[i, t0 // 16], t0 % 16)]])
        assert torch.equal(got.cpu(), torch.from_numpy(rows).to(torch.bfloat16))
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("prompts,drafts,hq,hkv,d,width", SHAPES[:4])
def test_loop_as_a_graph(pkv, prompts, drafts, hq, hkv, d, width):
    eager = Server(pkv, prompts, drafts, hq, hkv, d, steps=6, least_width=width)
    eager.prefill()
    want = [eager.step(eager.uniform[i], eager.choice[i]) for i in range(eager.steps)]
    s = Server(pkv, prompts, drafts, hq, hkv, d, steps=6, least_width=width)
    s.prefill()
    uniform, choice = s.uniform[0].clone(), s.choice[0].clone()
    state = [x.clone() for x in (s.lens, s.last)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step(uniform, choice)                              # warms up what the capture may not create
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = s.step(uniform, choice)
    s.lens.copy_(state[0])
    s.last.copy_(state[1])
    for i in range(s.steps):
        uniform.copy_(s.uniform[i])
        choice.copy_(s.choice[i])
        graph.replay()
        for key in ("new", "kept", "new_lens", "out"):
            assert torch.equal(r[key], want[i][key]), (i, key)
    for a, b in ((s.kc, eager.kc), (s.vc, eager.vc), (s.sc, eager.sc)):
        assert torch.equal(a, b)
    assert pkv.pkv_device_status(clear=True) == 0
