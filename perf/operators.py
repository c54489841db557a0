"""Measured cases of the int8-cache serving operators.

Three operators of a serving step over a paged KV cache, each with its plain
form (elementary torch operations in 32 bits, rounded once at the end) and,
where ``own`` is true, the library call a serving loop makes:

* ``chunk``  -- causal attention of a chunk of new tokens per sequence over an
  int8 paged cache (``pkv_multiquery_attention_q8``): for query t of a sequence
  with n tokens, nq of them new, ``out = sum_p softmax_p(scale q.K_p) V_p`` over
  p <= n - nq + t, where K_p and V_p are code * scale.
* ``gather`` -- reading a token range of each sequence back out of the paged
  cache into packed rows (``pkv_gather``, ``pkv_gather_q8``).
* ``verify`` -- verification of drafted tokens against the target's
  probabilities from given uniform numbers (``pkv_verify_drafts``): draft j is
  kept while u_j q_j(x_j) < p_j(x_j); the token after the kept ones is drawn
  from max(p - q, 0) at the first rejected position, from p if none was, as the
  first index whose running sum exceeds u times the whole sum.
"""

import math
import random

import torch

own = False

BLOCK = 16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the first prompt chunk of one short request
        dict(name="chunk-short", op="chunk", batch=1, q_heads=32, kv_heads=8, head_dim=128, context=200, chunk=40,
             mix=0),
        # a few new tokens per sequence over ragged contexts: long drafts, or prompts that arrive in small pieces
        dict(name="chunk-few-ragged", op="chunk", batch=16, q_heads=32, kv_heads=8, head_dim=128, context=4097,
             chunk=24, mix=11),
        # ragged chunks, three query heads per KV head
        dict(name="chunk-ragged-g3", op="chunk", batch=7, q_heads=24, kv_heads=8, head_dim=128, context=6001,
             chunk=777, mix=5),
        # head size 64, eight query heads per KV head
        dict(name="chunk-d64", op="chunk", batch=4, q_heads=16, kv_heads=2, head_dim=64, context=3001, chunk=1000,
             mix=3),
        # the chunked-prefill workload of this repository, over an int8 cache
        dict(name="chunk-prefill512", op="chunk", batch=8, q_heads=32, kv_heads=8, head_dim=128, context=8192,
             chunk=512, mix=0),
        # the next chunk of one long document, 64 query heads
        dict(name="chunk-long", op="chunk", batch=1, q_heads=64, kv_heads=8, head_dim=128, context=65536, chunk=256,
             mix=0),
        # one short sequence read back
        dict(name="gather-q8-short", op="gather", form="q8", out="bf16", batch=1, kv_heads=8, head_dim=128,
             context=300, mix=0),
        # the suffixes of a ragged batch out of a bf16 cache
        dict(name="gather-bf16-ragged", op="gather", form="bf16", out="bf16", batch=64, kv_heads=8, head_dim=128,
             context=8191, mix=7),
        # the whole int8 cache of the 8K decode workload
        dict(name="gather-q8-8k", op="gather", form="q8", out="bf16", batch=32, kv_heads=8, head_dim=128,
             context=8192, mix=0),
        # one user, four drafts, a small vocabulary: latency
        dict(name="verify-one", op="verify", dtype="f32", batch=1, drafts=4, vocab=32000, accept=0.7, mix=0),
        # the 32-sequence, four-draft step of the verification workload
        dict(name="verify-32", op="verify", dtype="f32", batch=32, drafts=4, vocab=131072, accept=0.7, mix=0),
        # a large ragged batch, bf16 probabilities, an odd vocabulary (rows off the 16-byte grid)
        dict(name="verify-ragged-bf16", op="verify", dtype="bf16", batch=200, drafts=7, vocab=50001, accept=0.8,
             mix=9),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "gather", "verify"])
    mix = rng.choice([0, rng.randrange(1, 1000), rng.randrange(1, 1000)])
    if op == "chunk":
        while True:
            kv = rng.choice([1, 2, 4, 8])
            case = dict(op=op, batch=_log_uniform(rng, 1, 24), q_heads=kv * rng.choice([1, 2, 3, 4, 5, 8]),
                        kv_heads=kv, head_dim=rng.choice([64, 128, 128]), context=_log_uniform(rng, 1, 32768),
                        chunk=_log_uniform(rng, 1, 2048), mix=mix)
            case["chunk"] = min(case["chunk"], case["context"])
            # the plain form holds every (query, token) pair of the padded batch
            if case["batch"] * case["q_heads"] * case["chunk"] * case["context"] <= 8 * 32 * 512 * 8192:
                return case
    if op == "gather":
        form = rng.choice(["q8", "q8", "bf16", "f32"])
        out = form if form != "q8" else rng.choice(["bf16", "f32"])
        while True:
            case = dict(op=op, form=form, out=out, batch=_log_uniform(rng, 1, 300), kv_heads=rng.choice([1, 2, 4, 8]),
                        head_dim=rng.choice([64, 128]), context=_log_uniform(rng, 1, 16384), mix=mix)
            if case["batch"] * case["context"] * case["kv_heads"] <= 24 * 8192 * 8:
                return case
    while True:
        case = dict(op=op, dtype=rng.choice(["f32", "f32", "bf16"]), batch=_log_uniform(rng, 1, 256),
                    drafts=rng.randrange(1, 9), vocab=_log_uniform(rng, 100, 260000),
                    accept=rng.choice([0.5, 0.7, 0.9]), mix=mix)
        if case["batch"] * (case["drafts"] + 1) * case["vocab"] <= 32 * 5 * 131072:
            return case


def _lengths(case):
    """Per sequence: chunk -> (tokens, new tokens); gather -> (tokens, first token read); verify -> drafts."""
    rng = random.Random(case["mix"])
    found = []
    for i in range(case["batch"]):
        if case["op"] == "verify":
            found.append(case["drafts"] if case["mix"] == 0 or i == 0 else rng.randrange(0, case["drafts"] + 1))
            continue
        n = case["context"] if case["mix"] == 0 or i == 0 else _log_uniform(rng, max(1, case["context"] // 32),
                                                                            case["context"])
        if case["op"] == "chunk":
            most = min(case["chunk"], n)
            found.append((n, most if case["mix"] == 0 or i == 0 else rng.randrange(0, most + 1)))
        else:
            found.append((n, 0 if case["mix"] == 0 else rng.randrange(0, max(1, n // 2))))
    return found


# ------------------------------------------------------------------ inputs
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def _quantized(shape, g):
    """Standard-normal rows (last axis) as int8 codes and their float32 scales."""
    x = torch.randn(shape, generator=g, device="cuda")
    scale = x.abs().amax(-1) / 127
    return (x / scale[..., None]).round_().clamp_(-127, 127).to(torch.int8), scale


def _paged(lens, g):
    """Block tables of sequences of these lengths over a shuffled pool: (tables, blocks)."""
    need = [(n + BLOCK - 1) // BLOCK for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, b in enumerate(need):
        tables[i, :b] = order[at:at + b]
        at += b
    return tables, total


def _offsets(counts):
    sums = [0]
    for c in counts:
        sums.append(sums[-1] + c)
    return torch.tensor(sums, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = _lengths(case)
    if case["op"] == "verify":
        return _prepare_verify(case, lens, g)
    tables, blocks = _paged([n for n, _ in lens], g)
    kv, d = case["kv_heads"], case["head_dim"]
    state = dict(op=case["op"], tables=tables, lens=torch.tensor([n for n, _ in lens], dtype=torch.int32, device="cuda"))
    if case["op"] == "chunk" or case["form"] == "q8":
        state["k"], ks = _quantized((blocks, kv, BLOCK, d), g)
        vc, vs = _quantized((blocks, kv, BLOCK, d), g)
        state["v"] = vc.transpose(2, 3).contiguous()                    # a coordinate's 16 tokens together
        state["scales"] = torch.stack([ks, vs], 2).contiguous()
    else:
        dt = TORCH[case["form"]]
        state["k"] = torch.randn((blocks, kv, BLOCK, d), generator=g, device="cuda").to(dt)
        state["v"] = torch.randn((blocks, kv, BLOCK, d), generator=g, device="cuda").to(dt)
        state["scales"] = None
    if case["op"] == "chunk":
        state["start"] = _offsets([q for _, q in lens])
        state["rows"] = sum(q for _, q in lens)
        state["most"] = max(1, max(q for _, q in lens))
        state["q"] = torch.randn((state["rows"], case["q_heads"], d), generator=g, device="cuda").to(torch.bfloat16)
        state["scale"] = 1.0 / math.sqrt(d)
    else:
        state["start"] = _offsets([n - f for n, f in lens])
        state["rows"] = sum(n - f for n, f in lens)
        state["first"] = torch.tensor([f for _, f in lens], dtype=torch.int32, device="cuda")
        state["out"] = TORCH[case["out"]]
    return state


def _prepare_verify(case, drafts, g):
    """A draft distribution per draft, the target's as accept * draft + (1 - accept) * another one."""
    v, dt = case["vocab"], TORCH[case["dtype"]]
    nd, nt = sum(drafts), sum(drafts) + len(drafts)
    soft = lambda rows: torch.softmax(4 * torch.randn((rows, v), generator=g, device="cuda"), -1)  # noqa: E731
    q = soft(max(1, nd))
    p = soft(nt)
    dstart, tstart = _offsets(drafts), _offsets([k + 1 for k in drafts])
    rows = torch.tensor([t for i, k in enumerate(drafts) for t in range(sum(drafts[:i]) + i, sum(drafts[:i]) + i + k)],
                        dtype=torch.int64, device="cuda")
    if nd:
        p[rows] = (1 - case["accept"]) * p[rows] + case["accept"] * q
    u = torch.rand((max(1, nd),), generator=g, device="cuda", dtype=torch.float64)
    tokens = (q.double().cumsum(-1) <= u[:, None]).sum(-1).clamp_(max=v - 1).to(torch.int32)
    return dict(op="verify", p=p.to(dt), q=q.to(dt), tokens=tokens, dstart=dstart, tstart=tstart,
                accept=torch.rand((max(1, nd),), generator=g, device="cuda"),
                sample=torch.rand((len(drafts),), generator=g, device="cuda"),
                lens=torch.full((len(drafts),), 100, dtype=torch.int32, device="cuda") + (tstart[1:] - tstart[:-1]),
                most=max(1, max(drafts)))


# ------------------------------------------------------------------ one pass
def run(state):
    return {"chunk": _chunk, "gather": _gather, "verify": _verify}[state["op"]](state)


def _chunk(s):
    if own:
        from paged_kv_cache_209_gb300 import pkv
        if "workspace" not in s:                                        # a serving loop keeps one
            need = pkv.pkv_multiquery_q8_workspace_size(s["lens"].shape[0], s["q"].shape[1], s["tables"].shape[1],
                                                        s["most"], s["k"])
            s["workspace"] = torch.zeros(max(256, need), dtype=torch.uint8, device="cuda")
        return pkv.pkv_multiquery_attention_q8(s["q"], s["k"], s["v"], s["scales"], s["tables"], s["lens"], s["start"],
                                               s["scale"], s["most"], workspace=s["workspace"])
    batch, width = s["tables"].shape
    kv, d = s["k"].shape[1], s["k"].shape[3]
    rows, heads, _ = s["q"].shape
    group, most, n = heads // kv, s["most"], width * BLOCK
    at = s["tables"].clamp(min=0).long()
    k = s["k"][at].float() * s["scales"][at][:, :, :, 0, :, None]       # [batch][width][kv][16][d]
    v = s["v"][at].float() * s["scales"][at][:, :, :, 1, None, :]       # [batch][width][kv][d][16]
    k = k.permute(0, 2, 4, 1, 3).reshape(batch, kv, d, n)
    v = v.permute(0, 2, 1, 4, 3).reshape(batch, kv, n, d)
    first, new = s["start"][:-1].long(), (s["start"][1:] - s["start"][:-1]).long()
    t = torch.arange(most, device="cuda")
    q = s["q"][(first[:, None] + t).clamp(max=max(0, rows - 1))].float()  # [batch][most][heads][d]
    q = q.reshape(batch, most, kv, group, d).transpose(1, 2).reshape(batch, kv, most * group, d)
    logits = (torch.matmul(q, k) * s["scale"]).reshape(batch, kv, most, group, n)
    last = s["lens"].long()[:, None] - new[:, None] + t                 # the last token each query sees
    hidden = torch.arange(n, device="cuda") > last[:, :, None]
    logits = logits.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    weights = logits.sub_(logits.amax(-1, keepdim=True)).exp_()
    total = weights.sum(-1, keepdim=True)
    out = torch.matmul(weights.reshape(batch, kv, most * group, n), v).reshape(batch, kv, most, group, d) / total
    out = out.transpose(1, 2).reshape(batch, most, heads, d)
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(s["start"].long(), row, right=True) - 1
    return out[seq, row - first[seq]].to(torch.bfloat16)


def _gather(s):
    if own:
        from paged_kv_cache_209_gb300 import pkv
        if s["scales"] is None:
            return pkv.pkv_gather(s["k"], s["v"], s["tables"], s["lens"], s["start"], s["rows"], token_start=s["first"])
        return pkv.pkv_gather_q8(s["k"], s["v"], s["scales"], s["tables"], s["lens"], s["start"], s["rows"],
                                 token_start=s["first"], out_dtype=s["out"])
    row = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["start"].long(), row, right=True) - 1
    token = s["first"][seq].long() + row - s["start"][seq].long()
    block, slot = s["tables"][seq, token // BLOCK].long(), token % BLOCK
    if s["scales"] is None:
        return s["k"][block, :, slot], s["v"][block, :, slot]
    k = s["k"][block, :, slot].float() * s["scales"][block, :, 0, slot][..., None]
    v = s["v"][block, :, :, slot].float() * s["scales"][block, :, 1, slot][..., None]
    return k.to(s["out"]), v.to(s["out"])


def _verify(s):
    if own:
        from paged_kv_cache_209_gb300 import pkv
        return pkv.pkv_verify_drafts(s["p"], s["q"], s["tokens"], s["accept"], s["sample"], s["tstart"], s["dstart"],
                                     s["most"], context_lens=s["lens"])
    batch, most = s["sample"].shape[0], s["most"]
    d0, t0 = s["dstart"][:-1].long(), s["tstart"][:-1].long()
    k = s["dstart"][1:].long() - d0
    j = torch.arange(most, device="cuda")
    there = j < k[:, None]
    drow = (d0[:, None] + j).clamp(max=s["tokens"].shape[0] - 1)
    trow = (t0[:, None] + j).clamp(max=s["p"].shape[0] - 1)
    token = s["tokens"][drow].long()
    # products of two 24-bit numbers, compared exactly in 64 bits
    kept = (s["accept"][drow].double() * s["q"][drow, token].double() < s["p"][trow, token].double()) & there
    accepted = kept.long().cumprod(1).sum(1)
    p = s["p"][t0 + accepted].float()
    q = s["q"][(d0 + accepted).clamp(max=s["tokens"].shape[0] - 1)].float() * (accepted < k)[:, None]
    rest = (p - q).clamp(min=0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, p)
    running = rest.double().cumsum(-1)                                  # 64 bits: a draw may lie next to a border
    aim = s["sample"].double() * running[:, -1]
    pick = (running <= aim[:, None]).sum(-1)
    positive = (rest > 0) * torch.arange(rest.shape[1], device="cuda")
    pick = torch.minimum(pick, positive.amax(-1))
    place = torch.arange(most + 1, device="cuda")
    padded = torch.cat([token, token.new_full((batch, 1), -1)], 1)
    tokens = torch.where(place < accepted[:, None], padded, torch.where(place == accepted[:, None], pick[:, None], -1))
    return tokens.to(torch.int32), accepted.to(torch.int32), s["lens"] - (k - accepted).to(torch.int32)


# ------------------------------------------------------------------ cost and definition
def work(case):
    lens = _lengths(case)
    if case["op"] == "chunk":
        kv, d, h = case["kv_heads"], case["head_dim"], case["q_heads"]
        tokens, rows = sum(n for n, q in lens if q), sum(q for _, q in lens)
        pairs = sum(q * (n - q) + q * (q + 1) // 2 for n, q in lens)
        return {"bytes": tokens * kv * (2 * d + 8) + rows * h * d * 4, "flops": 4 * pairs * h * d}
    if case["op"] == "gather":
        rows, width = sum(n - f for n, f in lens), case["kv_heads"] * case["head_dim"]
        size = {"f32": 4, "bf16": 2}
        read = 2 * width + 8 * case["kv_heads"] if case["form"] == "q8" else 2 * width * size[case["form"]]
        return {"bytes": rows * (read + 2 * width * size[case["out"]]), "flops": 2 * rows * width}
    # one target row per sequence, and one draft row where a draft is rejected
    elem = 4 if case["dtype"] == "f32" else 2
    rows = sum(2 - case["accept"] ** k for k in lens)
    return {"bytes": int(rows * case["vocab"] * elem), "flops": int(2 * rows * case["vocab"])}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits, sequence by sequence."""
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s)
    lens = _lengths(case)
    parts = []
    for i, (n, other) in enumerate(lens):
        blocks = s["tables"][i, :(n + BLOCK - 1) // BLOCK].long()
        if s["scales"] is None:
            k, v = s["k"][blocks].double(), s["v"][blocks].double()
        else:
            rec = s["scales"][blocks].double()
            k = s["k"][blocks].double() * rec[:, :, 0].unsqueeze(-1)
            v = s["v"][blocks].double().transpose(2, 3) * rec[:, :, 1].unsqueeze(-1)
        heads, d = k.shape[1], k.shape[3]
        k = k.transpose(0, 1).reshape(heads, -1, d)[:, :n]
        v = v.transpose(0, 1).reshape(heads, -1, d)[:, :n]
        if case["op"] == "gather":
            parts.append((k[:, other:].transpose(0, 1), v[:, other:].transpose(0, 1)))
            continue
        if other == 0:
            continue
        base = int(s["start"][i])
        q = s["q"][base:base + other].double()
        group = q.shape[1] // heads
        seen = torch.arange(n, device="cuda")[None] <= torch.arange(n - other, n, device="cuda")[:, None]
        out = torch.empty_like(q)
        for h in range(q.shape[1]):
            x = s["scale"] * (q[:, h] @ k[h // group].T)
            x = torch.where(seen, x, torch.full_like(x, -math.inf))
            w = torch.exp(x - x.max(1, keepdim=True).values)
            out[:, h] = (w @ v[h // group]) / w.sum(1, keepdim=True)
        parts.append(out)
    if case["op"] == "chunk":
        return torch.cat(parts) if parts else s["q"].double()
    return torch.cat([k for k, _ in parts]), torch.cat([v for _, v in parts])


def _exact_verify(s):
    dstart, tstart = s["dstart"].tolist(), s["tstart"].tolist()
    tokens, accepted, lens = [], [], []
    for i in range(len(dstart) - 1):
        k, row = dstart[i + 1] - dstart[i], []
        for j in range(k):
            x = int(s["tokens"][dstart[i] + j])
            u = float(s["accept"][dstart[i] + j])
            if not u * float(s["q"][dstart[i] + j, x]) < float(s["p"][tstart[i] + j, x]):
                break
            row.append(x)
        a = len(row)
        mass = s["p"][tstart[i] + a].float()
        if a < k:
            less = mass - s["q"][dstart[i] + a].float()
            less = torch.where(less > 0, less, torch.zeros_like(less))
            mass = less if bool((less > 0).any()) else mass
        some = torch.nonzero(mass > 0).flatten()
        sums = torch.cumsum(mass[some].double(), 0)
        at = torch.searchsorted(sums, float(s["sample"][i]) * sums[-1:], right=True)
        row.append(int(some[at.clamp(max=some.numel() - 1)]))
        tokens.append(row + [-1] * (s["most"] + 1 - len(row)))
        accepted.append(a)
        lens.append(int(s["lens"][i]) - (k - a))
    whole = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return whole(tokens), whole(accepted), whole(lens)
