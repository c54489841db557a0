"""Measured cases of a serving step over a 4-bit paged KV cache.

Four operators, each with its plain form (elementary torch operations in 32
bits, in 64 where a value lies next to a rounding border or an angle is far
out) and, where ``own`` is true, the library calls a serving loop makes:

* ``plan``   -- slots, positions, row offsets and block-table entries of a
  step's new tokens from the sequences' lengths and a stack of free blocks
  (``pkv_plan_step``).
* ``table``  -- cosines and sines of rotary positions (``pkv_rotary_table``).
* ``append`` -- rotary positions on q and k, k and v written into the paged
  cache (``pkv_append_rotary``). A 4-bit cache's rows are read back as the
  values they stand for (``pkv_gather_q4``).
* ``attend`` -- causal attention of each sequence's last tokens over the 4-bit
  paged cache (``pkv_decode_attention_q4``, ``pkv_multiquery_attention_q4``):
  ``out = sum_p softmax_p(scale q.K_p) V_p``, K_p and V_p being code * scale.

The 4-bit cache is one uint8 tensor [blocks][kv_heads][16 * head_dim + 128]: a
record holds the K codes of 16 tokens, their V codes, then 16 K scales and 16 V
scales in float32. A nibble is code + 8. K: a token's row is head_dim / 8 words
of 32 bits; nibble p of word w holds dimension 8 w + 2 (p % 4) + p // 4. V:
word (o, q, j) -- octet of dimensions, quad of tokens, pair of dimensions --
holds in nibble p dimension 8 o + 2 j + p % 2 of token 2 q + p // 4 + 8 (p // 2 % 2).
"""

import math
import random

import torch

own = False

BLOCK = 16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one short request: latency
        dict(name="attend-one", op="attend", batch=1, q_heads=32, kv_heads=8, head_dim=128, context=1000, chunk=1, mix=0),
        # one token each of a ragged batch, three query heads per KV head
        dict(name="attend-ragged-g3", op="attend", batch=64, q_heads=24, kv_heads=8, head_dim=128, context=8191, chunk=1,
             mix=7),
        # the 8K decode workload of this repository, over a 4-bit cache
        dict(name="attend-8k", op="attend", batch=32, q_heads=32, kv_heads=8, head_dim=128, context=8192, chunk=1, mix=0),
        # the four-draft verification workload of this repository, over a 4-bit cache
        dict(name="attend-drafts", op="attend", batch=32, q_heads=32, kv_heads=8, head_dim=128, context=8192, chunk=4,
             mix=0),
        # the chunked-prefill workload of this repository, over a 4-bit cache
        dict(name="attend-prefill512", op="attend", batch=8, q_heads=32, kv_heads=8, head_dim=128, context=8192,
             chunk=512, mix=0),
        # the new tokens of a 32-sequence decode step
        dict(name="append-step", op="append", cache="q4", batch=32, q_heads=32, kv_heads=8, head_dim=128, rotary=128,
             interleaved=False, context=8192, chunk=1, mix=0),
        # the new tokens of the chunked-prefill step
        dict(name="append-prefill512", op="append", cache="q4", batch=8, q_heads=32, kv_heads=8, head_dim=128, rotary=128,
             interleaved=False, context=8192, chunk=512, mix=0),
        # ragged prompts into a bf16 cache, neighbouring pairs in half of the head
        dict(name="append-bf16-partial", op="append", cache="bf16", batch=9, q_heads=24, kv_heads=8, head_dim=128,
             rotary=64, interleaved=True, context=4001, chunk=1777, mix=5),
        # a model's usual context
        dict(name="table-4k", op="table", positions=4096, rotary=64, base=10000.0, factor=1.0),
        # a long context, frequencies stretched eight times, magnitude factor
        dict(name="table-128k", op="table", positions=131072, rotary=128, base=500000.0, factor=1.2079, stretch=8.0),
        # a 32-sequence decode step
        dict(name="plan-step", op="plan", batch=32, context=8192, chunk=1, mix=0),
        # a thousand ragged sequences, prompts among decoding ones
        dict(name="plan-ragged", op="plan", batch=1000, context=4096, chunk=1024, mix=3),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "table", "plan"])
    mix = rng.choice([0, rng.randrange(1, 1000), rng.randrange(1, 1000)])
    if op == "attend":
        while True:
            kv = rng.choice([1, 2, 4, 8])
            case = dict(op=op, batch=_log_uniform(rng, 1, 100), q_heads=kv * rng.choice([1, 2, 3, 4, 5, 8]), kv_heads=kv,
                        head_dim=rng.choice([64, 128, 128]), context=_log_uniform(rng, 1, 32768),
                        chunk=rng.choice([1, 1, rng.randrange(2, 9), _log_uniform(rng, 9, 2048)]), mix=mix)
            case["chunk"] = min(case["chunk"], case["context"])
            # the plain form holds every (query, token) pair of the padded batch, and the cache in 32 bits
            if case["batch"] * case["q_heads"] * case["chunk"] * case["context"] <= 8 * 32 * 512 * 8192 and \
                    case["batch"] * kv * case["context"] <= 32 * 8 * 8192:
                return case
    if op == "append":
        while True:
            kv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128])
            case = dict(op=op, cache=rng.choice(["q4", "q4", "bf16"]), batch=_log_uniform(rng, 1, 200),
                        q_heads=kv * rng.choice([1, 2, 3, 4, 8]), kv_heads=kv, head_dim=d,
                        rotary=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.5,
                        context=_log_uniform(rng, 1, 16384), chunk=_log_uniform(rng, 1, 2048), mix=mix)
            case["chunk"] = min(case["chunk"], case["context"])
            if case["batch"] * case["chunk"] * (case["q_heads"] + 2 * kv) * d <= 8 * 512 * 48 * 128 and \
                    case["batch"] * case["context"] * kv <= 32 * 8 * 8192:
                return case
    if op == "table":
        return dict(op=op, positions=_log_uniform(rng, 1, 131072), rotary=2 * rng.randrange(8, 65),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), factor=rng.choice([1.0, 1.0, 1.1386]),
                    stretch=rng.choice([1.0, 4.0, 8.0]))
    while True:
        case = dict(op=op, batch=_log_uniform(rng, 1, 4000), context=_log_uniform(rng, 1, 16384),
                    chunk=_log_uniform(rng, 1, 2048), mix=mix)
        case["chunk"] = min(case["chunk"], case["context"])
        if case["batch"] * case["chunk"] <= 500000:
            return case


def _lengths(case):
    """Per sequence (tokens after the step, new tokens)."""
    rng = random.Random(case["mix"])
    found = []
    for i in range(case["batch"]):
        if case["mix"] == 0 or i == 0:
            found.append((case["context"], min(case["chunk"], case["context"])))
            continue
        n = _log_uniform(rng, max(1, case["context"] // 32), case["context"])
        most = min(case["chunk"], n)
        if case["op"] == "plan":                                        # most sequences decode, a few are prompts
            found.append((n, rng.randrange(0, most + 1) if rng.random() < 0.25 else rng.randrange(0, 2) if n else 0))
        elif case["chunk"] == 1:
            found.append((n, 1))
        else:
            found.append((n, rng.randrange(0, most + 1)))
    return found


# ------------------------------------------------------------------ inputs
def _paged(lens, g):
    """Block tables of sequences of these lengths over a shuffled pool: (tables, blocks)."""
    need = [(n + BLOCK - 1) // BLOCK for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(need))
    at = torch.tensor(need, device="cuda").cumsum(0) - torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")
    there = col < torch.tensor(need, device="cuda")[:, None]
    tables = torch.where(there, order[(at[:, None] + col).clamp(max=total - 1)], -1)
    return tables.to(torch.int32), total


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _offsets(counts):
    sums = [0]
    for c in counts:
        sums.append(sums[-1] + c)
    return _ints(sums)


def _rows_of(start, count):
    """(sequence, index within it) of each of `count` rows."""
    row = torch.arange(count, device="cuda")
    seq = torch.searchsorted(start.long(), row, right=True) - 1
    return seq, row - start[seq].long()


def _frequencies(case):
    """Angles per position, 64 bits; with `stretch`, slow turns are slowed down (those slower than a quarter of the
    usual context whole, faster ones than all of it not at all)."""
    half = case["rotary"] // 2
    found = [case["base"] ** (-2.0 * i / case["rotary"]) for i in range(half)]
    by = case.get("stretch", 1.0)
    if by != 1.0:
        turns = [8192 * f / (2 * math.pi) for f in found]
        part = [min(1.0, max(0.0, (t - 1.0) / (4.0 - 1.0))) for t in turns]
        found = [f * (p + (1.0 - p) / by) for f, p in zip(found, part)]
    return found


def _quantize(x):
    """Rows (last axis) as 4-bit codes (float32 whole numbers) and float32 scales, decided in 64 bits."""
    scale = x.abs().amax(-1) / 7
    codes = torch.round(x.double() / torch.where(scale > 0, scale, 1.0).double()[..., None]).clamp_(-7, 7)
    return codes.float(), scale


def _pack(kc, ks, vc, vs):
    """Records from codes [..., 16, head_dim] and scales [..., 16]."""
    lead, d = kc.shape[:-2], kc.shape[-1]
    two = lambda n: (n[..., 0::2] + 16 * n[..., 1::2]).to(torch.uint8)  # noqa: E731
    k = (kc + 8).reshape(*lead, BLOCK, d // 8, 4, 2).transpose(-1, -2).reshape(*lead, BLOCK, d // 8, 8)
    v = (vc + 8).reshape(*lead, 2, 4, 2, d // 8, 4, 2)                   # token: eight, quad, one; dimension: octet, pair, one
    n = len(lead)
    v = v.permute(*range(n), n + 3, n + 1, n + 4, n + 2, n, n + 5).reshape(*lead, d // 8, 4, 4, 8)
    parts = [two(k).reshape(*lead, 8 * d), two(v).reshape(*lead, 8 * d),
             torch.stack([ks, vs], -2).reshape(*lead, 32).contiguous().view(torch.uint8)]
    return torch.cat(parts, -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"attend": _prepare_attend, "append": _prepare_append, "table": _prepare_table,
            "plan": _prepare_plan}[case["op"]](case, g)


def _prepare_attend(case, g):
    lens = _lengths(case)
    tables, blocks = _paged([n for n, _ in lens], g)
    kv, d, rows = case["kv_heads"], case["head_dim"], sum(q for _, q in lens)
    parts = []
    for at in range(0, blocks, 4096):
        shape = (min(4096, blocks - at), kv, BLOCK, d)
        kc, ks = _quantize(torch.randn(shape, generator=g, device="cuda"))
        vc, vs = _quantize(torch.randn(shape, generator=g, device="cuda"))
        parts.append(_pack(kc, ks, vc, vs))
    return dict(op="attend", cache=torch.cat(parts), tables=tables, lens=_ints([n for n, _ in lens]),
                start=_offsets([q for _, q in lens]), most=max(1, max(q for _, q in lens)), decode=case["chunk"] == 1,
                q=torch.randn((rows, case["q_heads"], d), generator=g, device="cuda").to(torch.bfloat16),
                scale=1.0 / math.sqrt(d))


def _prepare_append(case, g):
    lens = _lengths(case)
    tables, blocks = _paged([n for n, _ in lens], g)
    hq, kv, d, rows = case["q_heads"], case["kv_heads"], case["head_dim"], sum(q for _, q in lens)
    start, longest = _offsets([q for _, q in lens]), max(n for n, _ in lens)
    seq, t = _rows_of(start, rows)
    first = _ints([n - q for n, q in lens])
    position = first[seq].long() + t
    slots = tables[seq, position // BLOCK].long() * BLOCK + position % BLOCK
    # q, k and v as one product leaves them; a chunk without new tokens leaves none
    qkv = torch.randn((rows, (hq + 2 * kv) * d), generator=g, device="cuda").to(torch.bfloat16)
    angle = torch.arange(longest, device="cuda", dtype=torch.float64)[:, None] * \
        torch.tensor(_frequencies(dict(case, base=10000.0)), dtype=torch.float64, device="cuda")
    if case["cache"] == "q4":
        pools = torch.zeros((blocks, kv, 16 * d + 128), dtype=torch.uint8, device="cuda"), None
    else:
        pools = tuple(torch.zeros((blocks, kv, BLOCK, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    return dict(op="append", q=qkv[:, :hq * d].view(rows, hq, d), k=qkv[:, hq * d:(hq + kv) * d].view(rows, kv, d),
                v=qkv[:, (hq + kv) * d:].view(rows, kv, d), interleaved=case["interleaved"], slots=slots,
                positions=position.to(torch.int32), table=torch.cat([angle.cos(), angle.sin()], 1).float(), pools=pools,
                tables=tables, lens=_ints([n for n, _ in lens]), start=start, first=first, rows=rows)


def _prepare_table(case, g):
    # the same frequencies drift with the seed, as those of another model
    drift = 1.0 + 1e-3 * float(torch.rand((), generator=g, device="cuda"))
    return dict(op="table", frequencies=torch.tensor([f * drift for f in _frequencies(case)], dtype=torch.float64, device="cuda"),
                positions=case["positions"], factor=case["factor"])


def _prepare_plan(case, g):
    lens = _lengths(case)
    old = [n - q for n, q in lens]
    held = [(n + BLOCK - 1) // BLOCK for n in old]                      # blocks of the tokens that are there
    width = max(1, max((n + BLOCK - 1) // BLOCK for n, _ in lens))
    total = sum((n + BLOCK - 1) // BLOCK for n, _ in lens) + 17
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    need, col = _ints(held, torch.int64), torch.arange(width, device="cuda")
    at = need.cumsum(0) - need
    tables = torch.where(col < need[:, None], order[(at[:, None] + col).clamp(max=total - 1)], -1).to(torch.int32)
    return dict(op="plan", lens=_ints(old), new=_ints([q for _, q in lens]), held=_ints(held), tables=tables.contiguous(),
                free=order[sum(held):].contiguous(), left=_ints([total - sum(held)]), rows=sum(q for _, q in lens))


# ------------------------------------------------------------------ one pass
def run(state):
    return {"attend": _attend, "append": _append, "table": _table, "plan": _plan}[state["op"]](state)


def _unpack(rec, d):
    """K and V values of records, float32 [..., 16, head_dim]."""
    lead = rec.shape[:-1]
    nibbles = lambda b: torch.stack([b & 15, b >> 4], -1).float() - 8  # noqa: E731
    k = nibbles(rec[..., :8 * d]).reshape(*lead, BLOCK, d // 8, 2, 4).transpose(-1, -2).reshape(*lead, BLOCK, d)
    v = nibbles(rec[..., 8 * d:16 * d]).reshape(*lead, d // 8, 4, 4, 2, 2, 2)
    n = len(lead)
    v = v.permute(*range(n), n + 4, n + 1, n + 3, n, n + 2, n + 5).reshape(*lead, BLOCK, d)
    scales = rec[..., 16 * d:].contiguous().view(torch.float32).reshape(*lead, 2, BLOCK, 1)
    return k * scales[..., 0, :, :], v * scales[..., 1, :, :]


def _attend(s):
    if own:
        from paged_kv_cache_209_gb300 import pkv
        if "workspace" not in s:                                        # a serving loop keeps one
            need = pkv.pkv_multiquery_q4_workspace_size(s["lens"].shape[0], s["q"].shape[1], s["tables"].shape[1],
                                                        s["most"], s["cache"])
            s["workspace"] = torch.zeros(max(256, need), dtype=torch.uint8, device="cuda")
        if s["decode"]:
            return pkv.pkv_decode_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["scale"],
                                               workspace=s["workspace"])
        return pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["start"], s["scale"],
                                               s["most"], workspace=s["workspace"])
    batch, width = s["tables"].shape
    rows, heads, d = s["q"].shape
    kv, most, n = s["cache"].shape[1], s["most"], width * BLOCK
    group = heads // kv
    k, v = _unpack(s["cache"][s["tables"].clamp(min=0).long()], d)      # [batch][width][kv][16][d]
    k = k.permute(0, 2, 4, 1, 3).reshape(batch, kv, d, n)
    v = v.permute(0, 2, 1, 3, 4).reshape(batch, kv, n, d)
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
    seq, at = _rows_of(s["start"], rows)
    return out[seq, at].to(torch.bfloat16)


def _turn(x, cos, sin, interleaved):
    """Rows x [T][heads][d] turned by [T][R / 2] cosines and sines."""
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _append(s):
    if own:
        from paged_kv_cache_209_gb300 import pkv
        q = pkv.pkv_append_rotary(s["q"], s["k"], s["v"], s["positions"], s["table"], s["slots"], *s["pools"],
                                  interleaved=s["interleaved"])
        if s["pools"][1] is not None:
            return q, *s["pools"]
        return q, *pkv.pkv_gather_q4(s["pools"][0], s["tables"], s["lens"], s["start"], s["rows"], token_start=s["first"],
                                     out_dtype=torch.float32)
    row = s["table"][s["positions"].long()]
    cos, sin = row[:, :row.shape[1] // 2], row[:, row.shape[1] // 2:]
    q = _turn(s["q"].float(), cos, sin, s["interleaved"]).to(torch.bfloat16)
    k = _turn(s["k"].double(), cos.double(), sin.double(), s["interleaved"]).float().to(torch.bfloat16)
    if s["pools"][1] is not None:
        block, slot = s["slots"] // BLOCK, s["slots"] % BLOCK
        s["pools"][0][block, :, slot] = k
        s["pools"][1][block, :, slot] = s["v"]
        return q, *s["pools"]
    kc, ks = _quantize(k.float())                                       # 64 bits: a quotient may lie next to a border
    vc, vs = _quantize(s["v"].float())
    return q, kc * ks[..., None], vc * vs[..., None]


def _table(s):
    if own:
        from paged_kv_cache_209_gb300 import pkv
        return pkv.pkv_rotary_table(s["frequencies"], s["positions"], factor=s["factor"])
    angle = torch.arange(s["positions"], device="cuda", dtype=torch.float64)[:, None] * s["frequencies"]
    return torch.cat([angle.cos(), angle.sin()], 1).mul_(s["factor"]).float()


def _plan(s):
    if own:
        from paged_kv_cache_209_gb300 import pkv
        return pkv.pkv_plan_step(s["lens"], s["new"], s["held"], s["free"], s["left"], s["tables"], s["rows"])[:-1] + \
            (s["tables"],)
    after = s["lens"] + s["new"]
    more = (torch.div(after + BLOCK - 1, BLOCK, rounding_mode="floor") - s["held"]).clamp(min=0)
    start = torch.cat([torch.zeros_like(after[:1]), s["new"].cumsum(0).to(torch.int32)])
    before = more.cumsum(0) - more                                      # blocks taken by the sequences before
    tables, batch, width = s["tables"], s["tables"].shape[0], s["tables"].shape[1]
    at = torch.arange(width, device="cuda") - s["held"][:, None]        # which of its new blocks an entry is
    taken = (at >= 0) & (at < more[:, None])
    stack = (s["left"].long() - 1 - before[:, None] - at).clamp(min=0, max=s["free"].shape[0] - 1)
    tables.copy_(torch.where(taken, s["free"][stack], tables))
    seq, t = _rows_of(start, s["rows"])
    position = s["lens"][seq].long() + t
    slots = tables[seq, position // BLOCK].long() * BLOCK + position % BLOCK
    return (slots, position.to(torch.int32), start, after, s["held"] + more.to(torch.int32),
            s["left"] - more.sum().to(torch.int32), tables)


# ------------------------------------------------------------------ cost and definition
def work(case):
    if case["op"] == "table":
        values = case["positions"] * case["rotary"]
        return {"bytes": values * 4 + case["rotary"] * 4, "flops": 2 * values}
    lens = _lengths(case)
    rows = sum(q for _, q in lens)
    if case["op"] == "plan":
        batch = case["batch"]
        more = sum((n + BLOCK - 1) // BLOCK - (n - q + BLOCK - 1) // BLOCK for n, q in lens)
        # lengths, new tokens and held blocks in, the first and last and the row offsets out; a stack entry and a
        # table entry per new block, a slot and a position per row
        return {"bytes": 24 * batch + 8 * more + 12 * rows, "flops": 4 * batch + 4 * rows}
    hq, kv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "attend":
        tokens = sum(n for n, q in lens if q)
        pairs = sum(q * (n - q) + q * (q + 1) // 2 for n, q in lens)
        return {"bytes": tokens * kv * (d + 8) + rows * hq * d * 4, "flops": 4 * pairs * hq * d}
    table = len({p for n, q in lens for p in range(n - q, n)}) * case["rotary"] * 4
    bytes_ = rows * (hq * d * 4 + 2 * kv * d * 2 + 12) + table
    if case["cache"] == "q4":
        bytes_ += rows * kv * (d + 8 + 2 * d * 4)                       # codes and scales, then the values
    else:
        bytes_ += rows * 2 * kv * d * 2
    return {"bytes": bytes_, "flops": rows * (hq + kv) * case["rotary"] * 3}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    if case["op"] == "plan":
        return None                                                     # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "table":
        p = torch.arange(s["positions"], dtype=torch.float64, device="cuda")
        columns = [torch.cos(p * f) for f in s["frequencies"]] + [torch.sin(p * f) for f in s["frequencies"]]
        return torch.stack(columns, 1) * s["factor"]
    return _exact_attend(case, s) if case["op"] == "attend" else _exact_append(case, s)


def _exact_codes(rec, d):
    """K and V values of records [blocks][record] in 64 bits, a dimension and a token at a time: [blocks][16][d]."""
    b = rec.long()
    scales = rec[:, 16 * d:].contiguous().view(torch.float32).double()
    code = lambda at, p: ((b[:, at + p // 2] >> (4 * (p % 2))) & 15).double() - 8  # noqa: E731  (nibble p of a word)
    k, v = (torch.empty((b.shape[0], BLOCK, d), dtype=torch.float64, device="cuda") for _ in range(2))
    token = torch.arange(BLOCK, device="cuda")
    for e in range(d):
        k[:, :, e] = code(token * (d // 2) + e // 8 * 4, e % 8 // 2 + 4 * (e % 2))
        for t in range(BLOCK):
            v[:, t, e] = code(8 * d + e // 8 * 64 + t % 8 // 2 * 16 + e % 8 // 2 * 4, 4 * (t % 2) + 2 * (t // 8) + e % 2)
    return k * scales[:, :BLOCK, None], v * scales[:, BLOCK:, None]


def _exact_attend(case, s):
    d, heads = case["head_dim"], case["kv_heads"]
    group, out = case["q_heads"] // heads, torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    if sum(n for n, _ in _lengths(case)) * heads * d > 32 * 8 * 8192 * 128:
        return None
    for h in range(heads):
        keys, values = _exact_codes(s["cache"][:, h], d)
        for i, (n, new) in enumerate(_lengths(case)):
            blocks = s["tables"][i, :(n + BLOCK - 1) // BLOCK].long()
            k, v = keys[blocks].reshape(-1, d)[:n], values[blocks].reshape(-1, d)[:n]
            base = int(s["start"][i])
            q = s["q"][base:base + new, h * group:(h + 1) * group].double()
            seen = torch.arange(n, device="cuda") <= torch.arange(n - new, n, device="cuda")[:, None]
            x = torch.where(seen[:, None], s["scale"] * (q @ k.T), torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
            if new:
                w = torch.exp(x - x.max(-1, keepdim=True).values)
                out[base:base + new, h * group:(h + 1) * group] = (w @ v) / w.sum(-1, keepdim=True)
    return out


def _exact_append(case, s):
    half = case["rotary"] // 2
    angle = s["table"].double()[s["positions"].long()]
    turned = []
    for x in (s["q"].double(), s["k"].double()):
        y = x.clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            c, w = angle[:, i, None], angle[:, half + i, None]
            y[..., a] = x[..., a] * c - x[..., b] * w
            y[..., b] = x[..., b] * c + x[..., a] * w
        turned.append(y)
    q, k = turned
    k = k.float().to(torch.bfloat16)                                    # the cache takes rows of this type
    if case["cache"] != "q4":
        at = s["slots"]
        for pool, x in zip(s["pools"], (k, s["v"])):
            pool[at // BLOCK, :, at % BLOCK] = x
        return q, s["pools"][0].double(), s["pools"][1].double()
    found = []
    for x in (k, s["v"]):
        top = x.float().abs().amax(-1, keepdim=True)
        step = (top / 7).double()
        n = torch.round(x.double() / torch.where(step > 0, step, torch.ones_like(step)))
        found.append(torch.minimum(torch.maximum(n, torch.full_like(n, -7)), torch.full_like(n, 7)) * step)
    return q, found[0], found[1]
