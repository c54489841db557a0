"""Inputs and bounds shared by the GPU tests of the 4-bit cache."""

from __future__ import annotations

import math

import numpy as np
import torch

from oracle import quant4 as Q

B = 16


def make(seed, lens, news, q_heads, kv_heads, d, spread=1.0, k_sizes=None, v_sizes=None, width=None, garbage=True):
    """A cache of sequences of these lengths on a shuffled pool, and their queries, on the device. Slots past a
    sequence's end hold arbitrary bytes (scales NaN and infinite among them)."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    need = [-(-n // B) for n in lens]
    blocks = sum(need) + 3
    order = rng.permutation(blocks)
    tables = np.full((len(lens), width or max(1, max(need, default=1))), -1, np.int32)
    at = 0
    for i, k in enumerate(need):
        tables[i, :k] = order[at:at + k]
        at += k
    kv = torch.randn((2, blocks, kv_heads, B, d), generator=g).numpy().astype(np.float32)
    for side, sizes in ((0, k_sizes), (1, v_sizes)):
        if sizes is not None:
            kv[side] *= sizes(rng, (blocks, kv_heads, B, 1)).astype(np.float32)
    kc, ks = Q.quantize_rows4(kv[0])
    vc, vs = Q.quantize_rows4(kv[1])
    cache = fast_pack(kc, vc, ks, vs)
    if garbage:
        used = np.zeros((blocks, B), bool)
        for i, n in enumerate(lens):
            for t in range(n):
                used[tables[i, t // B], t % B] = True
        waste = rng.integers(0, 256, cache.shape, dtype=np.uint8)
        scales = waste[..., 16 * d:].view(np.float32)
        scales[...] = rng.choice(np.array([np.nan, np.inf, -np.inf, 1e30, 0.0], np.float32), scales.shape)
        kcw, vcw, ksw, vsw = Q.unpack(waste, d)
        keep = used[:, None, :]
        kc, vc = (np.where(keep[..., None], a, b) for a, b in ((kc, kcw), (vc, vcw)))
        ks, vs = (np.where(keep, a, b) for a, b in ((ks, ksw), (vs, vsw)))
        cache = fast_pack(kc, vc, ks, vs)
    rows = sum(news)
    q = (torch.randn((rows, q_heads, d), generator=g) * spread).to(torch.bfloat16)
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    return dict(cache=dev(cache), tables=dev(tables), lens=dev(np.array(lens, np.int32)), start=dev(start), q=q.cuda(),
                scale=1.0 / math.sqrt(d), lens_list=list(lens), news=list(news), d=d)


def fast_pack(kc, vc, ks, vs):
    """Q.pack without its loops over tokens and dimensions (checked against it)."""
    lead, d = kc.shape[:-2], kc.shape[-1]
    n = len(lead)
    two = lambda x: (x[..., 0::2] | (x[..., 1::2] << 4)).astype(np.uint8)  # noqa: E731
    k = (kc + 8).astype(np.uint8).reshape(*lead, B, d // 8, 4, 2).swapaxes(-1, -2).reshape(*lead, B, d // 8, 8)
    v = (vc + 8).astype(np.uint8).reshape(*lead, 2, 4, 2, d // 8, 4, 2)
    v = v.transpose(*range(n), n + 3, n + 1, n + 4, n + 2, n, n + 5).reshape(*lead, d // 8, 4, 4, 8)
    scales = np.ascontiguousarray(np.concatenate([ks, vs], -1).astype(np.float32)).view(np.uint8)
    return np.concatenate([two(k).reshape(*lead, 8 * d), two(v).reshape(*lead, 8 * d), scales], -1)


def values64(s):
    """K and V values in float64 on the device, [blocks][kv_heads][16][d]."""
    k, v = Q.values(s["cache"].cpu().numpy(), s["d"])
    return torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()


def reference(s, decode=False):
    """(out, bound) in float64: attention from the definition, and how far a bf16 result may be from it.

    Errors of one output: its rounding to bf16, |out| 2^-8. The weights' and values' roundings to f16 or finer,
    at most three of 2^-11 each, on sum_p w_p |v_p| (w normalised). The K values' rounding, 2^-11 of each: a
    score is off by at most delta = |scale| 2^-11 max_p sum_d |q_d k_pd|, which moves the weights by factors
    within e^+-delta each, numerator and denominator: 2 delta sum_p w_p |v_p|, taken twice for delta's second order.
    fp32 sums: less than one more 2^-11 for the lengths here.
    """
    k, v = values64(s)
    q = s["q"].double()
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    kv, d = k.shape[1], s["d"]
    group = q.shape[1] // kv
    row = 0
    for i, n in enumerate(s["lens_list"]):
        new = 1 if decode else s["news"][i]
        blocks = s["tables"][i, :-(-n // B)].long()
        kk = k[blocks].transpose(0, 1).reshape(kv, -1, d)[:, :n]
        vv = v[blocks].transpose(0, 1).reshape(kv, -1, d)[:, :n]
        for h in range(kv):
            if n == 0 or new == 0:
                continue
            x = q[row:row + new, h * group:(h + 1) * group]
            seen = torch.arange(n, device="cuda") <= torch.arange(n - new, n, device="cuda")[:, None]
            z = (s["scale"] * (x @ kk[h].T)).masked_fill(~seen[:, None], -math.inf)
            w = torch.softmax(z, -1)
            o = w @ vv[h]
            mass = w @ vv[h].abs()
            delta = abs(s["scale"]) * 2.0 ** -11 * (x.abs() @ kk[h].abs().T).masked_fill(~seen[:, None], 0).amax(-1, keepdim=True)
            out[row:row + new, h * group:(h + 1) * group] = o
            bound[row:row + new, h * group:(h + 1) * group] = o.abs() * 2.0 ** -8 + mass * (4 * 2.0 ** -11 + 4 * delta)
        row += new
    return out, bound


def check(got, want, bound, mean=True):
    """Every output within its bound, and the whole within what the bf16 rounding alone gives at most in the mean
    (2^-8 / sqrt(3), the error being spread evenly over half a step) and a tenth."""
    got = got.double()
    assert torch.isfinite(got).all()
    worst = ((got - want).abs() - bound).max() if got.numel() else torch.tensor(0.0)
    assert worst <= 0, f"off by {float(worst)} more than the bound"
    norm = want.norm()
    if mean and norm > 0:
        assert (got - want).norm() / norm <= 1.1 * 2.0 ** -8 / math.sqrt(3)
