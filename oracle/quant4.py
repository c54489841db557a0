"""The 4-bit paged cache: quantization of a row, the packed record, the append,
reading back and attention. Test infrastructure: only tests and the smoke check use it.

Sources: Notebook 10, section 8 (fewer bits per coordinate) and its project demo's
``fake_quantize_rows`` (symmetric per row, ``limit = 2**(bits-1) - 1``, here 7).

Reading: the cache keeps a float32 scale, ``max|x|`` times ``float32(1/7)`` rounded to
float32 (0 for a zero row, whose codes are 0; NaN for a row that holds a NaN or an
infinity); the code is ``rint`` of the exact quotient
``x / scale``, clipped to +-7, so it is a function of the stored scale. A record (16 tokens
of one block and KV head) is laid out as include/pkv.h states it; this file packs and
unpacks it nibble by nibble from that statement.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

from .attention import softmax_attention

BLOCK = 16
LIMIT = 7
STEP = np.float32(1) / np.float32(7)


def record_bytes(d: int) -> int:
    return 16 * d + 128


def quantize_rows4(x):
    """Rows along the last axis -> (int8 codes -7..7, float32 scales)."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(axis=-1)
    x = np.where(bad[..., None], 0.0, x)
    scale = (np.max(np.abs(x), axis=-1).astype(np.float32) * STEP).astype(np.float32)
    wide = scale.astype(np.float64)[..., None]
    # float64 holds x and the scale exactly; their quotient lies on a border c + 1/2 or at least 2^-25 of
    # itself away from it (24-bit significands), farther than its rounding
    quotient = np.divide(x, wide, out=np.zeros_like(x), where=wide > 0)
    return np.clip(np.rint(quotient), -LIMIT, LIMIT).astype(np.int8), np.where(bad, np.float32(np.nan), scale)


def code_exactly(x: float, scale: float) -> int:
    """One code by rational arithmetic."""
    if scale == 0:
        return 0
    q = Fraction(float(x)) / Fraction(float(scale))
    return max(-LIMIT, min(LIMIT, round(q)))                # Python rounds half to even


def k_place(d: int, token: int, dim: int):
    """(byte, shift) of K's nibble in a record."""
    word, e = divmod(dim, 8)
    p = e // 2 + 4 * (e % 2)
    return token * (d // 2) + 4 * word + p // 2, 4 * (p % 2)


def v_place(d: int, token: int, dim: int):
    o, e = divmod(dim, 8)
    j, p0 = divmod(e, 2)
    quad, p2 = divmod(token % 8, 2)
    p = 4 * p2 + 2 * (token // 8) + p0
    return 8 * d + 64 * o + 16 * quad + 4 * j + p // 2, 4 * (p % 2)


def _places(d):
    k = np.array([[k_place(d, t, e) for e in range(d)] for t in range(BLOCK)])
    v = np.array([[v_place(d, t, e) for e in range(d)] for t in range(BLOCK)])
    return k, v                                             # [16][d][2]


def unpack(records, d: int):
    """uint8 [..., record] -> (k codes, v codes int8 [..., 16, d], k scales, v scales float32 [..., 16])."""
    records = np.ascontiguousarray(records)
    k, v = _places(d)
    codes = [((records[..., at[..., 0]] >> at[..., 1]) & 15).astype(np.int8) - np.int8(8) for at in (k, v)]
    scales = np.ascontiguousarray(records[..., 16 * d:]).view(np.float32)
    return codes[0], codes[1], scales[..., :BLOCK], scales[..., BLOCK:]


def pack(kc, vc, ks, vs):
    """The inverse of ``unpack``."""
    d = kc.shape[-1]
    out = np.zeros(kc.shape[:-2] + (record_bytes(d),), dtype=np.uint8)
    for codes, at in zip((kc, vc), _places(d)):
        for t in range(BLOCK):
            for e in range(d):
                out[..., at[t, e, 0]] |= ((codes[..., t, e].astype(np.int16) + 8) << at[t, e, 1]).astype(np.uint8)
    out[..., 16 * d:] = np.ascontiguousarray(np.concatenate([ks, vs], -1).astype(np.float32)).view(np.uint8)
    return out


def append_tokens_q4(cache, k_new, v_new, slots):
    """Append rows ``[tokens][kv_heads][d]`` into the uint8 cache ``[blocks][kv_heads][record]`` in place."""
    d = k_new.shape[-1]
    place = _places(d)
    for rows, at, first in ((k_new, place[0], 0), (v_new, place[1], BLOCK)):
        codes, scales = quantize_rows4(rows)
        for t, s in enumerate(np.asarray(slots).reshape(-1)):
            if s < 0:
                continue
            b, o = divmod(int(s), BLOCK)
            for h in range(cache.shape[1]):
                rec = cache[b, h]
                for e in range(d):
                    byte, shift = at[o, e]
                    rec[byte] = (rec[byte] & ~(15 << shift) & 255) | ((int(codes[t, h, e]) + 8) << shift)
                w = 16 * d + 4 * (first + o)
                rec[w:w + 4] = np.frombuffer(np.float32(scales[t, h]).tobytes(), np.uint8)


def values(cache, d: int):
    """K and V values in float64, ``[blocks][kv_heads][16][d]``."""
    kc, vc, ks, vs = unpack(cache, d)
    with np.errstate(invalid="ignore"):
        return kc * ks.astype(np.float64)[..., None], vc * vs.astype(np.float64)[..., None]


def attention_q4(q, cache, tables, lens, starts, scale):
    """Causal attention of each sequence's last tokens, float64. ``q`` [rows][q_heads][d]; ``starts`` None: one
    query per sequence (a sequence without tokens gives zeros). Absent blocks (ids out of range) carry no weight."""
    q = np.asarray(q, dtype=np.float64)
    rows, heads, d = q.shape
    nb, kv = cache.shape[:2]
    group = heads // kv
    out = np.zeros_like(q)
    for i, n in enumerate(int(x) for x in lens):
        q0, q1 = (i, i + 1) if starts is None else (int(starts[i]), int(starts[i + 1]))
        blocks = [int(b) for b in tables[i, :(n + BLOCK - 1) // BLOCK]]
        there = np.array([0 <= b < nb for b in blocks], dtype=bool).repeat(BLOCK)[:n]
        k, v = values(cache[[b if 0 <= b < nb else 0 for b in blocks]].reshape(-1, kv, cache.shape[2]), d)
        k = k.transpose(1, 0, 2, 3).reshape(kv, -1, d)[:, :n]
        v = v.transpose(1, 0, 2, 3).reshape(kv, -1, d)[:, :n]
        for r in range(q0, q1):
            seen = there & (np.arange(n) <= n - (q1 - r))
            if not seen.any():
                continue
            for h in range(kv):
                out[r, h * group:(h + 1) * group] = softmax_attention(q[r, h * group:(h + 1) * group], k[h, seen], v[h, seen],
                                                                      scale)
    return out
