"""Verification of drafted tokens in float64, sequence by sequence. Test
infrastructure: only tests and the smoke check use it.

Source: release page "NeuralOps v1.3.4", Architectural Breakdown 2
(speculative decoding pipeline): the target scores the K draft tokens in one
pass and rejection sampling keeps its output distribution.

Reading: draft j of a sequence (token x, acceptance number u) is kept while
``u * q_j[x] < p_j[x]``; after the first rejection the next token is drawn from
``max(p - q, 0)`` at that position, after no rejection from the target's last
row, as the lowest index whose running sum exceeds ``w`` times the whole sum.
Entries are float32 (or bf16) numbers; their difference is rounded to float32;
products and sums are float64. An entry that is not a finite number above zero
has no mass.
"""

from __future__ import annotations

import numpy as np


def masses(row: np.ndarray) -> np.ndarray:
    """float64 mass of every entry of a float32 row."""
    row = np.asarray(row, dtype=np.float32)
    with np.errstate(invalid="ignore"):
        return np.where((row > 0) & np.isfinite(row), row, np.float32(0)).astype(np.float64)


def draw(mass: np.ndarray, w: float) -> int:
    """Lowest index whose running sum exceeds w * sum(mass); -1 without mass."""
    some = np.flatnonzero(mass > 0)
    if len(some) == 0:
        return -1
    running = np.cumsum(mass[some])
    above = np.flatnonzero(running > w * running[-1])
    return int(some[above[0]] if len(above) else some[-1])


def verify_sequence(p_rows, q_rows, tokens, accept, w):
    """``p_rows`` [k+1][vocab] float32, ``q_rows`` [k][vocab] or None (certain
    drafts), k tokens and acceptance numbers. Returns (kept + [next], kept count)."""
    p_rows = np.asarray(p_rows, dtype=np.float32)
    k, vocab = len(tokens), p_rows.shape[1]
    kept = []
    for j in range(k):
        x = int(tokens[j])
        inside = 0 <= x < vocab
        q = 1.0 if q_rows is None else (float(q_rows[j][x]) if inside else 0.0)
        if not (inside and float(accept[j]) * q < float(p_rows[j][x])):
            break
        kept.append(x)
    a = len(kept)
    if a == k:
        return kept + [draw(masses(p_rows[k]), w)], a
    if q_rows is None:
        q_row = np.zeros(vocab, dtype=np.float32)
        if 0 <= int(tokens[a]) < vocab:
            q_row[int(tokens[a])] = 1
    else:
        q_row = np.asarray(q_rows[a], dtype=np.float32)
    with np.errstate(invalid="ignore"):
        rest = masses(p_rows[a] - q_row)
    if not (rest > 0).any():
        rest = masses(p_rows[a])
    return kept + [draw(rest, w)], a


def verify_batch(p, q, tokens, accept, sample, query_start, draft_start, max_draft_len):
    """Padded tokens [batch][max_draft_len + 1], kept counts [batch], rejected counts [batch]."""
    batch = len(sample)
    out = np.full((batch, max_draft_len + 1), -1, dtype=np.int32)
    kept = np.zeros(batch, dtype=np.int32)
    rejected = np.zeros(batch, dtype=np.int32)
    for i in range(batch):
        t0, t1, d0, d1 = query_start[i], query_start[i + 1], draft_start[i], draft_start[i + 1]
        if t0 == t1 and d0 == d1:
            continue
        row, a = verify_sequence(p[t0:t1], None if q is None else q[d0:d1], tokens[d0:d1], accept[d0:d1],
                                 float(sample[i]))
        out[i, :len(row)] = row
        kept[i], rejected[i] = a, (d1 - d0) - a
    return out, kept, rejected
