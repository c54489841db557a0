"""Pins of the draft-verification oracle: closed forms, the distribution it
leaves (exact, by integrating over the uniform numbers), and planted mistakes
that a pin catches."""

import numpy as np
import pytest

from oracle import verify as OV


def output_distribution(p, q, verify=OV.verify_sequence, grid=200):
    """Distribution of the first emitted token over draft x ~ q and a midpoint
    grid of u and w (exact up to 1/grid for step functions)."""
    got = np.zeros(len(p))
    mids = (np.arange(grid) + 0.5) / grid
    for x in range(len(p)):
        if q[x] == 0:
            continue
        for u in mids:
            row, a = verify([p, p], [q], [x], [u], 0.0)
            if a == 1:
                got[row[0]] += q[x] / grid
                continue
            for w in mids:
                got[verify([p, p], [q], [x], [u], w)[0][0]] += q[x] / grid / grid
    return got


P = np.array([0.5, 0.2, 0.05, 0.25, 0.0], dtype=np.float32)
Q = np.array([0.1, 0.4, 0.25, 0.0, 0.25], dtype=np.float32)


def test_the_targets_distribution_is_left_unchanged():
    assert np.abs(output_distribution(P, Q, grid=60) - P).max() < 2 / 60


def test_closed_forms():
    one = np.eye(4, dtype=np.float32)
    # certain target: the right drafts are kept, the wrong one is replaced by the target's token
    row, a = OV.verify_sequence([one[2], one[1], one[3]], [one[2], one[0]], [2, 0], [0.9, 0.0], 0.5)
    assert (row, a) == ([2, 1], 1)
    row, a = OV.verify_sequence([one[2], one[0], one[3]], [one[2], one[0]], [2, 0], [0.9, 0.99], 0.5)
    assert (row, a) == ([2, 0, 3], 2)
    # equal distributions: always kept; no draft: a draw from the row
    assert OV.verify_sequence([P, P], [P], [1], [0.999], 0.0)[1] == 1
    assert OV.verify_sequence([P], [], [], [], 0.6)[0] == [1]
    # borders: the lowest index whose running sum EXCEEDS w * sum
    assert OV.draw(np.array([0.25, 0.25, 0.5]), 0.25) == 1
    assert OV.draw(np.array([0.0, 0.25, 0.0, 0.75]), 0.0) == 1
    assert OV.draw(np.zeros(3), 0.3) == -1
    # NaN and infinities carry no mass
    assert OV.draw(OV.masses(np.array([np.nan, np.inf, -1, 0.5], dtype=np.float32)), 0.0) == 3
    # certain drafts: kept with the target's probability, then drawn from the others
    assert OV.verify_sequence([P, P], None, [0], [0.49], 0.0)[1] == 1
    assert OV.verify_sequence([P, P], None, [0], [0.51], 0.0) == ([1], 0)
    # p <= q everywhere (rounding): the draw falls back to p
    assert OV.verify_sequence([Q / 2, Q], [Q], [0], [0.9], 0.0) == ([0], 0)
    # an idle sequence, ragged counts
    out, kept, rej = OV.verify_batch(np.stack([one[1], one[1], one[0]]), np.stack([one[1]]), [1], [0.5], [0.1, 0.1, 0.1],
                                     [0, 2, 2, 3], [0, 1, 1, 1], 2)
    assert out.tolist() == [[1, 1, -1], [-1, -1, -1], [0, -1, -1]] and kept.tolist() == [1, 0, 0]


def mutant(name):
    def verify(p_rows, q_rows, tokens, accept, w):
        kept = []
        for j, x in enumerate(tokens):
            ok = accept[j] * q_rows[j][x] < p_rows[j][x]
            if name == "inverted":
                ok = accept[j] * p_rows[j][x] < q_rows[j][x]
            if not ok:
                break
            kept.append(x)
        a = len(kept)
        if a == len(tokens):
            return kept + [OV.draw(OV.masses(p_rows[a]), w)], a
        rest = p_rows[a] - q_rows[a]
        if name == "from p":
            rest = p_rows[a]
        if name == "absolute":
            rest = np.abs(rest)
        if name == "unscaled aim":
            return kept + [OV.draw(OV.masses(rest), w / OV.masses(rest).sum())], a
        return kept + [OV.draw(OV.masses(rest), w)], a
    return verify


@pytest.mark.parametrize("name", ["inverted", "from p", "absolute", "unscaled aim"])
def test_planted_mistakes_change_the_distribution(name):
    assert np.abs(output_distribution(P, Q, mutant(name), grid=60) - P).max() > 3 / 60
