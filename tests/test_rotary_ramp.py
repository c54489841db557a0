"""PKV_ROTARY_RAMP from the sentence of include/pkv.h, worked out here and nowhere else: where the ramp ends past the
last pair, lies inside the pairs, begins before them, or has no width."""

import math

import numpy as np
import pytest

BASE = 10000.0
# (base, rotary_dim, original_context, stretch, low_turns, high_turns), the dimensions between which the mix runs
CASES = [
    ((BASE, 128, 131072, 8.0, 1.0, 32.0), (45, 70)),        # past the last pair, 63
    ((BASE, 128, 65536, 4.0, 1.0, 32.0), (40, 65)),
    ((BASE, 64, 131072, 4.0, 1.0, 32.0), (22, 35)),
    ((BASE, 128, 4096, 8.0, 1.0, 32.0), (20, 46)),          # inside
    ((1e6, 128, 32768, 4.0, 1.0, 32.0), (23, 40)),
    ((100.0, 6, 4096, 4.0, 1.0, 32.0), (1, 5)),             # ends at R - 1
    ((100.0, 6, 1e7, 4.0, 1.0, 32.0), (7, 5)),              # every pair makes high_turns: nothing is stretched
    ((BASE, 128, 100, 2.0, 1.0, 32.0), (0, 20)),            # no pair makes high_turns
    ((BASE, 128, 3, 2.0, 1.0, 32.0), (0, -5)),              # none makes low_turns
]


@pytest.mark.parametrize("how,ends", CASES)
def test_ramp(how, ends):
    from paged_kv_cache_209_gb300 import pkv
    base, dim, context, stretch, low, high = how

    def makes(turns):                                       # the i at which context f_i / (2 pi) = turns
        return math.log(context / (2 * math.pi * turns)) / math.log(base) * dim / 2
    a, b = max(0, math.floor(makes(high))), min(dim - 1, math.ceil(makes(low)))
    assert (a, b) == ends
    want = []
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        if b <= a:
            mixed = 0.0 if i <= a else 1.0
        else:
            mixed = min(1.0, max(0.0, (i - a) / (b - a)))
        want.append(f * (1 - mixed) + f / stretch * mixed)
    got = pkv.pkv_rotary_frequencies(dim, base, "ramp", stretch=stretch, original_context=context, low_turns=low,
                                     high_turns=high).numpy()
    assert np.allclose(got, want, rtol=1e-12, atol=0)
