"""What the 4-bit attention's products of up to 32 rows keep of small parts beside large ones, to the bounds that
include/pkv.h states.

The tensor cores line the 16 products of an instruction up at the largest one's exponent, taking an operand below the
normal range at that range's end, and cut what lies 23 bits and more below. A code n sits in the low bits of such an
operand, of 10 bits in f16 (V: what is cut of n P' is below 2^-15 of the largest P' of the 16 tokens, in the sum over
code + 8 and in that of the eights, which is taken off: the two partly undo each other) and of 7 in bf16 (K: below 2^-18
of the largest q of the 16 dimensions, so 2^-14 of it in all 16)."""

import numpy as np
import pytest
import torch

from q4_cases import B, fast_pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def run(pkv, kc, vc, ks, vs, q, scale):
    """One sequence of one KV head, one query of as many heads as q has rows, against float64: (out, want, weights, V, scores' part)."""
    n, d = kc.shape
    blocks = -(-n // B)
    fill = lambda x: np.concatenate([x, np.zeros((blocks * B - n, *x.shape[1:]), x.dtype)])  # noqa: E731
    cache = fast_pack(*(fill(c).reshape(blocks, 1, B, d) for c in (kc, vc)), *(fill(s).reshape(blocks, 1, B) for s in (ks, vs)))
    q = torch.from_numpy(q).to(torch.bfloat16)
    got = pkv.pkv_decode_attention_q4(q.cuda()[None], torch.from_numpy(cache).cuda(),
                                      torch.arange(blocks, dtype=torch.int32, device="cuda")[None],
                                      torch.tensor([n], dtype=torch.int32, device="cuda"), scale)[0].double().cpu().numpy()
    x = q.double().numpy()
    k, v = kc * ks.astype(np.float64)[:, None], vc * vs.astype(np.float64)[:, None]
    z = scale * (x @ k.T)
    w = np.exp(z - z.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    # a score: its parts of 16 dimensions, 2^-14 of the largest |q| of each (the d / 16 largest |q| are no less), and what
    # their sum, 15 sum|q| at most, is rounded to: 2^-23 of it d / 16 times, twice, less than 2^-15 sum|q|
    size = np.sort(np.abs(x), -1)
    delta = scale * ks.max() * (2.0 ** -14 * size[:, -(d // 16):].sum(-1) + 2.0 ** -15 * size.sum(-1))[:, None]
    return got, w @ v, w, v, delta


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 5, 16, 32])
@pytest.mark.parametrize("top", [64.0, -100.0, 3.0])
@pytest.mark.parametrize("below", [14, 16, 18])
@pytest.mark.parametrize("where", [0, 5])
def test_scores_beside_a_large_dimension(pkv, d, rows, top, below, where):
    """One dimension of q is 2^14 to 2^18 times the others, and K's code there is the same for all tokens: the scores'
    differences come from the others, in half of the tokens of odd codes, in half of even ones."""
    n = 64
    rng = np.random.default_rng(d + rows)
    odd = (np.arange(n) % 2 == 1)[:, None]
    sign = rng.choice([-1, 1], (n, d))
    kc = np.where(odd, sign * rng.choice([1, 3], (n, d)), sign * rng.choice([2, 4], (n, d))).astype(np.int8)
    kc[:, where] = 3
    vc = np.broadcast_to(np.where(odd, 7, -7), (n, d)).astype(np.int8)
    q = np.full((rows, d), abs(top) * 2.0 ** -below)
    q[:, where] = top
    one = np.full(n, 1.0, np.float32)
    size = 0.1 / (2.0 ** -14 * abs(top))
    got, want, w, v, delta = run(pkv, kc, vc, one, one, q, float(np.float32(size)))
    # out moves by sum w (v - out) dz, at most 7 delta with values of +-7; a weight is rounded to f16 once, on either side of
    # the quotient; sums as below; one bf16 step
    bound = np.abs(want) * 2.0 ** -8 + 7 * (delta + 2.0 ** -11 + n * 2.0 ** -15 * w.max(-1, keepdims=True))
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 5, 16, 32])
@pytest.mark.parametrize("below", [6, 9, 12, 15])
@pytest.mark.parametrize("at", [0, 10, 33])
def test_values_beside_a_token_of_no_value(pkv, d, rows, below, at):
    """One token has nearly all of the weight and its codes are 0; the others, 2^-6 to 2^-15 of it, have codes."""
    n = 40
    rng = np.random.default_rng(d + rows + below)
    kc, vc = np.zeros((n, d), np.int8), rng.integers(-7, 8, (n, d)).astype(np.int8)
    kc[at, :], vc[at] = 7, 0
    ks, vs = np.full(n, 1.0, np.float32), rng.uniform(0.5, 1.0, n).astype(np.float32)
    q = np.full((rows, d), 1.0)
    scale = below * np.log(2) / (7 * d)
    got, want, w, v, delta = run(pkv, kc, vc, ks, vs, q, float(np.float32(scale)))
    product = w * vs
    # the other tokens' weights: delta, and one rounding to f16; the sums: 2^-15 of the largest product a token, and fp32's
    bound = np.abs(want) * 2.0 ** -8 + (w @ np.abs(v)) * (np.expm1(2 * delta) + 2.0 ** -11) + \
        n * 2.0 ** -15 * product.max(-1, keepdims=True) + (n / 4 + 368) * 2.0 ** -23 * product.sum(-1, keepdims=True)
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("news", [[1, 1], [4, 3], [8, 8]])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k_size,q_size,scale", [(1e-37, 1e37, 0.02), (1e-36, 1e36, 0.2), (1e36, 1e-37, 1.0), (1e37, 1e-39, 10.0)])
def test_queries_at_the_ends_of_the_range(pkv, news, d, k_size, q_size, scale):
    """Up to |scale| max|q| = 2^120 (4.5 of the spread at most), and down to q below the normal range."""
    from q4_cases import check, make, reference
    s = make(61, [200, 333], news, 8, 2, d, spread=q_size, k_sizes=lambda rng, shape: np.full(shape, k_size))
    s["scale"] = scale
    check(pkv.pkv_multiquery_attention_q4(s["q"], s["cache"], s["tables"], s["lens"], s["start"], s["scale"], max(news)), *reference(s))
