"""pkv_multiquery_attention_q8 where one token takes nearly all of a row's weight and
its value is nothing: the row is what the tail of small weights adds up to.

Tolerance per element: that of tests/test_gpu_chunk_q8.py but for the smallest weights.
There f16's smallest step counts as 2^-25 of the row's largest weight. The tile kernel
holds a weight that stands out this far at 2^9, the largest where none does at 2^0 or
more: here n tokens lose at most n 2^-34 max|V| (n 2^-32 is allowed).
Where the cache is split, the weight times the V scale is what is rounded, rows of zero
codes aside, and the largest of these is 2^8 or more: n tokens lose at most
2^-33 n max_p w_p vs_p times a code of at most 2^7, which is less than
2^-11 sum_p softmax_p vs_p up to 2^15 tokens and needs no term of its own. Rows of zero
codes lose nothing as V values either and are left out of that sum.
"""

import numpy as np
import pytest
import torch

import test_gpu_chunk_q8 as T
from oracle import attention as OA
from oracle import multiquery as OM
from oracle import quant as OQ
import cases
from test_gpu_chunk_q8 import pkv  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def sink_case(seed, lens, nqs, kv_heads, d, nats, where=0):
    """Scores about N(0, 1/2) with token `where` `nats` above, whose V row is zero; V elsewhere in 1 .. 2."""
    c = cases.multiquery_case(seed, lens, nqs, 4 * kv_heads, kv_heads, d, torch.bfloat16)
    rng = np.random.default_rng(seed)
    c["scale"] = float(np.float32(c["scale"]))
    q = c["q"].float() * 0.5
    q[..., 0] = 16
    c["q"] = q.to(torch.bfloat16)
    kp = rng.standard_normal((*c["k_pool"].shape[:3], d))
    kp[..., 0] = 0
    vp = rng.uniform(1, 2, kp.shape)
    b, s = c["tables"][:, where // 16], where % 16
    kp[b, :, s] = 0
    kp[b, :, s, 0] = nats / (16 * c["scale"])
    vp[b, :, s] = 0
    c["kc"], c["ks"] = OQ.quantize_rows(kp)
    c["vc"], c["vs"] = OQ.quantize_rows(vp)
    return c


def reference(c, few):
    kd, vd = OQ.dequantize_rows(c["kc"], c["ks"]), OQ.dequantize_rows(c["vc"], c["vs"])
    qf = OA.bf16_bits_to_f64(cases.host_view(c["q"]))
    attend = lambda v: OM.multiquery_attention(qf, kd, v, c["tables"], c["lens"], c["query_start"], c["scale"],  # noqa: E731
                                               c["kv_heads"], "f64")
    ref, size = attend(vd), attend(np.abs(vd))
    n = int(max(c["lens"]))
    vs = np.where((c["vc"] != 0).any(-1), c["vs"].astype(np.float64), 0.0)
    b = T.score_error(c["scale"], qf, np.linalg.norm(kd, axis=-1).max(), float(c["ks"].max()))[..., None]
    tol = 2.0 ** -8 * np.abs(ref) + size * (3 * 2.0 ** -11 + 2 * b + 2.0 ** -20 + n * 2.0 ** -23)
    tol += 2.0 ** -11 * attend(np.broadcast_to(vs[..., None], vd.shape))
    return ref, tol if few else tol + n * 2.0 ** -32 * np.abs(vd).max()


@pytest.mark.parametrize("nats", [10.0, 17.0, 18.0])
@pytest.mark.parametrize("n,nq,d,where", [(1200, 40, 64, 0), (1200, 40, 128, 0), (1200, 40, 128, 700), (8000, 200, 128, 3)])
def test_sink_of_zero_value(pkv, n, nq, d, where, nats):  # noqa: F811
    c = sink_case(31, [n], [nq], 1, d, nats, where)
    T.check(T.call(pkv, c), c, reference(c, False))
    assert pkv.pkv_device_status(clear=True) == 0


@pytest.mark.parametrize("nats", [10.0, 17.0, 18.0, 30.0])
@pytest.mark.parametrize("n,nq,where", [(1200, 4, 0), (300, 4, 0), (300, 1, 150), (250, 3, 3)])
def test_sink_of_zero_value_few_rows(pkv, n, nq, where, nats):  # noqa: F811
    """(So many sequences that the kernel that splits the cache leaves most of them whole.)"""
    batch = 1 if n > 300 else 90
    c = sink_case(32, [n] * batch, [nq] * batch, 4, 128, nats, where)
    want = reference(c, True)
    c["tables"] = np.pad(c["tables"], ((0, 0), (0, 8300 // batch)), constant_values=-1)      # that kernel takes the call
    T.check(T.call(pkv, c), c, want)
    assert pkv.pkv_device_status(clear=True) == 0
