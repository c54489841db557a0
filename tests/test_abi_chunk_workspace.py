"""The size of the int8 multi-query call's workspace is 0 for every size that the call
itself rejects (host checks; no GPU needed)."""

import pytest

import test_abi_serving as A
from test_abi_serving import lib  # noqa: F401  (fixture)


@pytest.mark.parametrize("kw", [dict(maxb=0), dict(maxb=-3), dict(maxb=1 << 27), dict(batch=1000, maxb=1 << 22),
                                dict(nq=0), dict(heads=30), dict(batch=-1)])
def test_rejected_sizes_have_no_workspace(lib, kw):  # noqa: F811
    a = dict(batch=2, heads=32, maxb=16, nq=64)
    a.update(kw)
    assert A.chunk(lib, **kw) == A.SHAPE
    assert lib.pkv_multiquery_q8_workspace_size(a["batch"], a["heads"], a["maxb"], a["nq"], A.desc()) == 0


def test_sizes_at_the_limits(lib):  # noqa: F811
    size = lambda batch, maxb: lib.pkv_multiquery_q8_workspace_size(batch, 32, maxb, 64, A.desc())  # noqa: E731
    assert size(1, (1 << 27) - 1) == size(2, 16) > 0
    assert size(1024, (1 << 21) - 1) > 0 and size(5000, (1 << 21) - 1) > 0 and size(1024, 1 << 21) == 0
    assert size(0, 0) > 0                                    # a call without sequences does nothing, whatever the width
