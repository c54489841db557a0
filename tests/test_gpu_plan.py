"""Planning a step on the GPU against the oracle, whole numbers throughout."""

import numpy as np
import pytest
import torch

from oracle.plan import plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_209_gb300 import pkv
    pkv.pkv_device_status(clear=True)
    yield pkv
    assert pkv.pkv_device_status(clear=True) == 0


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype))).cuda()


def compare(pkv, lens, new, held, free, left, tables, rows, num_blocks=0, bad=None):
    want = plan(lens, new, held, free, left, tables, rows, num_blocks or 1 << 31)
    t = dev(tables)
    got = pkv.pkv_plan_step(dev(lens), dev(new), dev(held), dev(free), dev([left]), t, rows, num_blocks)
    names = ("slots", "positions", "start", "lens", "held")
    for name, g in zip(names, got):
        assert np.array_equal(g.cpu().numpy(), want[name]), name
    assert got[5].item() == want["left"] and got[6].tolist() == want["result"]
    assert np.array_equal(t.cpu().numpy(), want["tables"])
    assert pkv.pkv_device_status(clear=True) == (pkv.PKV_DEVERR_RANGE if want["bad"] else 0)
    if bad is not None:
        assert want["bad"] == bad
    return want


def batch(seed, n, longest=300, most=40, spare=0, width=None):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, n)
    new = rng.integers(0, most + 1, n) * (rng.random(n) < 0.7)
    held = -(-lens // 16) + rng.integers(0, spare + 1, n)
    width = width or int(max((-(-(lens + new) // 16)).max(), held.max(), 1))
    held = np.minimum(held, width)
    need = int(np.maximum(-(-(lens + new) // 16) - held, 0).sum())
    order = rng.permutation(int(held.sum()) + need + 7)
    tables = np.full((n, width), -1, np.int32)
    at = 0
    for i in range(n):
        tables[i, :held[i]] = order[at:at + held[i]]
        at += held[i]
    return lens, new, held, order[at:], len(order) - at, tables


@pytest.mark.parametrize("n", [1, 2, 31, 33, 500, 1023, 1025, 3000, 16384])
@pytest.mark.parametrize("spare", [0, 3])
def test_against_the_oracle(pkv, n, spare):
    lens, new, held, free, left, tables = batch(n + spare, n, spare=spare, most=40 if n < 5000 else 3)
    rows = int(new.sum())
    compare(pkv, lens, new, held, free, left, tables, rows, bad=False)
    compare(pkv, lens, new, held, free, left, tables, rows + 4099, num_blocks=1 << 20, bad=False)


def test_long_prompts(pkv):
    lens, new, held, free, left, tables = batch(1, 5, most=60000)
    compare(pkv, lens, new, held, free, left, tables, int(new.sum()) + 1, bad=False)


def test_nothing_new(pkv):
    lens, new, held, free, left, tables = batch(2, 40)
    compare(pkv, lens, new * 0, held, free, left, tables, 0, bad=False)
    compare(pkv, lens, new * 0, held, free, left, tables, 9, bad=False)
    compare(pkv, lens, new * 0, held, free[:0], 0, tables, 9, bad=False)


@pytest.mark.parametrize("n", [3, 1500])
def test_out_of_blocks_changes_nothing(pkv, n):
    lens, new, held, free, left, tables = batch(3, n, most=90)
    rows = int(new.sum())
    need = int(np.maximum(-(-(lens + new) // 16) - held, 0).sum())
    assert need > 1
    exact = compare(pkv, lens, new, held, free, need, tables, rows, bad=False)
    assert exact["left"] == 0
    short = compare(pkv, lens, new, held, free, need - 1, tables, rows, bad=False)
    assert short["result"] == [0, 1] and np.array_equal(short["tables"], tables)
    t, r = dev(tables), torch.full((rows,), 77, dtype=torch.int64, device="cuda")
    out = (r, *(torch.full((k,), 77, dtype=torch.int32, device="cuda") for k in (rows, n + 1, n, n, 1, 2)))
    with pytest.raises(pkv.PkvError, match="PKV_ERR_OUT_OF_BLOCKS"):
        pkv.pkv_plan_step(dev(lens), dev(new), dev(held), dev(free), dev([need - 1]), t, rows, flags=pkv.PKV_FLAG_CHECKED, out=out)
    assert all(bool((x == 77).all()) for x in out) and np.array_equal(t.cpu().numpy(), tables)
    pkv.pkv_plan_step(dev(lens), dev(new), dev(held), dev(free), dev([need]), t, rows, flags=pkv.PKV_FLAG_CHECKED, out=out)
    assert np.array_equal(out[0].cpu().numpy(), exact["slots"])


def test_bad_numbers(pkv):
    lens, new, held, free, left, tables = batch(4, 30, spare=1)
    rows = int(new.sum())
    for what, i, value in (("lens", 3, -1), ("new", 4, -2), ("held", 5, -1), ("held", 6, tables.shape[1] + 1), ("lens", 7, 16 * int(held[7]) + 1),
                           ("new", 8, 16 * tables.shape[1]), ("new", 9, 2 ** 31 - 1), ("lens", 10, 2 ** 31 - 1)):
        given = dict(lens=lens.copy(), new=new.copy(), held=held.copy())
        given[what][i] = value
        compare(pkv, given["lens"], given["new"], given["held"], free, left, tables, rows, bad=True)
        with pytest.raises(pkv.PkvError, match="PKV_ERR_RANGE"):
            pkv.pkv_plan_step(dev(given["lens"]), dev(given["new"]), dev(given["held"]), dev(free), dev([left]), dev(tables), rows,
                              flags=pkv.PKV_FLAG_CHECKED)
    compare(pkv, lens, new, held, free, left, tables, rows - 1, bad=True)       # more rows than there is room for
    compare(pkv, lens, new, held, free, -1, tables, rows, bad=True)
    compare(pkv, lens, new, held, free, len(free) + 1, tables, rows, bad=True)
    all_new = np.full(30, 2 ** 31 - 1)
    compare(pkv, lens * 0, all_new, held, free, left, tables, rows, bad=True)


def test_bad_blocks(pkv):
    lens, new, held, free, left, tables = batch(5, 20)
    blocks = int(max(free.max(), tables.max())) + 1
    rows = int(new.sum())
    free, tables = free.copy(), tables.copy()
    free[left - 2] = blocks
    free[left - 3] = -4
    i = int(np.flatnonzero((new > 0) & (lens % 16 > 0))[0])
    tables[i, lens[i] // 16] = -1
    compare(pkv, lens, new, held, free, left, tables, rows, num_blocks=blocks, bad=True)


def test_empty_batch(pkv):
    none = dev(np.zeros(0))
    out = pkv.pkv_plan_step(none, none, none, dev([3, 4]), dev([2]), dev(np.zeros((0, 4))), 3)
    assert out[0].tolist() == [-1] * 3 and out[1].tolist() == [-1] * 3 and out[2].tolist() == [0]
    assert out[5].tolist() == [2] and out[6].tolist() == [0, 0]


def test_refusals(pkv):
    lens, new, held, free, left, tables = (dev(x) for x in batch(6, 4)[:4] + ([9],) + batch(6, 4)[5:])
    rows = int(new.sum())
    with pytest.raises(ValueError):
        pkv.pkv_plan_step(lens.long(), new, held, free, left, tables, rows)
    with pytest.raises(ValueError):
        pkv.pkv_plan_step(lens, new[:3], held, free, left, tables, rows)
    with pytest.raises(ValueError):
        pkv.pkv_plan_step(lens.cpu(), new, held, free, left, tables, rows)
    out = pkv.pkv_plan_step(lens, new, held, free, left, tables, rows)
    with pytest.raises(pkv.PkvError, match="PKV_ERR_OVERLAP"):
        pkv.pkv_plan_step(lens, new, held, free, left, tables, rows, out=(*out[:3], lens, *out[4:]))
    with pytest.raises(ValueError):
        pkv.pkv_plan_step(lens, new, held, free, left, tables, rows + 1, out=out)
    with pytest.raises(ValueError):
        pkv.pkv_plan_step(lens, new, held, free, left, tables, rows, out=out[:6])
