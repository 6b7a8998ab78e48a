"""Drafted trees whose query_start_loc names rows that do not exist: as in paged_attention, the call reports them."""
import numpy as np
import pytest
import torch

from test_gpu_candidates import BF, F32, Tree, check, pkv  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("more", [0, 140])
@pytest.mark.parametrize("what", ["past the end", "before the start", "descending"])
def test_tree_rows_that_cannot_be_addressed_are_flagged(pkv, what, more, dtype, d):  # noqa: F811
    b = Tree(31 + more, [100, 40, 30] + [20] * more, [3, 4, 5] + [2] * more, 8, 2, dtype=dtype, d=d)
    want, tol = b.expected()
    last = len(b.nodes) - 1
    hit = 0 if what == "before the start" else last
    first, end = int(b.qsl[hit]), int(b.qsl[hit + 1])
    if what == "past the end":
        b.qsl[-1] += 40
    elif what == "before the start":
        b.qsl[0] = -3
    else:
        b.qsl[-1] = b.qsl[-2] - 1
    got = b.run(pkv, out=torch.full(b.q.shape, 7.0, dtype=dtype, device="cuda"))
    assert pkv.pkv_peek_error_bits() == 0b100
    assert pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX
    # what exists of the request's rows is zero; a request that ends before it begins has none
    assert (got[first:end] == (7 if what == "descending" else 0)).all()
    rest = np.r_[0:first, end:int(want.shape[0])]
    check(got[rest], want[rest], tol[rest])


def test_tree_requests_without_rows_are_not_flagged(pkv):  # noqa: F811
    b = Tree(32, [100, 0, 30, 0], [3, 0, 5, 0], 8, 2)
    check(b.run(pkv), *b.expected())
    assert pkv.pkv_get_last_error() == 0
