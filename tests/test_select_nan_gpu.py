"""kvq_select_blocks with NaN among the queries: all scores of such a query are NaN, so its list goes by the
blocks' order, and no other query's list changes."""

import numpy as np
import pytest
import torch

from test_select_blocks_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [[1, 2], [4, 7], [40, 9]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_queries(new, D):
    c = Case([1600, 700], new, 2, 3, D, 8, seed=D + new[0])
    r = np.random.RandomState(1)
    c.q = c.q * 2.0 ** -3
    hit = [0, c.T - 3] + r.randint(0, c.T - 2, 4).tolist()
    for t in hit:
        c.q[t, r.randint(0, 6), r.randint(0, D)] = float("nan")
    c.q[1, 5, :] = float("nan")
    c.check(9, 1, 2)
    got, _ = c.run(9, 0, 0)
    assert (got[1, 1] == np.arange(9)).all()
