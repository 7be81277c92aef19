"""A long chunk given to the choice of blocks and to attention in pieces, each with the sequence's length up
to its own last token: the same lists, and attention within its tolerance of the same rows."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
from kvq_testutil import DEV
from test_query_attention_gpu import Case as Paged
from test_select_blocks_gpu import Case
from test_sparse_attention_gpu import _check, _lists

pytestmark = pytest.mark.gpu
i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)
CUTS = (0, 1, 9, 10, 87, 300)


@pytest.mark.parametrize("D", [64, 256])
def test_lists_in_pieces(D):
    c = Case([3000], [300], 2, 4, D, 8, seed=3, spare=0)
    want = c.want(12)
    sel, q, bounds, table = i32(np.full(want.shape, -7)), c.q.to(DEV), c.bounds.to(DEV), i32(c.table)
    for a, b in zip(CUTS, CUTS[1:]):
        kvq.kvq_select_blocks(bounds, table, i32([2700 + b]), 3000, 8, q[a:b], i32([0, b - a]), b - a, sel[a:b])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(sel.cpu().numpy(), want)


def test_attention_in_pieces():
    c = Paged([3000], [300], 2, 4, 128, 16, seed=4, spare=0)
    lists = _lists(c, 40)
    out, q, table, sel = torch.zeros((300, 8, 128), dtype=torch.bfloat16, device=DEV), c.q.to(DEV), c.table.to(DEV), i32(lists)
    for a, b in zip(CUTS, CUTS[1:]):
        kvq.kvq_sparse_attention(c.pool, table, i32([2700 + b]), 3000, q[a:b], i32([0, b - a]), b - a, sel[a:b], c.scale, out[a:b])
    torch.cuda.synchronize()
    _check(c, lists, out)
