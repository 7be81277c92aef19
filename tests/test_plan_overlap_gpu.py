"""kvq_plan_pages refuses outputs that overlap another of its arrays: every thread block reads
the inputs while others write.  Arrays that only touch are fine."""

import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
from kvq_testutil import DEV

pytestmark = pytest.mark.gpu
NAMES = ["cached_lens", "new_lens", "free_blocks", "block_table", "seq_lens", "query_starts", "slot_ids", "positions", "num_used",
         "dev_status"]
S, FREE, BLOCKS, T = 6, 9, 4, 12
COUNTS = [S, S, FREE, S * BLOCKS, S, S + 1, 2 * T, T, 1, 1]  # int32 words


def arrays(shift=None):
    """All arrays in one buffer, one behind the other without a gap; shift = (i, j): array j begins
    where array i's last word lies."""
    words = torch.zeros(2 * sum(COUNTS) + 64, dtype=torch.int32, device=DEV)
    at, out = 0, []
    order = [6] + [i for i in range(10) if i != 6]  # slot_ids are 64-bit: at the start
    where = {}
    for i in order:
        where[i] = at
        at += COUNTS[i]
    if shift is not None:
        i, j = shift
        where[j] = where[i] + COUNTS[i] - 1
        if j == 6 and where[j] % 2:
            where[j] -= 1
    for i, n in enumerate(COUNTS):
        t = words[where[i]:where[i] + n]
        out.append(t.view(torch.int64) if i == 6 else t.view(S, BLOCKS) if i == 3 else t)
    return out


def call(a):
    a[0].fill_(3)
    a[1].fill_(2)
    a[2].copy_(torch.arange(FREE))
    kvq.kvq_plan_pages(a[0], a[1], a[2], 16, a[3], a[4], a[5], a[6], a[7], a[8], a[9])


def test_neighbours_are_fine():
    a = arrays()
    call(a)
    assert a[4].tolist() == [5] * S and a[5].tolist() == list(range(0, 2 * S + 1, 2)) and int(a[9]) == 0


@pytest.mark.parametrize("i,o", [(i, o) for o in range(3, 10) for i in range(o)])
def test_overlaps(i, o):
    for shift in ((i, o), (o, i)):
        a = arrays(shift)
        with pytest.raises(kvq.KvqError, match="overlap"):
            kvq.kvq_plan_pages(a[0], a[1], a[2], 16, a[3], a[4], a[5], a[6], a[7], a[8], a[9])
    a = arrays()
    kvq.kvq_plan_pages(a[0], a[1], a[2], 16, a[3], a[4], a[5], a[6], None, a[8], None)
