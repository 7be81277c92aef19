"""A NaN in q or in a K row reaches the outputs of the queries that see it, whichever kernel and
split count serve them, and no other output: neither zeros nor a row left as it was.

The other outputs are held to the definition, as in test_query_attention_gpu.py, and not to the
bits of a run without the NaN: the rows of a warp move their softmax references together, when
any one of them asks for it, and a row that is NaN asks for none.  Another reference scales P' by
another 2^x before its rounding to f16, so both results are within 2^-9 |o| + 2^-11 vmax of o,
and up to twice that from each other."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
from kvq_testutil import DEV, poison_bf16, status_word
from test_query_attention_gpu import Case

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4

# whole pages, rows (3 heads; pages of 8), tiles; of one split and of many
LAYOUTS = [(2, 4, 16), (3, 2, 16), (2, 4, 8)]
LENGTHS = [([90, 40], [2, 2]), ([6000, 300], [2, 1]), ([150, 90], [60, 33]), ([6000, 300], [60, 33])]


class poison_k:
    """NaN in token t's K row of one head, within the block of the with statement."""

    def __init__(self, c, s, t, head):
        slot = int(c.slots[s][t])
        plane, col, self.nan = (c.pool.k_bscale, 1, 0x7F) if c.pool.fmt == NV else (c.pool.k_codes, 5, 0xFF)
        self.at = plane[slot, head, col:col + 1]

    def __enter__(self):
        self.was = self.at.clone()
        self.at.fill_(self.nan)

    def __exit__(self, *_):
        self.at.copy_(self.was)


@pytest.mark.parametrize("lens,new", LENGTHS)
@pytest.mark.parametrize("H,group,bs", LAYOUTS)
@pytest.mark.parametrize("fmt", [PG, F8, NV])
@pytest.mark.parametrize("opts", [{}, {"softcap": 20.0, "slopes": 1}])
def test_attention(lens, new, H, group, bs, fmt, opts):
    if opts:
        opts = {"softcap": 20.0, "slopes": np.linspace(0.001, 0.01, H * group).astype(np.float32)}
    c = Case(lens, new, H, group, 128, bs, fmt, seed=41)
    want, st = c.run(**opts)
    assert st == 0
    q = c.q.clone()
    row, qh = int(c.starts[1]) - 1, H * group - 2
    q[row, qh, 3] = float("nan")
    out, st = c.run(q=q.to(DEV), **opts)
    assert st == 0 and out[row, qh].isnan().all()
    out[row, qh] = want[row, qh]
    c.check(out, **opts)
    assert c.untouched(out, slice(c.starts[-1], c.T))
    head = H - 1
    heads = slice(head * group, (head + 1) * group)
    # the key of sequence 0's first query, which all its queries see; that of its last, which no
    # other sees
    for t, first in ((lens[0] - new[0], 0), (lens[0] - 1, new[0] - 1)):
        with poison_k(c, 0, t, head):
            out, st = c.run(**opts)
        assert st == 0 and out[first:new[0], heads].isnan().all()
        out[first:new[0], heads] = want[first:new[0], heads]
        c.check(out, **opts)


@pytest.mark.parametrize("n", [2, 60])
def test_nan_page_scales(n):
    for plane in ("k_rscale", "v_rscale"):
        c = Case([130], [n], 2, 4, 128, seed=42)
        getattr(c.pool, plane)[int(c.table[0, 8]), 1] = float("nan")  # the last page, 2 tokens of it in use
        out, st = c.run()
        assert st == 0 and out[n - 1, 4:].isnan().all()
        assert not out[:n, :4].isnan().any()


@pytest.mark.parametrize("lens", [[90, 40, 0], [6000, 300, 0]])
@pytest.mark.parametrize("H,group,D,bs", [(8, 4, 128, 16), (4, 3, 256, 16), (2, 4, 128, 16), (3, 2, 64, 16), (8, 12, 128, 16)])
@pytest.mark.parametrize("fmt", [PG, F8, NV])
def test_decode(lens, H, group, D, bs, fmt):
    c = Case(lens, [1, 1, 0], H, group, D, bs, fmt, seed=43)
    S, Hq = 3, H * group
    q = c.q[:S].to(DEV)

    def call():
        out, st = poison_bf16((S, Hq, D)), status_word()
        kvq.kvq_decode_attention(c.pool, c.table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), max(lens), q,
                                 c.scale, out, dev_status=st)
        assert int(st.item()) == 0
        return out

    want = call()
    q[1, 2, D - 1] = float("nan")
    out = call()
    assert out[1, 2].isnan().all() and (out[2] == 0).all()
    out[1, 2] = want[1, 2]
    c.check(out, seqs=[0, 1])
    q[1, 2, D - 1] = c.q[1, 2, D - 1].to(DEV)
    with poison_k(c, 0, lens[0] // 2, 1):
        out = call()
    assert out[0, group:2 * group].isnan().all()
    out[0, group:2 * group] = want[0, group:2 * group]
    c.check(out, seqs=[0, 1])


def test_bad_entries_are_told_from_nan():
    """A NaN row beside a row that stays as it was for a bad block entry, split and not."""
    for lens, new in LENGTHS:
        c = Case(lens, new, 2, 4, 128, seed=44)
        q = c.q.clone()
        q[0, 0, 0] = float("nan")
        t = c.table.clone()
        t[1, 0] = -1
        out, st = c.run(q=q.to(DEV), table=t)
        assert st == kvq.DEV_BAD_BLOCK and out[0, 0].isnan().all() and not out[0, 1:].isnan().any()
        assert c.untouched(out, slice(c.starts[1], c.starts[2]))
