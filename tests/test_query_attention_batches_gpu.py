"""kvq_attention at KV head counts above 8, and over steps that mix single tokens, drafts and
prompt chunks in one call."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
from kvq_testutil import DEV, poison_bf16, status_word
from test_query_attention_gpu import Case

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4


@pytest.mark.parametrize("H,group,D", [(16, 1, 128), (32, 1, 64), (12, 2, 128), (16, 4, 64), (40, 1, 128), (16, 1, 256)])
@pytest.mark.parametrize("new", [[1, 1], [5, 2], [70, 33]])
@pytest.mark.parametrize("fmts", [(PG, None), (NV, None), (F8, NV)])
def test_many_kv_heads(H, group, D, new, fmts):
    c = Case([333, 90], new, H, group, D, 16, *fmts, seed=91)
    for opts in ({}, {"window": 50, "softcap": 20.0}, {"slopes": np.linspace(0.002, 0.3, H * group).astype(np.float32)}):
        out, st = c.run(**opts)
        assert st == 0 and c.untouched(out, slice(c.starts[-1], c.T))
        c.check(out, **opts)


@pytest.mark.parametrize("H,group,D,bs,fmt", [(2, 4, 128, 16, PG), (4, 2, 64, 16, NV), (3, 2, 128, 8, F8), (1, 4, 256, 32, PG)])
def test_mixed_steps(H, group, D, bs, fmt):
    """Decoding requests, drafts, two chunks, a whole prompt, requests without a new token and an
    empty one, in an order of their own."""
    rng = np.random.default_rng(H)
    new = [1] * 40 + [4] * 6 + [130, 300, 64, 0, 0]
    lens = [int(x) for x in rng.integers(1, 900, 40)] + [int(x) for x in rng.integers(4, 500, 6)] + [500, 1200, 64, 33, 0]
    order = rng.permutation(len(new))
    c = Case([lens[i] for i in order], [new[i] for i in order], H, group, D, bs, fmt, seed=92)
    for opts in ({}, {"softcap": 30.0, "window": 200}):
        out, st = c.run(**opts)
        assert st == 0 and c.untouched(out, slice(c.starts[-1], c.T))
        c.check(out, **opts)
    # the single tokens alone are the same attention
    ones = [s for s in range(len(c.new)) if c.new[s] == 1]
    rows = torch.tensor([int(c.starts[s]) for s in ones])
    q, table = c.q[rows].to(DEV), c.table[ones].contiguous().to(DEV)
    dec, st = poison_bf16(tuple(q.shape)), status_word()
    kvq.kvq_decode_attention(c.pool, table, torch.tensor([c.lens[s] for s in ones], dtype=torch.int32, device=DEV), max(c.lens), q,
                             c.scale, dec, dev_status=st)
    assert int(st.item()) == 0
    full = poison_bf16(tuple(c.q.shape))
    full[rows.to(DEV)] = dec
    c.check(full, seqs=ones)
