"""Query rows behind a long context of keys that are each far fainter than one sink: together
they are the output.  A block table of one page over and over stands in for the long cache."""

import math

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
from kvq_testutil import DEV, poison_bf16, status_word

pytestmark = pytest.mark.gpu


def behind_a_sink(D, H, S, fmt, bs, new):
    """V is 1 but for the sink, whose V is 0.  With w = 2^-26.5 a key and n of them the output is
    n w / (1 + n w), about 2^-8.5.  P' of such a key is 2^-20.5 or more in f16, off by at most
    2^-25, so the output is off by at most 2^-4.5 of itself + 2^-8 of itself; without the keys it
    would be 0."""
    n = 1 << 18
    pool = kvq.KvPool.empty(2 * bs, H, D, bs, fill=0, fmt=fmt)
    k, v = torch.zeros((2 * bs, H, D)), torch.ones((2 * bs, H, D))
    k[0, :, 0] = 6.0  # the sink: exact in both formats
    v[0] = 0.0
    kvq.kvq_quant_scatter(k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), torch.arange(2 * bs, device=DEV), pool)
    q = torch.zeros((S * new, H, D))
    q[..., 0] = 1.0
    gap = 26.5 * math.log(2)
    table = torch.ones((S, n // bs), dtype=torch.int32)
    table[:, 0] = 0
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    out, st = poison_bf16((S * new, H, D)), status_word()
    kvq.kvq_attention(pool, table.to(DEV), i32([n] * S), n, q.to(torch.bfloat16).to(DEV), i32(list(range(0, S * new + 1, new))), new,
                      gap / 6.0, out, dev_status=st)
    assert int(st.item()) == 0
    w = np.exp(-np.float64(np.float32(gap / 6.0)) * 6.0)
    seen = (n - new + 1 + np.arange(new) - 1).astype(np.float64)  # keys beside the sink, of each row
    want = np.tile(seen * w / (1 + seen * w), S)[:, None, None]
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= (2.0 ** -4.5 + 2.0 ** -8) * want).all(), (got.min(), got.max(), want.min())


@pytest.mark.parametrize("D,H,S,fmt", [(128, 8, 20, kvq.FMT_FP8_PAGE), (64, 8, 20, kvq.FMT_NVFP4), (256, 8, 20, kvq.FMT_FP8_PAGE)])
def test_many_rows(D, H, S, fmt):
    behind_a_sink(D, H, S, fmt, 16, 20)


@pytest.mark.parametrize("D,H,S,fmt,bs,new", [(128, 8, 400, kvq.FMT_FP8_PAGE, 16, 1), (64, 8, 400, kvq.FMT_NVFP4, 16, 3),
                                              (128, 8, 400, kvq.FMT_FP8, 8, 1), (256, 8, 200, kvq.FMT_FP8, 16, 2)])
def test_few_rows_of_sequences_that_are_not_split(D, H, S, fmt, bs, new):
    behind_a_sink(D, H, S, fmt, bs, new)
