"""Queries near the end of bf16's range over keys near its start: ordinary scores.  The power of
two that brings a query into f16 has to reach bf16's largest exponent."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
from kvq_testutil import DEV, poison_bf16, status_word
from test_query_attention_gpu import Case

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4


@pytest.mark.parametrize("H,group,D,bs", [(8, 2, 128, 16), (3, 4, 64, 16), (4, 4, 256, 8)])
@pytest.mark.parametrize("fmt", [PG, F8, NV])
@pytest.mark.parametrize("up", [40, 116, 122])
def test_they_are_scaled_exactly(H, group, D, bs, fmt, up):
    for new in (1, 3, 60):
        c = Case([150, 70], [new, new], H, group, D, bs, fmt, seed=81)
        c.q = (c.q.double().clamp(-30, 30) * 2.0 ** up).to(torch.bfloat16)
        assert torch.isfinite(c.q).all()
        c.pool.k_rscale.mul_(2.0 ** -(up // 2)).mul_(2.0 ** (up // 2 - up))
        out, st = c.run()
        assert st == 0
        c.check(out)
        if new == 1:
            out, st = poison_bf16((2, H * group, D)), status_word()
            kvq.kvq_decode_attention(c.pool, c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV), 150,
                                     c.q[:2].to(DEV), c.scale, out, dev_status=st)
            assert int(st.item()) == 0
            c.check(out)
