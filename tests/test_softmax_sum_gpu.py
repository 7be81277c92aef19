"""kvq_attention where V's page scales differ strongly from step to step: keys whose V is zero or
tiny still take their part of the softmax sum.  The tolerance is that of
test_query_attention_gpu.py; V zero in half of the keys halves the output, so a sum without
them is off by its own size."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
from kvq_testutil import DEV
from test_query_attention_gpu import Case

pytestmark = pytest.mark.gpu

OPTS = [{}, {"softcap": 5.0}, {"slopes": np.linspace(0.0005, 0.004, 8).astype(np.float32)},
        {"slopes": np.linspace(0.0005, 0.004, 8).astype(np.float32), "softcap": 5.0}, {"window": 333}]


def restore_v(c, s, first, last, factor):
    """Tokens first .. last - 1 of sequence s (whole pages) stored again with their V times a factor."""
    n = last - first
    table = torch.tensor(c.slots[s][first:last:c.bs] // c.bs, dtype=torch.int32, device=DEV).view(1, -1)
    v = torch.zeros((1, n, c.H, c.D), dtype=torch.bfloat16, device=DEV)
    kvq.kvq_restore(c.pool, table, torch.tensor([n], dtype=torch.int32, device=DEV), n, None, v)
    kvq.kvq_quant_scatter(None, (v[0].float() * factor).to(torch.bfloat16), torch.tensor(c.slots[s][first:last], device=DEV), c.pool)


@pytest.mark.parametrize("zeros", [(256, 512), (0, 256), (128, 640)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("opts", range(len(OPTS)))
def test_steps_of_zero_v_count_in_the_sum(D, zeros, opts):
    c = Case([640], [40], 2, 4, D, seed=21)
    restore_v(c, 0, 0, 640, 300.0)
    restore_v(c, 0, *zeros, 0.0)
    out, st = c.run(**OPTS[opts])
    assert st == 0
    c.check(out, **OPTS[opts])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_zero_steps_of_a_split_sequence(D):
    c = Case([5008, 300], [40, 64], 2, 4, D, seed=22)
    restore_v(c, 0, 0, 5008, 300.0)
    for a in range(256, 4864, 512):
        restore_v(c, 0, a, a + 256, 0.0)
    for opts in OPTS:
        out, st = c.run(**opts)
        assert st == 0
        c.check(out, **opts)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("loud,quiet", [(60, -60), (40, -62), (-60, 60), (64, -64)])
def test_scales_far_apart(D, loud, quiet):
    c = Case([768], [40], 2, 4, D, seed=23)
    for (a, b), e in (((0, 256), loud), ((256, 512), quiet), ((512, 640), loud)):
        pages = torch.unique(torch.tensor(c.slots[0][a:b], device=DEV) // c.bs)
        c.pool.v_rscale[pages] *= 2.0 ** e
    for opts in OPTS:
        out, st = c.run(**opts)
        assert st == 0
        c.check(out, **opts)


@pytest.mark.parametrize("new", [1, 3, 40])
def test_all_v_zero(new):
    """Every V row zero (scale 2^-126): the output is zero, not NaN."""
    c = Case([320], [new], 2, 4, 128, seed=24)
    restore_v(c, 0, 0, 320, 0.0)
    out, st = c.run()
    assert st == 0 and (out[:new] == 0).all()
