"""The sparse step in the last blocks of a pool whose planes and bounds are longer than 2^32 bytes: the same
bits as in a small pool."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
import sparse_ref as X
from kvq_testutil import DEV, status_word
from quantized_kv_cache_nvfp4_gb300 import synth

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4


@pytest.mark.parametrize("fk,fv", [(PG, F8), (NV, PG)])
def test_far_blocks(fk, fv):
    H, g, D, bs, T, mb = 8, 2, 256, 4, 70, 40
    Hq, far = H * g, 2 ** 20 + 7  # blocks: codes of 8 bits 2^33 bytes, bounds 2^33
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)
    qkv = synth.normal_bf16((2 * T, Hq + 2 * H, D), 1, 3).to(DEV)
    cs, got = X.angles(2 * T, D).to(DEV), []
    for nb in (mb, far):
        pool = kvq.KvPool.empty(nb * bs, H, D, bs, fmt=fk, v_fmt=fv)
        bounds = torch.empty((nb, H, 2, D), dtype=torch.bfloat16, device=DEV)
        last = torch.arange(nb - mb, nb, device=DEV)
        for t in pool._planes():  # what the step may read or raise, as if the pool were new
            if t is not None and t.numel():
                t.view(nb, -1)[nb - mb:].zero_()
        bounds[nb - mb:] = 0
        table = last.flip(0).to(torch.int32).view(1, mb).contiguous()
        st, sel, out = status_word(), i32(np.full((T, H, 6), -1)), torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV)
        for at in (0, T):  # a prompt, then the chunk that asks
            p = torch.arange(at, at + T, device=DEV)
            x = qkv[at:at + T].clone()
            slots = table[0].long()[p // bs] * bs + p % bs
            kvq.kvq_append(x[:, Hq:Hq + H], x[:, Hq + H:], slots, pool, cos_sin=cs, positions=p.to(torch.int32), q=x[:, :Hq],
                           q_out=x[:, :Hq], key_bounds=bounds, dev_status=st)
        for n in (T, 2):  # tiles, then single queries
            lens, starts = i32([2 * T]), i32([0, n])
            kvq.kvq_select_blocks(bounds, table, lens, mb * bs, bs, x[T - n:, :Hq], starts, n, sel[:n], dev_status=st)
            kvq.kvq_sparse_attention(pool, table, lens, mb * bs, x[T - n:, :Hq], starts, n, sel[:n], D ** -0.5, out[:n], dev_status=st)
            got.append((sel.clone(), out.clone()))
        assert int(st.item()) == 0
        got[-1] += (bounds[nb - mb:].clone(), *(t.view(nb, -1)[nb - mb:].clone() for t in pool._planes() if t is not None and t.numel()))
        del pool, bounds
        torch.cuda.empty_cache()
    for a, b in ((got[0], got[2]), (got[1], got[3])):
        for x, y in zip(a, b):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
    assert (got[0][0] >= 0).all() and got[0][1].abs().amax() > 0
