"""A workspace of kvq_sparse_attention or kvq_select_blocks sized for the largest step serves smaller ones."""

import numpy as np
import pytest
import torch

from kvq_testutil import DEV


@pytest.mark.parametrize("H,group,D", [(8, 4, 128), (1, 16, 64), (3, 7, 128), (8, 1, 256), (128, 1, 64)])
@pytest.mark.parametrize("topk,bs", [(512, 16), (4096, 1), (64, 16), (65, 16), (40, 64), (3, 1000), (8, 32)])
def test_more_tokens_and_longer_lists_never_need_less(kvq_lib_path, H, group, D, topk, bs):
    import quantized_kv_cache_nvfp4_gb300 as kvq

    size = lambda T, k: kvq.kvq_sparse_attention_workspace(T, H, H * group, D, bs, k)
    by_tokens = [size(T, topk) for T in [*range(1, 1300), 5000, 100000, 2 ** 30 // (H * group)]]
    assert by_tokens == sorted(by_tokens)
    for T in (1, 4, 100, 2000):
        by_topk = [size(T, k) for k in range(1, topk + 1, max(1, topk // 50))]
        assert by_topk == sorted(by_topk)
    select = [kvq.kvq_select_blocks_workspace(T, H, n, bs) for T, n in ((1, 1), (1, 50), (2, 50), (2, 5000), (300, 5000))]
    assert select == sorted(select)


@pytest.mark.gpu
@pytest.mark.parametrize("D,most", [(128, 100), (256, 100), (64, 1)])
def test_smaller_steps_in_the_largest_steps_workspace(D, most):
    import quantized_kv_cache_nvfp4_gb300 as kvq
    from test_query_attention_gpu import Case as Paged
    from test_sparse_attention_gpu import _check, _lists, _run

    H, group, bs, topk = 8, 2, 16, 512
    size = kvq.kvq_sparse_attention_workspace(most, H, H * group, D, bs, topk)
    room = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    for T in (1, 3, 9, 40, 75, 76, 100):
        if T > most:
            continue
        lens = [3000, 150, 9000, 20][:T]
        new = [1] * len(lens)
        new[0] = T - len(lens) + 1
        c = Paged(lens, new, H, group, D, bs, kvq.FMT_FP8_PAGE, seed=T, spare=0)
        lists = _lists(c, topk)
        out, st = _run(c, lists, workspace=room[:size])
        assert st == 0 and (room[size:] == 0xA5).all()
        rows = np.unique(np.linspace(0, T - 1, 6).astype(int))
        _check(c, lists, out, rows=rows)


def test_the_bound_covers_what_each_call_uses(kvq_lib_path):
    from quantized_kv_cache_nvfp4_gb300 import _abi

    lib = _abi.load()
    falls = 0
    for H, Hq, D, bs, topk in ((8, 32, 128, 16, 512), (8, 16, 256, 16, 64), (1, 16, 64, 1, 4096), (5, 35, 128, 33, 77)):
        exact = [lib.kvq_sparse_attention_workspace_exact(T, H, Hq, D, bs, topk) for T in range(1, 1500)]
        bound = [lib.kvq_sparse_attention_workspace(T, H, Hq, D, bs, topk) for T in range(1, 1500)]
        assert all(e <= b for e, b in zip(exact, bound)) and bound == sorted(bound)
        falls += exact != sorted(exact)
    assert falls > 0  # why the bound is asked for, and not the largest step's own use
    assert lib.kvq_sparse_attention_workspace_exact(0, 2, 8, 128, 16, 4) == 0
    assert lib.kvq_sparse_attention_workspace_exact(8, 2, 1, 128, 16, 4) == 0
