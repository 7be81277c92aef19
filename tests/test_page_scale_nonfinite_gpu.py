"""Stores of infinities and NaN into page-scaled pools: they cost their own elements, not the
page."""

import numpy as np
import pytest
import torch

import paged_ref as R
import quantized_kv_cache_nvfp4_gb300 as kvq
from kvq_testutil import DEV, status_word
from quantized_kv_cache_nvfp4_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [16, 48, 128, 512])
@pytest.mark.parametrize("bs,first,count", [(16, 5, 1), (16, 5, 11), (16, 0, 40), (200, 3, 180), (7, 2, 30)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_they_cost_their_own_elements(D, bs, first, count, value):
    """Held rows before the call, ordinary rows beside the odd one in it: the definition's codes
    and scales with the odd elements left out, and those at the largest code (NaN: NaN)."""
    H = 3
    pool = kvq.KvPool.empty(4 * bs + 16 * bs * (bs < 16), H, D, bs, fill=0, fmt=kvq.FMT_FP8_PAGE)
    held = synth.normal_bf16((max(first, 1), H, D), 1, synth.STREAM_K)
    kvq.kvq_quant_scatter(held.to(DEV), None, torch.arange(max(first, 1), device=DEV), pool)
    want = pool.k_codes.cpu().numpy().copy(), pool.k_rscale.cpu().numpy().copy()
    x = (synth.normal_bf16((count, H, D), 2, synth.STREAM_K).float() * 3).to(torch.bfloat16)
    odd = torch.zeros(x.shape, dtype=torch.bool)
    odd[0, 1, D - 1] = odd[count // 2, 0, 3] = odd[count - 1, 2, 8:11] = True
    slots = np.arange(first, first + count)
    R.page_store(*want, torch.where(odd, 0, x).double().numpy(), slots, bs)
    code = {float("inf"): 0x7E, float("-inf"): 0xFE}.get(value, 0x7F)
    want[0][slots] = np.where(odd.numpy(), code, want[0][slots])
    st = status_word()
    kvq.kvq_quant_scatter(torch.where(odd, value, x).to(torch.bfloat16).to(DEV), None, torch.tensor(slots, device=DEV), pool, st)
    got = pool.k_codes.cpu().numpy()
    if code == 0x7F:  # either sign
        got[slots] = np.where(odd.numpy(), got[slots] & 0x7F, got[slots])
    np.testing.assert_array_equal(pool.k_rscale.cpu().numpy(), want[1])
    np.testing.assert_array_equal(got, want[0])
    assert int(st.item()) == 0


def test_a_row_of_infinities_leaves_the_page():
    pool = kvq.KvPool.empty(16, 1, 64, 16, fill=0, fmt=kvq.FMT_FP8_PAGE)
    x = synth.normal_bf16((4, 1, 64), 1, synth.STREAM_K).to(DEV)
    kvq.kvq_quant_scatter(x, x, torch.arange(4, device=DEV), pool)
    codes, scale = pool.k_codes[:4].clone(), pool.k_rscale.clone()
    kvq.kvq_quant_scatter(torch.full_like(x[:1], float("inf")), None, torch.tensor([4], device=DEV), pool)
    assert torch.equal(pool.k_codes[:4], codes) and torch.equal(pool.k_rscale, scale) and (pool.k_codes[4] == 0x7E).all()
