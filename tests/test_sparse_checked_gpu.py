"""The sparse step's kernels under the checked build (see test_checked_access_gpu.py)."""

import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_SCRIPT = r"""
import sys, torch
sys.path.insert(0, sys.argv[1])
from quantized_kv_cache_nvfp4_gb300 import _abi, build
_abi.load(build.build(checked=True))
import quantized_kv_cache_nvfp4_gb300 as kvq
from quantized_kv_cache_nvfp4_gb300 import synth

dev = torch.device("cuda", 0)
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4
for D, H, g, bs, fk, fv, rot, pairs in ((128, 8, 4, 16, PG, PG, 128, False), (64, 4, 16, 16, PG, NV, 32, True),
                                        (256, 2, 9, 3, F8, NV, 96, False), (128, 3, 2, 1, NV, NV, 112, False),
                                        (64, 1, 1, 64, F8, F8, 64, True)):
    S, new = 3, (300, 17, 1)
    mb, T = 300 // bs + 2, 323
    nb = S * mb
    table = torch.zeros((S, mb), dtype=torch.int32, device=dev)
    lens, starts, used = i32(0, 0, 0), i32(0, 0, 0, 0), i32(0)
    slots, pos = torch.zeros(T, dtype=torch.int64, device=dev), torch.zeros(T, dtype=torch.int32, device=dev)
    pool = kvq.KvPool.empty(nb * bs, H, D, bs, fill=0xFF, fmt=fk, v_fmt=fv)
    bounds = torch.zeros((nb, H, 2, D), dtype=torch.bfloat16, device=dev)
    kvq.kvq_plan_pages(i32(0, 0, 0), i32(*new), synth.block_permutation(nb, 1).to(dev), bs, table, lens, starts, slots, pos, used)
    k, v, q = (synth.normal_bf16((T, n, D), 2, j, device="cuda") for j, n in ((1, H), (2, H), (3, H * g)))
    cs = torch.rand((301, rot), device=dev)
    kvq.kvq_append(k, v, slots, pool, cos_sin=cs, positions=pos, interleaved=pairs, q=q, q_out=q, key_bounds=bounds)
    kvq.kvq_append(k[:5], v[:5], slots[:5], pool, key_bounds=bounds)
    for topk in (1, 7, 500):
        sel = torch.full((T, H, topk), -1, dtype=torch.int32, device=dev)
        for b in (bounds, torch.ones_like(bounds)):  # and all scores again in 64 bits
            kvq.kvq_select_blocks(b, table, lens, 300, bs, q, starts, 300, sel, first_blocks=1, last_blocks=0)
        kvq.kvq_sparse_attention(pool, table, lens, 300, q, starts, 300, sel, 0.1, torch.empty_like(q), softcap=20.0)
        one, st = q[:S].contiguous(), i32(0, 1, 2, 3)
        kvq.kvq_select_blocks(bounds, table, lens, 300, bs, one, st, 1, sel[:S].contiguous(), last_blocks=0)
        kvq.kvq_sparse_attention(pool, table, lens, 300, one, st, 1, sel[:S].contiguous(), 0.1, torch.empty_like(one))
torch.cuda.synchronize()
print("done")
"""

_EXPECTED = {"append_kernel", "score_kernel", "select_kernel", "sparse_rows_kernel", "query_merge_kernel"}


@pytest.mark.gpu
def test_sparse_kernels_stay_inside_their_registered_buffers():
    r = subprocess.run([sys.executable, "-c", _SCRIPT, ROOT], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-3000:]
    lines = [ln for ln in r.stderr.splitlines() if ln.startswith("[kvq checked]")]
    seen = {re.match(r"\[kvq checked\] (\w+):", ln).group(1) for ln in lines}
    assert _EXPECTED <= seen, sorted(_EXPECTED - seen)
    bad = [ln for ln in lines if "sync=no error bad=0" not in ln]
    assert not bad, bad[:5]
