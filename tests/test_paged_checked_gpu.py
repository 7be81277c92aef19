"""The paged operators' kernels under the checked build (see test_checked_access_gpu.py): one
small call of each kernel in a child process; every launch must report a clean sync and no
access outside the buffers registered for it."""

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
for D, H, bs, fk, fv in ((128, 8, 16, PG, PG), (64, 4, 16, PG, NV), (256, 4, 32, PG, PG), (256, 2, 8, F8, NV),
                         (128, 3, 16, NV, NV), (64, 1, 16, F8, F8)):
    S, mb, T = 3, 300 // bs + 2, 700
    table = torch.zeros((S, mb), dtype=torch.int32, device=dev)
    lens, starts, used = i32(0, 0, 0), i32(0, 0, 0, 0), i32(0)
    slots, pos = torch.zeros(T, dtype=torch.int64, device=dev), torch.zeros(T, dtype=torch.int32, device=dev)
    nb = S * mb
    free = synth.block_permutation(nb, 1).to(dev)
    pool = kvq.KvPool.empty(nb * bs, H, D, bs, fill=0xFF, fmt=fk, v_fmt=fv)
    new = (300, 17, 1)
    kvq.kvq_plan_pages(i32(0, 0, 0), i32(*new), free, bs, table, lens, starts, slots, pos, used)
    k, v = (synth.normal_bf16((T, H, D), 2, j, device="cuda") for j in (1, 2))
    kvq.kvq_quant_scatter(k, v, slots, pool)
    ko, vo = (torch.empty((S, 300, H, D), dtype=torch.bfloat16, device=dev) for _ in range(2))
    kvq.kvq_restore(pool, table, lens, 300, ko, vo)
    q = synth.normal_bf16((T, 2 * H, D), 3, 9, device="cuda")
    kvq.kvq_decode_attention(pool, table, lens, 300, q[:S], 0.1, torch.empty_like(q[:S]))
    slopes = torch.full((2 * H,), 0.1, device=dev)
    for st, n in ((starts, 300), (i32(0, 1, 2, 3), 1), (i32(0, 6, 12, 13), 6)):
        out = torch.empty_like(q)
        kvq.kvq_attention(pool, table, lens, 300, q, st, n, 0.1, out)
        kvq.kvq_attention(pool, table, lens, 300, q, st, n, 0.1, out, softcap=20.0, alibi_slopes=slopes, window=100,
                          prefix_lens=lens, key_starts=torch.zeros(T, dtype=torch.int32, device=dev))
torch.cuda.synchronize()
print("done")
"""

_EXPECTED = {"plan_pages_kernel", "page_encode_kernel", "query_rows_kernel", "query_page_kernel", "query_tile_kernel",
             "query_merge_kernel", "decode_attn_page_kernel", "decode_attn_kernel", "nvfp4_decode_kernel"}


@pytest.mark.gpu
def test_paged_kernels_stay_inside_their_registered_buffers():
    r = subprocess.run([sys.executable, "-c", _SCRIPT, ROOT], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-3000:]
    lines = [ln for ln in r.stderr.splitlines() if ln.startswith("[kvq checked]")]
    seen = {re.match(r"\[kvq checked\] (\w+):", ln).group(1) for ln in lines}
    assert _EXPECTED <= seen, sorted(_EXPECTED - seen)
    bad = [ln for ln in lines if "sync=no error bad=0" not in ln]
    assert not bad, bad[:5]
