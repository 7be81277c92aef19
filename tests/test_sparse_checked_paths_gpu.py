"""Paths of the sparse step that test_sparse_checked_gpu.py does not ask for, under the checked build: tokens that
kvq_append skips, both score kernels, sequences of very unlike lengths."""

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
for D, H, g, bs, fk, fv in ((128, 8, 4, 16, PG, NV), (64, 3, 2, 160, PG, PG), (256, 2, 8, 7, F8, PG), (128, 1, 1, 64, NV, F8)):
    for T in (1, 37, 700, 11000):
        nb = T // bs + 2
        pool = kvq.KvPool.empty(nb * bs, H, D, bs, fill=0x38, fmt=fk, v_fmt=fv)
        bounds = torch.zeros((nb, H, 2, D), dtype=torch.bfloat16, device=dev)
        k, v, q = (synth.normal_bf16((T, n, D), 2, j, device="cuda") for j, n in ((1, H), (2, H), (3, H * g)))
        slots, pos = torch.arange(T, device=dev), torch.arange(T, dtype=torch.int32, device=dev) % 300
        cs = torch.rand((300, D), device=dev)
        pos[3::11], pos[7::23], pos[40:80] = -1, 300, -5
        pos[5::29] = 2 ** 31 - 1
        slots[9::17], slots[11::19], slots[-2:] = -1, nb * bs, 2 ** 40
        kvq.kvq_append(k, v, slots, pool, cos_sin=cs, positions=pos, q=q, q_out=q, key_bounds=bounds)
        pos[:] = -1
        kvq.kvq_append(k, v, slots, pool, cos_sin=cs, positions=pos, key_bounds=bounds)
    S, new = 4, (300, 1, 9, 5)
    lens, mb = (3000, 1, 9, 2000), 3000 // bs + 1
    nb = S * mb
    table = synth.block_permutation(nb, 1).to(dev)[:S * mb].view(S, mb).int().contiguous()
    table[0, 3], table[3, 0] = -1, nb
    b = torch.rand((nb, H, 2, D), device=dev).to(torch.bfloat16)
    q = synth.normal_bf16((320, H * g, D), 2, 3, device="cuda")
    for max_q, starts in ((300, (0, 300, 301, 310, 315)), (8, (0, 8, 8, 8, 13)), (2, (0, 1, 2, 2, 4)), (9, (0, 9, 9, 9, 14))):
        for topk in (2, 10):
            kvq.kvq_select_blocks(b, table, i32(*lens), 3000, bs, q, i32(*starts), max_q,
                                  torch.full((320, H, topk), -1, dtype=torch.int32, device=dev))
torch.cuda.synchronize()
print("done")
"""

_EXPECTED = {"append_kernel", "score_kernel", "score_tile_kernel", "select_kernel"}


@pytest.mark.gpu
def test_skips_and_both_score_kernels_stay_inside_their_buffers():
    r = subprocess.run([sys.executable, "-c", _SCRIPT, ROOT], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-3000:]
    lines = [ln for ln in r.stderr.splitlines() if ln.startswith("[kvq checked]")]
    seen = {re.match(r"\[kvq checked\] (\w+):", ln).group(1) for ln in lines}
    assert _EXPECTED <= seen, sorted(_EXPECTED - seen)
    bad = [ln for ln in lines if "sync=no error bad=0" not in ln]
    assert not bad, bad[:5]
