"""The checked build (see test_checked_access_gpu.py) where block tables have entries outside the
pool, masks leave rows without keys and stores hold infinities: no access outside the buffers."""

import os
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
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4
for D, H, bs, fk, fv in ((128, 8, 16, PG, PG), (64, 4, 16, PG, NV), (256, 4, 32, PG, PG), (256, 2, 8, F8, NV), (128, 3, 16, NV, NV)):
    L, n0 = 500, 6
    mb = L // bs + 1
    pool = kvq.KvPool.empty(2 * mb * bs, H, D, bs, fill=0xFF, fmt=fk, v_fmt=fv)
    table = synth.block_permutation(2 * mb, 1).view(2, mb).contiguous().to(dev)
    p = torch.arange(L, device=dev)
    for s in range(2):
        k, v = (synth.normal_bf16((L, H, D), 2 + s, j, device="cuda") for j in (1, 2))
        if PG in (fk, fv):
            k[3, 0, 0] = v[100, H - 1, 5] = float("inf") if s else 1.0
        kvq.kvq_quant_scatter(k, v, table[s, p // bs].long() * bs + p % bs, pool)
    for n in (1, n0, 150):
        T = 2 * n
        q = synth.normal_bf16((T, 2 * H, D), 3, 9, device="cuda")
        out = torch.empty_like(q)
        ks = torch.randint(-3, L + 9, (T,), generator=torch.Generator().manual_seed(n)).to(torch.int32).to(dev)
        for page in (0, mb // 2, (L - 1) // bs):
            for blk in (-1, 2 * mb, 2 ** 31 - 1):
                t = table.clone()
                t[0, page] = blk
                st = i32([0])
                kvq.kvq_attention(pool, t, i32([L, L]), L, q, i32([0, n, T]), n, 0.1, out, key_starts=ks, dev_status=st)
                kvq.kvq_attention(pool, t, i32([L, L]), L, q, i32([0, n, T]), n, 0.1, out, window=40, prefix_lens=i32([90, 10 ** 9]))
                if n == 1:
                    kvq.kvq_decode_attention(pool, t, i32([L, L]), L, q, 0.1, out)
torch.cuda.synchronize()
print("done")
"""


@pytest.mark.gpu
def test_gaps_and_masks_stay_inside_the_buffers():
    r = subprocess.run([sys.executable, "-c", _SCRIPT, ROOT], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-3000:]
    lines = [ln for ln in r.stderr.splitlines() if ln.startswith("[kvq checked]")]
    bad = [ln for ln in lines if "sync=no error bad=0" not in ln]
    assert len(lines) > 200 and not bad, bad[:5]
