"""Queries whose mask hides keys with far larger V from them, beside queries that see those: each
row is as exact as its own keys allow.  The tolerance is that of test_query_attention_gpu.py,
with the largest |v| taken over the keys that the row sees."""

import numpy as np
import pytest
import torch

import paged_ref as R
import quantized_kv_cache_nvfp4_gb300 as kvq
from kvq_testutil import DEV
from test_bad_block_rows_gpu import visible
from test_query_attention_gpu import Case, decoded

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4


def scale_v(c, s, first, last, factor):
    """V of tokens first .. last - 1 (whole pages where a scale is a page's) times a power of two."""
    rows = c.slots[s][first:last]
    if (c.pool.fmt if c.pool.v_fmt is None else c.pool.v_fmt) == PG:
        rows = np.unique(rows // c.bs)
    assert rows.size == 0 or rows.max() < c.pool.v_rscale.size(0)
    c.pool.v_rscale[torch.tensor(rows, device=DEV)] *= factor


def check_rows(c, out, **opts):
    p, fv = c.pool, c.pool.fmt if c.pool.v_fmt is None else c.pool.v_fmt
    K = [decoded(p.fmt, p.k_codes, p.k_bscale, p.k_rscale, sl, c.bs) for sl in c.slots]
    V = [decoded(fv, p.v_codes, p.v_bscale, p.v_rscale, sl, c.bs) for sl in c.slots]
    ref, top = R.attention(c.q.double().numpy(), K, V, c.lens, c.starts, c.scale, **opts)
    got = out.double().cpu().numpy()
    for s, r, lo, hi in visible(c, opts):
        if lo >= hi:
            assert (got[r] == 0).all()
            continue
        vmax = np.repeat(np.abs(V[s][lo:hi]).max((0, 2)), c.group)
        d = 2.0 ** -20 * opts.get("softcap", 0.0) + 2.0 ** -21 * top[r] + 2.0 ** -22 * np.sqrt(c.D)
        bound = 2.0 ** -8 * np.abs(ref[r]) + ((2.0 ** -10 + 4 * d) * vmax)[:, None]
        err = np.abs(got[r] - ref[r])
        assert (err <= bound).all(), (s, r, lo, hi, np.nanmax(err / np.maximum(bound, 1e-300)))


LAYOUTS = [(2, 4, 128, 16), (8, 2, 64, 16), (3, 4, 128, 16), (2, 2, 128, 8), (4, 4, 256, 16), (1, 8, 128, 32)]


@pytest.mark.parametrize("H,group,D,bs", LAYOUTS)
@pytest.mark.parametrize("lens,new", [([402], [4]), ([226, 66], [60, 33]), ([2002, 130], [4, 2])])
@pytest.mark.parametrize("fmts", [(PG, None), (NV, None), (F8, NV)])
@pytest.mark.parametrize("exp", [7, 13, 40])
def test_loud_keys_of_some_rows(H, group, D, bs, lens, new, fmts, exp):
    L, n = lens[0], new[0]
    near = (L - n) // 32 * 32 - 32  # a page's start before the queries
    ks = np.zeros(sum(new) + 2, np.int64)
    ks[1:n:2] = near
    # rows in turn see everything and only the quiet end; then only the loud end and everything;
    # then loud keys that come last, behind rows that do not see them; louder and louder ones
    for loud in ([(0, near, exp)], [(near, L, exp)], [(L // 32 * 32, L, exp)],
                 [(a, a + 32, min(60, 4 * (a // 32))) for a in range(0, near, 32)]):
        c = Case(lens, new, H, group, D, bs, *fmts, seed=61)
        for a, b, e in loud:
            scale_v(c, 0, a, b, 2.0 ** e)
        for opts in ({"key_starts": ks}, {"window": 40, "softcap": 20.0},
                     {"key_starts": ks, "slopes": np.linspace(0.001, 0.3, H * group).astype(np.float32)}):
            out, st = c.run(**opts)
            assert st == 0
            check_rows(c, out, **opts)


@pytest.mark.parametrize("new", [4, 16, 90])
def test_quiet_documents_among_loud_ones(new):
    """Documents of random loudness, 32 tokens each, every row its own document."""
    for fmts in ((PG, None), (NV, None)):
        c = Case([640, 333], [new, new], 2, 1, 128, 16, *fmts, seed=62)
        rng = np.random.default_rng(new)
        for s, L in enumerate(c.lens):
            for a in range(0, L, 32):
                scale_v(c, s, a, min(a + 32, L), 2.0 ** int(rng.integers(-30, 30)))
        ks = np.concatenate([(np.arange(L - new, L) // 32) * 32 for L in c.lens] + [[0, 0]])
        for k in (ks, np.maximum(ks - 32 * rng.integers(0, 3, len(ks)), 0)):
            out, st = c.run(key_starts=k)
            assert st == 0
            check_rows(c, out, key_starts=k)
