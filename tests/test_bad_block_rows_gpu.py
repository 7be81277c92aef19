"""Block entries outside the pool among the keys of some query rows only: those rows keep what
they held, the others are whole."""

import numpy as np
import pytest
import torch

import paged_ref as R
import quantized_kv_cache_nvfp4_gb300 as kvq
from kvq_testutil import DEV
from test_query_attention_gpu import Case, decoded

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4


def visible(c, opts):
    """(sequence, row, lo, hi) of every query row."""
    for s, (n, L) in enumerate(zip(c.new, c.lens)):
        for i in range(n):
            r, p = int(c.starts[s]) + i, L - n + i
            lo = max(0, p + 1 - opts["window"] if opts.get("window") else 0, opts["key_starts"][r] if "key_starts" in opts else 0)
            yield s, r, lo, max(p + 1, min(opts["prefix"][s], L) if "prefix" in opts else 0)


@pytest.mark.parametrize("H,group,bs", [(2, 4, 16), (8, 2, 16), (3, 4, 16), (2, 4, 8), (1, 4, 64)])
@pytest.mark.parametrize("lens,new", [([300, 90], [4, 3]), ([300, 90], [60, 33]), ([5000, 90], [4, 3]), ([3000, 90], [150, 33])])
@pytest.mark.parametrize("fmts", [(PG, PG), (NV, NV), (F8, NV)])
def test_only_rows_that_need_the_entry_keep_theirs(H, group, bs, lens, new, fmts):
    c = Case(lens, new, H, group, 128, bs, *fmts, seed=51)
    rng = np.random.default_rng(bs + H)
    near = np.concatenate([rng.integers(max(0, L - n - 40), L + 2, n) for L, n in zip(lens, new)] + [[0, 0]])
    far = np.where(rng.random(c.T) < 0.5, rng.integers(0, lens[0] - new[0], c.T), near)
    for opts in ({"key_starts": near}, {"key_starts": far}, {"window": 20}, {"key_starts": near, "prefix": [lens[0], 30]}):
        K = [decoded(fmts[0], c.pool.k_codes, c.pool.k_bscale, c.pool.k_rscale, sl, bs) for sl in c.slots]
        V = [decoded(fmts[1], c.pool.v_codes, c.pool.v_bscale, c.pool.v_rscale, sl, bs) for sl in c.slots]
        ref, top = R.attention(c.q.double().numpy(), K, V, c.lens, c.starts, c.scale, **opts)
        for page in (lens[0] - new[0] // 2) // bs, (lens[0] - new[0] - 10) // bs, (lens[0] - 1) // bs:
            for blk in (-1, 10 ** 6):
                t = c.table.clone()
                t[0, page] = blk
                out, st = c.run(table=t, **opts)
                got, kept, whole = out.double().cpu().numpy(), 0, 0
                for s, r, lo, hi in visible(c, opts):
                    if s == 0 and lo < hi and lo < (page + 1) * bs and hi > page * bs:
                        assert c.untouched(out, slice(r, r + 1)), (r, lo, hi)
                        kept += 1
                        continue
                    vmax = np.repeat(np.abs(V[s]).max((0, 2)), group)
                    d = 2.0 ** -21 * top[r] + 2.0 ** -22 * np.sqrt(128)
                    bound = 2.0 ** -8 * np.abs(ref[r]) + ((2.0 ** -10 + 4 * d) * vmax)[:, None]
                    assert (np.abs(got[r] - ref[r]) <= bound).all(), (s, r, lo, hi)
                    whole += 1
                assert whole and (st == kvq.DEV_BAD_BLOCK or kept == 0)
                assert c.untouched(out, slice(c.starts[-1], c.T))


@pytest.mark.parametrize("new", [1, 4, 60])
def test_rubbish_in_the_pool_stays_out(new):
    """What a skipped entry's place holds (a ring stage's former rows, block 0) is NaN here."""
    for fmt in (PG, NV):
        c = Case([700], [new], 2, 4, 128, 16, fmt, seed=52)
        ks = np.full(c.T, 700 - new)
        want, _ = c.run(key_starts=ks)
        t = c.table.clone()
        t[0, 0:40] = -5
        out, st = c.run(table=t, key_starts=ks)
        assert st == 0 and torch.equal(out[:new], want[:new])
        ks[:new:2] = 0  # rows that need them beside rows that do not
        out, st = c.run(table=t, key_starts=ks)
        assert st == kvq.DEV_BAD_BLOCK and c.untouched(out, slice(0, 1)) and torch.isfinite(out[1:new:2]).all()
        if new > 1:
            assert (out[1:new:2].float() - want[1:new:2].float()).abs().max() <= 2.0 ** -6 * want[:new].float().abs().max()


@pytest.mark.parametrize("bs,H,new", [(1, 2, 1), (1, 2, 60), (16, 2, 3)])
def test_a_bad_entry_at_the_end_of_a_long_table(bs, H, new):
    """Half a million tokens of one page over and over, the last entry bad: the rows' walk over
    their entries is a warp's and ends soon."""
    L, D = 1 << 19, 64
    pool = kvq.KvPool.empty(4 * bs, H, D, bs, fill=0, fmt=F8)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    table = torch.zeros((1, L // bs), dtype=torch.int32, device=DEV)
    table[0, -1] = -1
    q = torch.ones((new, H * 2, D), dtype=torch.bfloat16, device=DEV)
    out, st = torch.full_like(q, 7.0), i32([0])
    ks = i32([0] * new)
    ks[0] = L  # sees nothing
    kvq.kvq_attention(pool, table, i32([L]), L, q, i32([0, new]), new, 0.1, out, key_starts=ks, dev_status=st)
    torch.cuda.synchronize()
    assert (out[0] == 0).all()
    need = torch.arange(L - new, L, device=DEV) >= (L // bs - 1) * bs
    need[0] = False
    want = torch.where(need, 7.0, 0.0)
    assert (out[:, 0, 0].float() == want).all() and int(st.item()) == (kvq.DEV_BAD_BLOCK if new > 1 else 0)
