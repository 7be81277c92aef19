"""kvq_sparse_attention against attention in 64 bits over the decoded rows of the listed blocks;
the tolerance is that of kvq_attention (sparse_ref.close)."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
import sparse_ref as X
from kvq_testutil import DEV, poison_bf16, status_word
from test_query_attention_gpu import Case as Paged, decoded

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4


def _lists(c, topk, seed=0, sort=True):
    """Random distinct blocks for each (token, head), -1 behind the last."""
    r = np.random.RandomState(seed)
    out = np.full((c.T, c.H, topk), -1, np.int32)
    for s in range(len(c.lens)):
        for i in range(c.new[s]):
            vis = (c.lens[s] - c.new[s] + i) // c.bs + 1
            for h in range(c.H):
                m = min(topk, vis)
                pick = r.permutation(vis)[:m]
                out[c.starts[s] + i, h, :m] = np.sort(pick) if sort else pick
    return out


def _run(c, lists, out=None, softcap=0.0, stream=None, lens=None, table=None, max_q=None, max_len=None, q=None, workspace=None):
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)
    st = status_word()
    out = poison_bf16(tuple(c.q.shape)) if out is None else out
    kvq.kvq_sparse_attention(c.pool, (c.table if table is None else table).to(DEV), i32(c.lens if lens is None else lens),
                             max_len or max(c.lens), c.q.to(DEV) if q is None else q, i32(c.starts), max_q or max(c.new),
                             i32(lists), c.scale, out, softcap=softcap, workspace=workspace, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    return out, int(st.item())


def _check(c, lists, out, softcap=0.0, rows=None):
    p = c.pool
    K = [decoded(p.fmt, p.k_codes, p.k_bscale, p.k_rscale, sl, c.bs) for sl in c.slots]
    V = [decoded(p.fmt if p.v_fmt is None else p.v_fmt, p.v_codes, p.v_bscale, p.v_rscale, sl, c.bs) for sl in c.slots]
    ref, top, vmax = X.sparse_attention(c.q.double().numpy(), K, V, c.lens, c.starts, lists, c.bs, c.scale, softcap)
    rows = np.arange(c.starts[-1]) if rows is None else rows
    X.close(out.double().cpu().numpy()[rows], ref[rows], top[rows], vmax[rows], c.D, softcap)
    return ref


@pytest.mark.parametrize("lens,new", [([1, 17, 300], [1, 1, 1]), ([40, 5, 333, 64], [4, 5, 1, 3]), ([130, 0, 257], [60, 0, 31])])
@pytest.mark.parametrize("H,group,D", [(2, 4, 128), (1, 8, 64), (3, 7, 64), (2, 1, 256), (1, 16, 128), (1, 12, 256)])
def test_shapes(lens, new, H, group, D):
    c = Paged(lens, new, H, group, D, seed=D + group)
    for topk in (1, 6):
        lists = _lists(c, topk, seed=topk)
        out, st = _run(c, lists)
        assert st == 0 and c.untouched(out, slice(c.starts[-1], c.T))
        _check(c, lists, out)


@pytest.mark.parametrize("fmt_k,fmt_v", [(NV, NV), (F8, F8), (PG, NV), (NV, PG), (F8, PG), (PG, PG)])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 8), (128, 33), (256, 16), (64, 1), (128, 64), (256, 3)])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_formats(fmt_k, fmt_v, D, bs, softcap):
    c = Paged([170, 260], [2, 5], 2, 4, D, bs, fmt_k, fmt_v, seed=bs)
    if softcap:
        c.q = (c.q.float() * 4).to(torch.bfloat16)  # logits that the cap bends
    lists = _lists(c, max(3, 70 // bs))
    out, st = _run(c, lists, softcap=softcap)
    assert st == 0
    _check(c, lists, out, softcap)


@pytest.mark.parametrize("topk,bs", [(40, 64), (300, 16), (1000, 4), (10, 64), (25, 32), (50, 16), (75, 7)])
@pytest.mark.parametrize("fmt", [PG, NV])
@pytest.mark.parametrize("group,D", [(4, 128), (11, 256), (16, 64)])
def test_long_lists_in_splits(topk, bs, fmt, group, D):
    """Few rows with long lists: the list is split over thread blocks and joined again, up to 8 splits
    in a cluster, more through the workspace."""
    c = Paged([5000, 700], [1, 2], 2, group, D, bs, fmt, seed=topk)
    assert (kvq.kvq_sparse_attention_workspace(c.T, 2, 2 * group, D, bs, topk) > 0) == (topk * bs > 1024 or D == 256)
    lists = _lists(c, topk)
    out, st = _run(c, lists)
    assert st == 0 and c.untouched(out, slice(c.starts[-1], c.T))
    _check(c, lists, out)


@pytest.mark.parametrize("D,bs", [(128, 16), (64, 8), (256, 32)])
def test_all_blocks_is_plain_attention(D, bs):
    c = Paged([300, 190], [3, 40], 2, 4, D, bs, seed=4)
    lists = np.full((c.T, 2, 40), -1, np.int32)
    lists[:] = np.arange(40)  # those behind a query count for nothing
    out, st = _run(c, lists)
    assert st == 0
    _check(c, lists, out)
    c.check(out)


def test_lists_of_any_order_repeats_and_gaps():
    """Unsorted lists, entries in the middle that count for nothing, blocks that stand there twice."""
    c = Paged([700, 333], [3, 1], 2, 4, 128, 16, seed=6)
    lists = _lists(c, 30, sort=False)
    lists[:, :, 4] = -5
    lists[:, :, 9] = 10 ** 9
    lists[:, :, 10] = 2 ** 31 - 1
    lists[:, :, 11] = lists[:, :, 12]
    lists[:, 1, 13:20] = lists[:, 1, 3:4]
    lists[:, :, 29] = 60  # behind the queries
    out, st = _run(c, lists)
    assert st == 0
    _check(c, lists, out)


def test_rows_that_see_nothing_are_zero():
    c = Paged([700, 333, 40], [2, 1, 1], 2, 4, 64, 16, seed=7)
    lists = _lists(c, 8)
    lists[0, 0] = -1
    lists[1] = 10 ** 6
    lists[3, 1] = 30  # behind the query
    for topk in (8, 300):  # one thread block a row, and splits
        wide = np.full((c.T, 2, topk), -1, np.int32)
        wide[:, :, topk - 8:] = lists
        out, st = _run(c, wide)
        assert st == 0
        _check(c, wide, out)
        assert (out[0, :4] == 0).all() and (out[1] == 0).all() and (out[3, 4:] == 0).all()


@pytest.mark.parametrize("fmt", [PG, F8, NV])
@pytest.mark.parametrize("bs", [16, 8])
def test_other_blocks_are_not_read(fmt, bs):
    """Rows of blocks that no list names hold NaN codes and scales."""
    c = Paged([400, 200], [1, 2], 2, 4, 128, bs, fmt, seed=8)
    lists = _lists(c, 5)
    named = set()
    for s in range(2):
        for b in np.unique(lists[c.starts[s]:c.starts[s + 1]]):
            if b >= 0:
                named.add(int(c.table[s, b]))
    want, _ = _run(c, lists)
    _check(c, lists, want)
    for blk in range(c.pool.num_slots // bs):
        if blk in named:
            continue
        sl = slice(blk * bs, (blk + 1) * bs)
        for t in (c.pool.k_codes, c.pool.v_codes, c.pool.k_bscale, c.pool.v_bscale):
            if t is not None:
                t[sl] = 0xFF
        for t in (c.pool.k_rscale, c.pool.v_rscale):
            t[blk if fmt == PG else sl] = float("nan")
    out, st = _run(c, lists)
    assert st == 0 and torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("topk", [6, 200])
def test_bad_table_entries_keep_their_rows_only(topk):
    c = Paged([700, 300], [2, 1], 2, 4, 128, 16, seed=9)
    lists = np.full((c.T, 2, topk), -1, np.int32)
    lists[:, :, :6] = np.array([0, 1, 3, 7, 9, 11])
    lists[1, 0, 2], lists[0, 1, 3] = 5, 20
    want, _ = _run(c, lists)
    _check(c, lists, want)
    table = c.table.clone()
    table[0, 5], table[0, 20], table[0, 21] = -1, c.pool.num_slots // 16, -9
    out, st = _run(c, lists, table=table)
    assert st == kvq.DEV_BAD_BLOCK
    kept = torch.zeros(c.T, 8, dtype=torch.bool)
    kept[1, :4], kept[0, 4:], kept[c.starts[-1]:] = True, True, True
    held = (out.cpu().contiguous().view(torch.int16) == -23131).all(-1)  # 0xA5A5
    assert torch.equal(held, kept)
    live = (~kept).nonzero()
    assert torch.equal(out.cpu()[live[:, 0], live[:, 1]], want.cpu()[live[:, 0], live[:, 1]])


def test_refused_sequences():
    c = Paged([700, 300, 90], [2, 1, 1], 2, 4, 128, 16, seed=10)
    lists = _lists(c, 6)
    want, _ = _run(c, lists)
    for kw, bad in ((dict(lens=[700, -1, 90]), 1), (dict(lens=[701, 300, 90]), 0), (dict(max_q=1), 0)):
        out, st = _run(c, lists, max_len=700, **kw)
        assert st == kvq.DEV_BAD_SEQLEN
        rows = slice(c.starts[bad], c.starts[bad + 1])
        assert c.untouched(out, rows)
        ok = [r for r in range(c.starts[-1]) if not rows.start <= r < rows.stop]
        assert torch.equal(out[ok], want[ok])


def test_nan_scores_reach_their_own_output():
    c = Paged([700], [3], 2, 4, 128, 16, seed=11)
    c.q[1, 2, 5] = float("nan")
    lists = _lists(c, 6)
    out, st = _run(c, lists)
    nan = torch.isnan(out[:3]).any(-1).cpu()
    assert st == 0 and nan[1, 2] and nan.sum() == 1


@pytest.mark.parametrize("topk", [50, 300])  # splits that merge in a cluster, and through the workspace
def test_views_graphs_and_streams(topk):
    c = Paged([5000, 700], [1, 2], 2, 4, 128, 16, seed=12)
    lists = _lists(c, topk)
    want, _ = _run(c, lists)
    _check(c, lists, want)
    wide = torch.zeros((c.T, 20, 128), dtype=torch.bfloat16, device=DEV)
    wide[:, 5:13] = c.q.to(DEV)
    got, _ = _run(c, lists, q=wide[:, 5:13])
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)
    table, lens, starts, q, sel = c.table.to(DEV), i32(c.lens), i32(c.starts), c.q.to(DEV), i32(lists)
    size = kvq.kvq_sparse_attention_workspace(c.T, 2, 8, 128, 16, topk)
    assert (size > 0) == (topk > 64)
    outs, graphs = [poison_bf16(tuple(c.q.shape)) for _ in range(2)], []
    for o in outs:
        ws = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvq.kvq_sparse_attention(c.pool, table, lens, 5000, q, starts, 2, sel, c.scale, o, workspace=ws)
        graphs.append((g, ws))
    for g, _ in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = _run(c, lists, stream=side)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
