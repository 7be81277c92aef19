"""kvq_append with tokens that their position keeps out in the middle of a block: the block's other rows
make one run, as if the skipped tokens were not in the call.  Bit for bit (see test_append_gpu.py)."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
import sparse_ref as X
from kvq_testutil import DEV, bits, poison_bf16, status_word
from test_append_gpu import Cache, _rows, _same_pool

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4


def _append(c, k, v, slots, pos, cs, q=None):
    """The call on all tokens, the definition on those whose position has angles."""
    slots, pos = np.asarray(slots, np.int64), np.asarray(pos, np.int32)
    st, q_out = status_word(), None if q is None else poison_bf16(tuple(q.shape))
    kvq.kvq_append(k.to(DEV), v.to(DEV), torch.tensor(slots, device=DEV), c.pool, cos_sin=cs.to(DEV),
                   positions=torch.tensor(pos, device=DEV), q=None if q is None else q.to(DEV), q_out=q_out,
                   key_bounds=c.bounds, dev_status=st)
    torch.cuda.synchronize()
    live = (pos >= 0) & (pos < cs.size(0))
    rows = cs.numpy()[pos[live]]
    f = lambda t: t.float().numpy()[live]
    if live.any():
        X.append(c.want, c.fmts, c.bs, f(k), f(v), slots[live], c.wb, rows)
    _same_pool(c.pool, c.want)
    np.testing.assert_array_equal(c.bounds.float().cpu().numpy(), c.wb, err_msg="bounds")
    if q is not None:
        got, turn = q_out.cpu(), torch.tensor(X.turned(f(q), rows, False)).to(torch.bfloat16)
        np.testing.assert_array_equal(bits(got)[live], bits(turn))
        assert (got.contiguous().view(torch.uint8).numpy()[~live] == 0xA5).all()
    return int(st.item())


@pytest.mark.parametrize("fk,fv", [(PG, PG), (F8, NV), (NV, PG), (PG, F8)])
@pytest.mark.parametrize("out", [(5,), (0,), (15,), (0, 1, 2), (7, 8, 9, 10, 11, 12, 13, 14, 15), tuple(range(1, 16, 2)),
                                 tuple(range(15)), tuple(range(16))])
def test_positions_skipped_inside_a_page(fk, fv, out):
    """A page of 16 begun, with some of its tokens skipped; then the same page continued, with others."""
    H, D, bs = 4, 128, 16
    c = Cache(4, H, D, bs, fk, fv, fill=0x38)
    for t in (c.pool.k_rscale, c.pool.v_rscale):
        t.fill_(2.0 ** -6)
    c.want = tuple(tuple(None if t is None else t.cpu().numpy().copy() for t in p) for p in (
        (c.pool.k_codes, c.pool.k_bscale, c.pool.k_rscale), (c.pool.v_codes, c.pool.v_bscale, c.pool.v_rscale)))
    cs = X.angles(40, D)
    pos = np.arange(16, dtype=np.int32)
    pos[list(out)] = -1
    k, v = _rows(16, H, D, 1), _rows(16, H, D, 2, 3.0)
    k[list(out)] *= 64  # what is skipped is the largest: neither scales nor bounds may see it
    v[list(out)] *= 64
    assert _append(c, k, v, np.arange(32, 48), pos, cs, _rows(16, 7, D, 3)) == 0
    # rows 1, 3, .. of the page alone: not its first slot
    slots, pos = np.arange(33, 48), np.arange(1, 16, dtype=np.int32)
    pos[1::2] = 40  # past the angles
    assert _append(c, _rows(15, H, D, 4, 5.0), _rows(15, H, D, 5), slots, pos, cs) == kvq.DEV_BAD_POS


@pytest.mark.parametrize("D", [64, 256, 96])
@pytest.mark.parametrize("fk,fv", [(PG, PG), (NV, F8)])
@pytest.mark.parametrize("lead,gap", [(0, 40), (40, 1), (70, 3), (31, 33), (33, 64), (0, 159), (32, 0)])
def test_long_pages(D, fk, fv, lead, gap):
    """Pages longer than a warp's stage and than a chunk of tokens, whose first `lead` tokens and every other
    `gap` are skipped."""
    H, bs, T = 2, 160, 200
    c = Cache(4, H, D, bs, fk, fv)
    cs = X.angles(300, D)
    for i, (at, f) in enumerate(((0, 1.0), (200, 4.0))):
        pos = np.arange(at, at + T, dtype=np.int32) % 300
        pos[:lead] = -1
        if gap:
            pos[lead + 2:lead + 2 + gap] = -1
        assert _append(c, _rows(T, H, D, i, f), _rows(T, H, D, 7 + i, f), np.arange(at, at + T), pos, cs) == 0


@pytest.mark.parametrize("fk,fv,bs", [(PG, PG, 16), (NV, PG, 64), (F8, F8, 5)])
@pytest.mark.parametrize("T", [130, 3000, 11000, 21000])
def test_any_skips(T, fk, fv, bs):
    """Three tokens of ten skipped, in runs of several lengths, whole pages among them, over every chunk length;
    padding that names a stored page's slot behind the last."""
    H, D = 2, 64
    r = np.random.RandomState(T + bs)
    nb = T // bs + 1
    c = Cache(nb + 1, H, D, bs, fk, fv)
    table = r.permutation(nb)
    p = np.arange(T)
    slots, pos = table[p // bs].astype(np.int64) * bs + p % bs, (p % 500).astype(np.int32)
    for at in r.randint(0, T, T // 20):
        pos[at:at + r.choice([1, 1, 2, 5, 40])] = r.choice([-1, -7])
    slots[-6:], pos[-6:] = slots[0], -1
    assert _append(c, _rows(T, H, D, 1), _rows(T, H, D, 2), slots, pos, X.angles(500, D)) == 0
