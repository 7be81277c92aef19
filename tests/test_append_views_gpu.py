"""Which views kvq_append takes for q_out beside q, k and v: those that share no element with them."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
import sparse_ref as X
from kvq_testutil import DEV, bits
from quantized_kv_cache_nvfp4_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,D", [(1, 3, 64), (37, 2, 64), (20, 5, 128), (9, 1, 16)])
@pytest.mark.parametrize("order", [(0, 1, 2), (2, 0, 1)])
def test_heads_of_q_k_and_v_side_by_side(T, H, D, order):
    """A projection whose heads are (q, k, v) triples, Q turned where it stands."""
    x = synth.normal_bf16((T, H, 3, D), T, synth.STREAM_K)
    on = x.to(DEV)
    q, k, v = (on[:, :, i] for i in order)
    a, b = (kvq.KvPool.empty(64, H, D, 16, fill=0, fmt=kvq.FMT_FP8) for _ in range(2))
    cs, slots = X.angles(T, D), torch.arange(T, device=DEV)
    turn = dict(cos_sin=cs.to(DEV), positions=torch.arange(T, dtype=torch.int32, device=DEV))
    kvq.kvq_append(k.contiguous(), v.contiguous(), slots, b, **turn)
    kvq.kvq_append(k, v, slots, a, q=q, q_out=q, **turn)
    torch.cuda.synchronize()
    for one, two in zip(a._planes(), b._planes()):
        assert torch.equal(one, two)
    got = on.cpu()
    want = torch.tensor(X.turned(x[:, :, order[0]].float().numpy(), cs.numpy(), False)).to(torch.bfloat16)
    np.testing.assert_array_equal(bits(got[:, :, order[0]].contiguous()), bits(want))
    for i in order[1:]:
        assert torch.equal(got[:, :, i], x[:, :, i])


def test_refused_where_an_element_is_shared_and_only_there():
    """Random views of one buffer against the sets of their elements."""
    r = np.random.RandomState(0)
    D, size = 16, 4096
    buf = torch.zeros(size, dtype=torch.bfloat16, device=DEV)
    pools = {h: kvq.KvPool.empty(16, h, D, 16, fill=0, fmt=kvq.FMT_FP8) for h in (1, 2, 3)}
    cs = X.angles(8, D).to(DEV)

    def at(T, h, off, row, head):
        return off + (np.arange(T)[:, None, None] * row + np.arange(h)[None, :, None] * head + np.arange(D)).ravel()

    seen = {True: 0, False: 0}
    for _ in range(1500):
        T, hq, hk = r.randint(1, 5), r.randint(1, 5), r.randint(1, 4)
        row = 8 * r.randint(0, 24)
        heads = [8 * r.randint(0, 14) for _ in range(2)]
        if r.randint(2):
            heads[1] = heads[0]
        offs = 8 * r.randint(0, 40, 2)
        mine, theirs = at(T, hq, offs[0], row, heads[0]), at(T, hk, offs[1], row, heads[1])
        if len(set(mine)) < len(mine):  # q_out has one place for each of its elements
            continue
        view = lambda h, off, head: buf.as_strided((T, h, D), (row, head, 1), int(off))
        q, k = view(hq, offs[0], heads[0]), view(hk, offs[1], heads[1])
        share = bool(set(mine) & set(theirs))
        call = lambda: kvq.kvq_append(k, None, torch.arange(T, device=DEV), pools[hk], cos_sin=cs, q=q, q_out=q,
                                      positions=torch.arange(T, dtype=torch.int32, device=DEV))
        if share:
            with pytest.raises(kvq.KvqError, match="overlaps"):
                call()
        else:
            call()
        seen[share] += 1
    torch.cuda.synchronize()
    assert min(seen.values()) > 50, seen
