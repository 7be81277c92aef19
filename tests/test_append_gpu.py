"""kvq_append against its definition: codes, scales, turned queries and bounds, bit for bit.

Every step of the definition is one binary32 operation rounded once (the products and sums of
the rotation, the codecs' divisions), which numpy's float32 does the same way, so no
tolerance is needed.  Bounds are compared as values: a zero's sign is not specified."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
import sparse_ref as X
from quantized_kv_cache_nvfp4_gb300 import synth
from kvq_testutil import DEV, bits, poison_bf16, status_word

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4


def _rows(T, H, D, seed, factor=1.0):
    return (synth.normal_bf16((T, H, D), seed, synth.STREAM_K, 0.01, 20.0).float() * factor).to(torch.bfloat16)


def _host(pool):
    n = lambda t: None if t is None else t.cpu().numpy().copy()
    return ((n(pool.k_codes), n(pool.k_bscale), n(pool.k_rscale)), (n(pool.v_codes), n(pool.v_bscale), n(pool.v_rscale)))


def _same_pool(pool, want):
    for got, ref, name in zip(_host(pool), want, "kv"):
        for a, b, part in zip(got, ref, ("codes", "block scales", "scales")):
            if a is not None:
                np.testing.assert_array_equal(a.view(np.uint8), b.view(np.uint8), err_msg=f"{name} {part}")


class Cache:
    """A pool with its bounds on the GPU, and the definition's copy of both on the host."""

    def __init__(self, nb, H, D, bs, fk, fv=None, fill=0xFF):
        self.pool = kvq.KvPool.empty(nb * bs, H, D, bs, fill=fill, fmt=fk, v_fmt=fv)
        self.bounds = torch.full((nb, H, 2, D), 7.0, dtype=torch.bfloat16, device=DEV)
        self.want, self.wb = _host(self.pool), self.bounds.float().cpu().numpy()
        self.fmts, self.bs = (fk, fk if fv is None else fv), bs

    def append(self, k, v, slots, pos=None, cs=None, pairs=False, q=None, skip=None, stream=None):
        """The call and the definition; skip: tokens that the call has to leave out."""
        st = status_word()
        d = lambda t: None if t is None else t.to(DEV)
        q_out = None if q is None else poison_bf16(tuple(q.shape))
        kvq.kvq_append(d(k), d(v), torch.tensor(slots, device=DEV), self.pool, cos_sin=d(cs),
                       positions=None if pos is None else torch.tensor(pos, dtype=torch.int32, device=DEV),
                       interleaved=pairs, q=d(q), q_out=q_out, key_bounds=None if k is None else self.bounds,
                       dev_status=st, stream=stream)
        torch.cuda.synchronize()
        f = lambda t: None if t is None else t.float().numpy()
        at = np.asarray(slots).copy()
        if skip is not None:
            at[skip] = -1
        rows = None if cs is None else cs.numpy()[np.clip(pos, 0, cs.size(0) - 1)]
        X.append(self.want, self.fmts, self.bs, f(k), f(v), at, None if k is None else self.wb, rows, pairs)
        _same_pool(self.pool, self.want)
        np.testing.assert_array_equal(self.bounds.float().cpu().numpy(), self.wb, err_msg="bounds")
        if q is not None:
            turn = torch.tensor(X.turned(f(q), rows, pairs)).to(torch.bfloat16)
            live = (np.asarray(pos) >= 0) & (np.asarray(pos) < cs.size(0))
            np.testing.assert_array_equal(bits(q_out.cpu())[live], bits(turn)[live], err_msg="q")
            assert (q_out.cpu().contiguous().view(torch.uint8).numpy()[~live] == 0xA5).all()
        return int(st.item())


@pytest.mark.parametrize("fk,fv", [(PG, PG), (F8, NV), (NV, PG), (NV, F8)])
@pytest.mark.parametrize("D,rot,pairs,bs", [(128, 128, False, 16), (128, 64, True, 16), (64, 16, False, 8), (64, 64, True, 32),
                                            (256, 256, False, 16), (256, 96, False, 64), (96, 48, False, 7), (16, 16, False, 1),
                                            (512, 512, True, 16), (48, 32, True, 16), (128, 112, False, 200)])
def test_prompt_then_steps(fk, fv, D, rot, pairs, bs):
    """A prompt that ends inside a block, then single tokens, some of growing size."""
    H, Hq, T = 3, 7, 300 if bs == 200 else 75
    nb = 2 * (T // bs + 2) + (T if bs == 1 else 0)
    c = Cache(nb, H, D, bs, fk, fv)
    table = np.random.RandomState(D + bs).permutation(nb)
    slot = lambda p: int(table[p // bs]) * bs + p % bs
    cs = X.angles(T + 10, rot)
    assert c.append(_rows(T, H, D, 1), _rows(T, H, D, 2, 3.0), [slot(p) for p in range(T)], np.arange(T), cs, pairs,
                    _rows(T, Hq, D, 3)) == 0
    for i, f in enumerate((0.1, 8.0, 1000.0, 1.0)):
        p = T + i
        assert c.append(_rows(1, H, D, 5 + i, f), _rows(1, H, D, 9 + i, 1 / f), [slot(p)], [p], cs, pairs, _rows(1, Hq, D, 4)) == 0


@pytest.mark.parametrize("fk,fv", [(PG, PG), (NV, NV), (F8, PG)])
def test_without_a_rotation_it_is_the_store(fk, fv):
    H, D, bs, T = 4, 128, 16, 333
    slots = list(range(5, 5 + T))
    a, b = (kvq.KvPool.empty(400, H, D, bs, fill=0x11, fmt=fk, v_fmt=fv) for _ in range(2))
    k, v = _rows(T, H, D, 1).to(DEV), _rows(T, H, D, 2).to(DEV)
    kvq.kvq_quant_scatter(k, v, torch.tensor(slots, device=DEV), a)
    kvq.kvq_append(k, v, torch.tensor(slots, device=DEV), b)
    torch.cuda.synchronize()
    _same_pool(b, _host(a))


@pytest.mark.parametrize("tokens", [1, 40, 700, 5000, 11000, 21000])
@pytest.mark.parametrize("fk,fv", [(PG, PG), (NV, F8)])
def test_ragged_requests(tokens, fk, fv):
    """Several requests in one call, each beginning and ending inside a block, from a fused
    projection's views; Q turned in place."""
    H, Hq, D, bs = 4, 8, 128, 16
    r = np.random.RandomState(tokens)
    slots, pos, nb = [], [], 0
    for c in r.randint(0, 40, 6):
        n = max(1, tokens // 6)
        blocks = np.arange(nb, nb + (c + n) // bs + 1)[::-1]
        nb += len(blocks)
        slots += [int(blocks[p // bs]) * bs + p % bs for p in range(c, c + n)]
        pos += list(range(c, c + n))
    T = len(slots)
    cache = Cache(nb, H, D, bs, fk, fv, fill=0x38)
    for t in (cache.pool.k_rscale, cache.pool.v_rscale):
        t.fill_(2.0 ** -6)
    cache.want = _host(cache.pool)
    qkv = synth.normal_bf16((T, Hq + 2 * H, D), 3, synth.STREAM_K)
    on = qkv.to(DEV)
    cs = X.angles(max(pos) + 1, 128, 500000.0)
    kvq.kvq_append(on[:, Hq:Hq + H], on[:, Hq + H:], torch.tensor(slots, device=DEV), cache.pool, cos_sin=cs.to(DEV),
                   positions=torch.tensor(pos, dtype=torch.int32, device=DEV), q=on[:, :Hq], q_out=on[:, :Hq],
                   key_bounds=cache.bounds)
    torch.cuda.synchronize()
    rows = cs.numpy()[pos]
    x = qkv.float().numpy()
    X.append(cache.want, cache.fmts, bs, x[:, Hq:Hq + H], x[:, Hq + H:], slots, cache.wb, rows)
    _same_pool(cache.pool, cache.want)
    np.testing.assert_array_equal(cache.bounds.float().cpu().numpy(), cache.wb)
    got = on.cpu()
    np.testing.assert_array_equal(bits(got[:, :Hq].contiguous()), bits(torch.tensor(X.turned(x[:, :Hq], rows, False)).to(torch.bfloat16)))
    np.testing.assert_array_equal(bits(got[:, Hq:].contiguous()), bits(qkv[:, Hq:].contiguous()))


def test_parts_of_the_call():
    """K alone, V alone, Q alone; no bounds."""
    H, D, bs, T = 2, 64, 16, 37
    cs, pos = X.angles(T, 32), np.arange(T)
    c = Cache(4, H, D, bs, NV, PG)
    assert c.append(_rows(T, H, D, 1), None, pos, pos, cs) == 0
    assert c.append(None, _rows(T, H, D, 2), pos, pos, cs) == 0
    assert c.append(None, _rows(T, H, D, 3), pos) == 0
    q = _rows(T, 5, D, 4)
    out = poison_bf16(tuple(q.shape))
    before = _host(c.pool)
    got = kvq.kvq_append(None, None, None, c.pool, cos_sin=cs.to(DEV), positions=torch.tensor(pos, dtype=torch.int32, device=DEV),
                         q=q.to(DEV), q_out=out)
    torch.cuda.synchronize()
    assert got is out
    np.testing.assert_array_equal(bits(out.cpu()), bits(torch.tensor(X.turned(q.float().numpy(), cs.numpy(), False)).to(torch.bfloat16)))
    _same_pool(c.pool, before)


def test_rows_on_16_byte_boundaries():
    H, D, bs, T = 2, 64, 16, 40
    c = Cache(4, H, D, bs, PG)
    wide = synth.normal_bf16((T, H, D + 8), 6, synth.STREAM_K)
    on = wide.to(DEV)
    out = poison_bf16((T, H, D + 8))
    cs, pos = X.angles(T + 5, D), np.arange(5, 5 + T)
    kvq.kvq_append(on[:, :, 8:], on[:, :, :D], torch.tensor(pos, device=DEV), c.pool, cos_sin=cs.to(DEV),
                   positions=torch.tensor(pos, dtype=torch.int32, device=DEV), q=on[:, :, 8:], q_out=out[:, :, 8:],
                   key_bounds=c.bounds)
    torch.cuda.synchronize()
    x, rows = wide.float().numpy(), cs.numpy()[pos]
    X.append(c.want, c.fmts, bs, x[:, :, 8:], x[:, :, :D], pos, c.wb, rows)
    _same_pool(c.pool, c.want)
    np.testing.assert_array_equal(c.bounds.float().cpu().numpy(), c.wb)
    np.testing.assert_array_equal(bits(out.cpu()[:, :, 8:].contiguous()), bits(torch.tensor(X.turned(x[:, :, 8:], rows, False)).to(torch.bfloat16)))
    assert (out[:, :, :8].contiguous().view(torch.uint8) == 0xA5).all()


@pytest.mark.parametrize("fk", [PG, NV])
def test_skipped_tokens(fk):
    """Padding behind the last token, a token without a slot, one past the pool, one past the angles."""
    H, D, bs = 2, 128, 16
    c = Cache(6, H, D, bs, fk)
    slots = [3, 4, 5, -1, 16, 17, 10 ** 9, 34, 49, 96, 64, 65, -1, -1]
    pos = [3, 4, 5, 2, 6, 7, 7, 50, 9, 9, 4, 5, -1, -1]
    cs = X.angles(50, D)
    skip = [6, 7, 9]  # (-1 slots are skipped as they are)
    st = c.append(_rows(14, H, D, 1), _rows(14, H, D, 2), slots, pos, cs, q=_rows(14, 4, D, 3), skip=skip)
    assert st == kvq.DEV_BAD_SLOT | kvq.DEV_BAD_POS
    # a skipped position whose slot is valid
    st = c.append(_rows(3, H, D, 4), _rows(3, H, D, 5), [33, 34, 81], [1, -1, 3], cs, q=_rows(3, 4, D, 6), skip=[1])
    assert st == 0


@pytest.mark.parametrize("fk", [PG, F8, NV])
def test_zeros_and_tiny_rows(fk):
    H, D, bs, T = 2, 64, 16, 20
    c = Cache(3, H, D, bs, fk)
    k = _rows(T, H, D, 1)
    k[3] = 0
    k[4, 1] = 0
    k[5] = (k[5].float() * 2.0 ** -128).to(torch.bfloat16)
    k[6] = (k[6].float() * 2.0 ** 120).to(torch.bfloat16)
    # without a rotation, and with one by angle 0 (where every product is exact)
    assert c.append(k, k, np.arange(T)) == 0
    assert c.append(k, k, np.arange(16, 16 + T), np.zeros(T, np.int32), X.angles(1, D)) == 0


def test_bounds_of_nan_and_infinity():
    """A NaN key does not count; an infinity does."""
    H, D, bs = 1, 64, 16
    pool = kvq.KvPool.empty(32, H, D, bs, fill=0, fmt=F8)
    bounds = torch.zeros((2, H, 2, D), dtype=torch.bfloat16, device=DEV)
    k = _rows(16, H, D, 1)
    want = k.clone()
    k[2, 0, 5], k[3, 0, 6] = float("nan"), float("inf")
    want[2, 0, 5], want[3, 0, 6] = want[1, 0, 5], float("inf")
    kvq.kvq_append(k.to(DEV), None, torch.arange(16, device=DEV), pool, key_bounds=bounds)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bounds[0, :, 0].float().cpu().numpy(), want.float().amin(0).numpy())
    np.testing.assert_array_equal(bounds[0, :, 1].float().cpu().numpy(), want.float().amax(0).numpy())
    assert (bounds[1] == 0).all()


def test_infinite_key_costs_its_own_element():
    """In a page-scaled pool without a rotation, as in the store."""
    H, D, bs = 2, 128, 16
    k = _rows(16, H, D, 1)
    k[3, 1, 7] = float("-inf")
    a, b = (kvq.KvPool.empty(16, H, D, bs, fill=0, fmt=PG) for _ in range(2))
    kvq.kvq_quant_scatter(k.to(DEV), k.to(DEV), torch.arange(16, device=DEV), a)
    kvq.kvq_append(k.to(DEV), k.to(DEV), torch.arange(16, device=DEV), b)
    torch.cuda.synchronize()
    _same_pool(b, _host(a))


def test_graph_and_side_stream():
    """A captured step, replayed with other tokens in its buffers; and a call on a given stream."""
    H, Hq, D, bs = 2, 4, 128, 16
    c = Cache(4, H, D, bs, PG, NV)
    cs = X.angles(64, D)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    k, v, q = (torch.zeros((2, n, D), dtype=torch.bfloat16, device=DEV) for n in (H, H, Hq))
    slots, pos, out, on = torch.full((2,), -1, device=DEV), i32([-1, -1]), torch.zeros_like(q), cs.to(DEV)

    def call():
        kvq.kvq_append(k, v, slots, c.pool, cos_sin=on, positions=pos, q=q, q_out=out, key_bounds=c.bounds)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for step in range(20):
        hk, hv, hq = (_rows(2, n, D, 10 * step + n + j, 1.0 + step) for j, n in enumerate((H, H, Hq)))
        where, at = [step, 32 + step], [step, step + 7]
        k.copy_(hk), v.copy_(hv), q.copy_(hq)
        slots.copy_(torch.tensor(where)), pos.copy_(torch.tensor(at))
        g.replay()
        torch.cuda.synchronize()
        rows = cs.numpy()[at]
        X.append(c.want, c.fmts, bs, hk.float().numpy(), hv.float().numpy(), where, c.wb, rows)
        _same_pool(c.pool, c.want)
        np.testing.assert_array_equal(c.bounds.float().cpu().numpy(), c.wb)
        np.testing.assert_array_equal(bits(out.cpu()), bits(torch.tensor(X.turned(hq.float().numpy(), rows, False)).to(torch.bfloat16)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert c.append(_rows(2, H, D, 90), _rows(2, H, D, 91), [20, 52], [20, 21], cs, q=_rows(2, Hq, D, 92), stream=side) == 0


def test_overlapping_queries_are_refused():
    """q_out may be q itself or lie elsewhere, beside it in a fused row too; nothing in between."""
    H, D, bs, T = 2, 64, 16, 8
    pool = kvq.KvPool.empty(32, H, D, bs, fill=0, fmt=F8)
    x = _rows(T + 1, 8, D, 1).to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    call = lambda q, o, k: kvq.kvq_append(k, k, torch.arange(T, device=DEV), pool, cos_sin=X.angles(T, D).to(DEV), positions=pos,
                                          q=q, q_out=o)
    other = _rows(T, H, D, 2).to(DEV)
    for q, o, k in ((x[:T, :4], x[1:, :4], other), (x[:T, :4], x[:T, 1:5], other), (x[:T, :4], x[:T, 3:7], other),
                    (x[:T, :2], x[:T, 4:6], x[:T, 5:7]), (other, x[:T, :2], x[:T, 1:3])):
        with pytest.raises(kvq.KvqError, match="overlaps"):
            call(q, o, k)
    before = x.clone()
    call(x[:T, :2], x[:T, 4:6], x[:T, 6:])  # side by side in one row
    torch.cuda.synchronize()
    want = torch.tensor(X.turned(before[:T, :2].float().cpu().numpy(), X.angles(T, D).numpy(), False)).to(torch.bfloat16)
    assert torch.equal(x[:T, 4:6].cpu(), want) and torch.equal(x[:T, :4], before[:T, :4]) and torch.equal(x[:T, 6:], before[:T, 6:])


def test_host_memory_is_refused():
    H, D, T = 2, 64, 4
    pool = kvq.KvPool.empty(32, H, D, 16, fill=0, fmt=F8)
    k, slots = _rows(T, H, D, 1), torch.arange(T)
    for args in ((k, k.to(DEV), slots.to(DEV)), (k.to(DEV), k.to(DEV), slots)):
        with pytest.raises(kvq.KvqError, match="NOT_DEVICE_PTR"):
            kvq.kvq_append(*args, pool)


@pytest.mark.parametrize("rows", [33, 64, 100, 161])
@pytest.mark.parametrize("D", [64, 256, 512])
def test_blocks_of_many_rows(rows, D):
    """Blocks of 160 tokens, longer than a warp's stage and than a chunk of tokens, begun, continued and
    rescaled."""
    H, bs = 2, 160
    c = Cache(4, H, D, bs, PG, PG)
    cs = X.angles(400, D)
    at = 0
    for i, f in enumerate((1.0, 5.0, 0.5)):
        slots = np.arange(at, at + rows) + 7
        st = c.append(_rows(rows, H, D, i, f), _rows(rows, H, D, 9 + i, 2 * f), slots, np.arange(at, at + rows) % 400, cs)
        assert st == 0
        at += rows
