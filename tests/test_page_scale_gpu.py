"""FP8 cache with one scale per (block, head): scatter, restore and decode attention.

Codes and scales are compared byte for byte with the definition in 64 bits: s is a power
of two, so x / s and code * (s0 / s) are exact in binary32 and the one rounding to E4M3 is
the definition's.  Restored values are exact products (an E4M3 value has 4 significant
bits).  Decode attention has the tolerance of the other formats (test_attention_gpu.py)."""

import math

import numpy as np
import pytest
import torch

import oracle as O
import quantized_kv_cache_nvfp4_gb300 as kvq
import paged_ref as R
from quantized_kv_cache_nvfp4_gb300 import synth
from kvq_testutil import DEV, bits, poison_bf16, status_word

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4


def _rows(T, H, D, seed, factor=1.0, stream=synth.STREAM_K):
    return (synth.normal_bf16((T, H, D), seed, stream, 0.01, 20.0).float() * factor).to(torch.bfloat16)


def _host(pool):
    return [t.cpu().numpy().copy() for t in (pool.k_codes, pool.k_rscale, pool.v_codes, pool.v_rscale)]


def _store_both(pool, k, v, slots):
    """The call on the GPU and the definition on the host; both must agree on every byte."""
    want = _host(pool)
    st = status_word()
    kvq.kvq_quant_scatter(None if k is None else k.to(DEV), None if v is None else v.to(DEV),
                          torch.tensor(slots, device=DEV), pool, st)
    torch.cuda.synchronize()
    for x, j in ((k, 0), (v, 2)):
        if x is not None:
            with np.errstate(invalid="ignore"):
                R.page_store(want[j], want[j + 1], x.double().numpy(), np.asarray(slots), pool.block_size)
    got = _host(pool)
    for a, b, name in zip(got, want, ("k codes", "k scales", "v codes", "v scales")):
        np.testing.assert_array_equal(a.view(np.uint8), b.view(np.uint8), err_msg=name)
    return int(st.item())


@pytest.mark.parametrize("D", [16, 48, 64, 128, 256, 512])
@pytest.mark.parametrize("bs", [1, 7, 16, 64, 200])
def test_prompt_then_steps(D, bs):
    """A prompt, then single tokens whose growing values rescale the page they land in."""
    H, T, nb = 3, 300 if bs == 200 else 100, 30
    pool = kvq.KvPool.empty(nb * bs * (8 if bs == 1 else 1), H, D, bs, fill=0xFF, fmt=PG)
    table = np.random.RandomState(D).permutation(pool.num_slots // bs)
    slot = lambda p: int(table[p // bs]) * bs + p % bs
    assert _store_both(pool, _rows(T, H, D, 1), _rows(T, H, D, 1, 3.0, synth.STREAM_V), [slot(p) for p in range(T)]) == 0
    for i, f in enumerate((0.1, 8.0, 1000.0, 1.0)):
        p = T + i
        assert _store_both(pool, _rows(1, H, D, 5 + i, f), _rows(1, H, D, 9 + i, 1 / f), [slot(p)]) == 0


@pytest.mark.parametrize("tokens", [1, 33, 500, 4000])
def test_ragged_requests_of_many_pages(tokens):
    """Several requests in one call, each beginning and ending inside a page; K a view of a
    wider tensor, V on its own."""
    H, D, bs = 4, 128, 16
    r = np.random.RandomState(tokens)
    cached, slots, nb = r.randint(0, 40, 6), [], 0
    for c in cached:
        n = max(1, tokens // 6)
        blocks = np.arange(nb, nb + (c + n) // bs + 1)[::-1]
        nb += len(blocks)
        slots += [int(blocks[p // bs]) * bs + p % bs for p in range(c, c + n)]
    T = len(slots)
    pool = kvq.KvPool.empty(nb * bs, H, D, bs, fill=0, fmt=PG)
    pool.k_codes.copy_(torch.randint(0, 126, pool.k_codes.shape, dtype=torch.uint8))
    pool.k_rscale.fill_(2.0 ** -6)
    qkv = synth.normal_bf16((T, 3 * H, D), 3, synth.STREAM_K)
    assert _store_both(pool, qkv[:, H:2 * H], _rows(T, H, D, 4), slots) == 0
    assert _store_both(pool, None, _rows(T, H, D, 5, 100.0), slots) == 0


def test_rows_on_16_byte_boundaries():
    """Views whose rows start 16 bytes past a 32-byte boundary."""
    H, D, bs, T = 2, 64, 16, 40
    pool = kvq.KvPool.empty(4 * bs, H, D, bs, fill=0, fmt=PG)
    wide = synth.normal_bf16((T, H, D + 8), 6, synth.STREAM_K).to(DEV)
    want = _host(pool)
    kvq.kvq_quant_scatter(wide[:, :, 8:], wide[:, :, :D], torch.arange(5, 5 + T, device=DEV), pool)
    torch.cuda.synchronize()
    x = wide.cpu().double().numpy()
    R.page_store(want[0], want[1], x[:, :, 8:], np.arange(5, 5 + T), bs)
    R.page_store(want[2], want[3], x[:, :, :D], np.arange(5, 5 + T), bs)
    for a, b in zip(_host(pool), want):
        np.testing.assert_array_equal(a.view(np.uint8), b.view(np.uint8))


def test_scatter_under_graph_capture_appends_on_every_replay():
    H, D, bs = 2, 128, 16
    pool = kvq.KvPool.empty(2 * bs, H, D, bs, fill=0, fmt=PG)
    want = _host(pool)
    x = torch.zeros((1, H, D), dtype=torch.bfloat16, device=DEV)
    slot = torch.zeros(1, dtype=torch.int64, device=DEV)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        kvq.kvq_quant_scatter(x, x, slot, pool)
    for t in range(20):
        row = _rows(1, H, D, t, 1.5 ** t)
        x.copy_(row)
        slot.fill_(t)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for j in (0, 2):
            R.page_store(want[j], want[j + 1], row.double().numpy(), np.array([t]), bs)
    for a, b in zip(_host(pool), want):
        np.testing.assert_array_equal(a.view(np.uint8), b.view(np.uint8))


def test_extreme_values_and_scales():
    H, D, bs = 2, 32, 8
    pool = kvq.KvPool.empty(4 * bs, H, D, bs, fill=0, fmt=PG)
    x = torch.zeros((5, H, D))
    x[0, 0, :4] = torch.tensor([448.0, -448.0, 449.0, 2.0 ** -9])
    x[1, 1, 0] = 3.0e38
    x[2, 0, 0] = 2.0 ** -133  # a bf16 subnormal
    x[3, 0, :2] = torch.tensor([448 * 2.0 ** -126, -0.0])
    x = x.to(torch.bfloat16)
    for rows, slots in ((x[0:1], [0]), (x[1:2], [1]), (x[2:3], [bs]), (x[3:4], [2 * bs]), (x[4:5], [3 * bs]),
                        (x[0:1], [2 * bs + 1]), (x[1:2], [3 * bs + 1])):
        assert _store_both(pool, rows, rows, slots) == 0
    # a stored scale that is none (NaN, infinity, negative, 0) is replaced, one that is not a
    # power of two is kept while it reaches
    for bad in (float("nan"), float("inf"), -1.0, 0.0, 0.75):
        pool.k_rscale.fill_(bad)
        if bad != 0.75:
            assert _store_both(pool, _rows(1, H, D, 2), None, [5]) == 0
    pool.k_rscale.fill_(0.75)
    x = torch.full((1, H, D), 1.5).to(torch.bfloat16)  # 1.5 / 0.75 = 2 up to the rounding of 1 / 0.75
    kvq.kvq_quant_scatter(x.to(DEV), None, torch.tensor([6], device=DEV), pool)
    assert (pool.k_rscale[0] == 0.75).all() and (pool.k_codes[6] == 0x40).all()


def test_skipped_and_bad_slots():
    H, D, bs = 2, 64, 16
    pool = kvq.KvPool.empty(3 * bs, H, D, bs, fill=0, fmt=PG)
    assert _store_both(pool, _rows(6, H, D, 1), _rows(6, H, D, 2), [-1, 0, 1, -1, 40, -9]) == 0
    assert _store_both(pool, _rows(3, H, D, 1), None, [3 * bs, 20, 1 << 60]) == kvq.DEV_BAD_SLOT


def test_page_filled_token_by_token_restores_what_one_call_gives():
    """Within half a step of E4M3's subnormal range at the final scale, as the definition says."""
    H, D, bs = 2, 64, 16
    x = _rows(bs, H, D, 3)
    one, many = (kvq.KvPool.empty(bs, H, D, bs, fill=0, fmt=PG) for _ in range(2))
    kvq.kvq_quant_scatter(x.to(DEV), x.to(DEV), torch.arange(bs, device=DEV), one)
    for t in range(bs):
        kvq.kvq_quant_scatter(x[t:t + 1].to(DEV), x[t:t + 1].to(DEV), torch.tensor([t], device=DEV), many)
    assert torch.equal(one.k_rscale, many.k_rscale)
    a, b = (R.e4m3_value(p.k_codes.cpu().numpy()) for p in (one, many))
    assert np.abs(a - b).max() <= 2.0 ** -9  # one subnormal step: two roundings against one


@pytest.mark.parametrize("fmt_k,fmt_v", [(PG, None), (PG, NV), (F8, PG)])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 5), (96, 32)])
def test_restore(fmt_k, fmt_v, D, bs):
    H, lens = 3, [37, 0, 1, 64]
    mb = 64 // bs + 1
    S, nb = len(lens), len(lens) * mb
    pool = kvq.KvPool.empty(nb * bs, H, D, bs, fill=0xFF, fmt=fmt_k, v_fmt=fmt_v)
    table = synth.block_permutation(nb, 3).view(S, mb).contiguous()
    k, v = _rows(64 * S, H, D, 1), _rows(64 * S, H, D, 2)
    for s, n in enumerate(lens):
        p = torch.arange(n)
        if n:
            slots = (table[s, p // bs].long() * bs + p % bs).to(DEV)
            kvq.kvq_quant_scatter(k[s * 64:s * 64 + n].to(DEV), v[s * 64:s * 64 + n].to(DEV), slots, pool)
    ko, vo = poison_bf16((S, 64, H, D)), poison_bf16((S, 64, H, D))
    poison = ko.clone()
    st = status_word()
    kvq.kvq_restore(pool, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), 64, ko, vo, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for s, n in enumerate(lens):
        assert torch.equal(ko[s, n:].view(torch.int16), poison[s, n:].view(torch.int16))
        if not n:
            continue
        p = torch.arange(n)
        blk, slots = table[s, p // bs].numpy(), (table[s, p // bs].long() * bs + p % bs).numpy()
        for f, codes, sc, out in ((fmt_k, pool.k_codes, pool.k_rscale, ko), (fmt_v or fmt_k, pool.v_codes, pool.v_rscale, vo)):
            if f == PG:
                want = R.e4m3_value(codes.cpu().numpy()[slots]) * sc.cpu().numpy()[blk][..., None]
                np.testing.assert_array_equal(out[s, :n].double().cpu().numpy(), want)


def _decode_case(lens, H, group, D, bs, fmt_k, fmt_v, seed):
    S, Tmax = len(lens), max(lens)
    mb = -(-Tmax // bs)
    table = synth.block_permutation(S * mb + 3, seed)[: S * mb].view(S, mb).contiguous()
    pool = kvq.KvPool.empty((S * mb + 3) * bs, H, D, bs, fill=0xFF, fmt=fmt_k, v_fmt=fmt_v)  # NaN everywhere
    k, v = _rows(S * Tmax, H, D, seed), _rows(S * Tmax, H, D, seed, 1.0, synth.STREAM_V)
    for s, n in enumerate(lens):
        p = torch.arange(n)
        if n:
            slots = (table[s, p // bs].long() * bs + p % bs).to(DEV)
            kvq.kvq_quant_scatter(k[s * Tmax:s * Tmax + n].to(DEV), v[s * Tmax:s * Tmax + n].to(DEV), slots, pool)
    q = synth.normal_bf16((S, H * group, D), seed, 9)
    return pool, table, torch.tensor(lens, dtype=torch.int32), q, v.view(S, Tmax, H, D), Tmax


@pytest.mark.parametrize("fmt_k,fmt_v", [(PG, PG), (PG, NV), (F8, PG), (F8, F8), (NV, NV)])
@pytest.mark.parametrize("H,group,D,bs", [(8, 4, 128, 16), (4, 8, 64, 32), (16, 1, 128, 16), (2, 4, 128, 16),
                                          (3, 7, 64, 16), (2, 12, 256, 16), (8, 4, 128, 24),
                                          (4, 3, 256, 16), (8, 16, 256, 32)])
def test_decode_attention_over_pages_with_rubbish_behind_the_sequences(fmt_k, fmt_v, H, group, D, bs):
    """Both decode kernels (and their splits); whatever lies behind a sequence's last token,
    NaN codes and scales here, must not reach its output."""
    lens = [1, 37, 700, 0, 16]
    pool, table, lt, q, v, Tmax = _decode_case(lens, H, group, D, bs, fmt_k, fmt_v, 7 * H + D)
    st, out = status_word(), poison_bf16(tuple(q.shape))
    scale = 1.0 / math.sqrt(D)
    kvq.kvq_decode_attention(pool, table.to(DEV), lt.to(DEV), Tmax, q.to(DEV), scale, out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0

    def plane(f, codes, bscale, sc):
        sc = sc.cpu().numpy()
        if f == PG:
            sc = np.repeat(sc, bs, axis=0)
        return np.ascontiguousarray(codes.cpu().numpy()), None if bscale is None else bscale.cpu().numpy(), np.ascontiguousarray(sc)

    pk = plane(fmt_k, pool.k_codes, pool.k_bscale, pool.k_rscale)
    pv = plane(fmt_v, pool.v_codes, pool.v_bscale, pool.v_rscale)
    as_row = lambda f: F8 if f == PG else f
    ref, _ = O.decode_attention(pk, pv, as_row(fmt_k), as_row(fmt_v), bs, table.numpy(), lt.numpy(), bits(q), scale)
    got = out.double().cpu().numpy()
    for s, n in enumerate(lens):
        if n == 0:
            assert (got[s] == 0).all()
            continue
        # a decoded |v| is at most 1 + 2^-3 times the input's maximum (E2M1; E4M3 is closer)
        vmax = np.repeat(v[s, :n].float().abs().amax(dim=(0, 2)).numpy(), group) * 1.125
        bound = 2.0 ** -8 * np.abs(ref[s]) + 2.0 ** -10 * vmax[:, None]
        err = np.abs(got[s] - ref[s])
        assert (err <= bound).all(), (s, np.max(err / bound))


@pytest.mark.parametrize("H,D", [(8, 128), (4, 256), (2, 64)])
def test_decode_bad_sequences_keep_their_rows(H, D):
    lens = [300, 40, 17]
    pool, table, lt, q, v, Tmax = _decode_case(lens, H, 2, D, 16, PG, PG, 3)
    scale = D ** -0.5
    call = lambda t, n, o, st: kvq.kvq_decode_attention(pool, t.to(DEV), n.to(DEV), Tmax, q.to(DEV), scale, o, dev_status=st)
    good = poison_bf16(tuple(q.shape))
    call(table, lt, good, None)
    for bad_len in (-1, 10 ** 6):
        n, out, st = lt.clone(), poison_bf16(tuple(q.shape)), status_word()
        n[1] = bad_len
        call(table, n, out, st)
        assert int(st.item()) == kvq.DEV_BAD_SEQLEN and (out[1].contiguous().view(torch.uint8) == 0xA5).all()
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    t, out, st = table.clone(), poison_bf16(tuple(q.shape)), status_word()
    t[1, 1] = -7
    call(t, lt, out, st)
    assert int(st.item()) == kvq.DEV_BAD_BLOCK and (out[1].contiguous().view(torch.uint8) == 0xA5).all()
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


@pytest.mark.parametrize("H,D", [(8, 128), (4, 256)])
def test_decode_without_a_workspace_and_in_a_graph(H, D):
    lens = [2000, 3, 900]
    pool, table, lt, q, v, Tmax = _decode_case(lens, H, 4, D, 16, PG, PG, 5)
    table, lt, q = table.to(DEV), lt.to(DEV), q.to(DEV)
    a, b, c = (torch.zeros_like(q) for _ in range(3))
    kvq.kvq_decode_attention(pool, table, lt, Tmax, q, 0.1, a)
    kvq.kvq_decode_attention_noalloc(pool, table, lt, Tmax, q, 0.1, b)
    ws = torch.empty(kvq.kvq_decode_attention_workspace(3, H, 4 * H, D, Tmax), dtype=torch.uint8, device=DEV)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        kvq.kvq_decode_attention(pool, table, lt, Tmax, q, 0.1, c, ws)
    for _ in range(3):
        c.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(a, c)


def test_short_sequences_over_row_scales_need_no_workspace():
    """Only page-scaled pools split below 256 tokens."""
    lens = [200, 17, 256, 3]
    for fmt in (F8, NV):
        pool, table, lt, q, _, Tmax = _decode_case(lens, 8, 4, 128, 16, fmt, None, 3)
        out, ref = poison_bf16(tuple(q.shape)), poison_bf16(tuple(q.shape))
        args = (pool, table.to(DEV), lt.to(DEV), Tmax, q.to(DEV), 0.1)
        kvq.kvq_decode_attention(*args, out, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
        kvq.kvq_decode_attention(*args, ref)
        assert torch.equal(out, ref)
    pool, table, lt, q, _, Tmax = _decode_case(lens, 8, 4, 128, 16, PG, None, 3)
    assert kvq.kvq_decode_attention_workspace(4, 8, 32, 128, Tmax) > 0
    with pytest.raises(Exception, match="workspace"):
        kvq.kvq_decode_attention(pool, table.to(DEV), lt.to(DEV), Tmax, q.to(DEV), 0.1, poison_bf16(tuple(q.shape)),
                                 workspace=torch.empty(0, dtype=torch.uint8, device=DEV))


def test_nothing_to_attend():
    pool = kvq.KvPool.empty(64, 8, 128, 16, fill=0, fmt=PG)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    q = torch.ones((3, 8, 128), dtype=torch.bfloat16, device=DEV)
    out = poison_bf16((3, 8, 128))
    kvq.kvq_decode_attention(pool, z(3, 2), z(3), 0, q, 0.1, out)
    assert (out == 0).all()
    kvq.kvq_decode_attention(pool, z(0, 2), z(0), 32, q[:0], 0.1, out[:0])


def test_cache_past_4_gib():
    """Codes at byte offsets above 2^32: store, restore, decode and prompt attention there give
    what the same rows give at the pool's start."""
    H, D, bs, T = 8, 128, 16, 200
    nb = (5 << 30) // (bs * H * D)
    pool = kvq.KvPool.empty(nb * bs, H, D, bs, fmt=PG)
    k, v = _rows(T, H, D, 1).to(DEV), _rows(T, H, D, 2).to(DEV)
    q = synth.normal_bf16((T, 2 * H, D), 3, 9).to(DEV)
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    got = []
    for first in (0, nb - 13):
        table = torch.arange(first, first + 13, dtype=torch.int32, device=DEV).view(1, 13)
        p = torch.arange(T, device=DEV)
        st = status_word()
        kvq.kvq_quant_scatter(k, v, table[0, p // bs].long() * bs + p % bs, pool, st)
        ko, vo = (torch.zeros((1, T, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        kvq.kvq_restore(pool, table, lens, T, ko, vo, st)
        one, few, many = (torch.zeros((n, 2 * H, D), dtype=torch.bfloat16, device=DEV) for n in (1, 4, T))
        kvq.kvq_decode_attention(pool, table, lens, T, q[:1], 0.1, one, dev_status=st)
        for n, o in ((4, few), (T, many)):
            starts = torch.tensor([0, n], dtype=torch.int32, device=DEV)
            kvq.kvq_attention(pool, table, lens, T, q[:n], starts, n, 0.1, o, dev_status=st)
        assert int(st.item()) == 0
        got.append((ko, vo, one, few, many))
    for a, b in zip(*got):
        assert torch.equal(a, b) and a.abs().sum() > 0
