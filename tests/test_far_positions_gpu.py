"""kvq_attention at positions past 2^24, where a position itself is no binary32 number: the bias
goes by the distance of key and query, which is one.  A block table of one page over and over
stands in for the long cache, and a window keeps the keys to the last few pages."""

import math

import numpy as np
import pytest
import torch

import paged_ref as R
import quantized_kv_cache_nvfp4_gb300 as kvq
from kvq_testutil import DEV, poison_bf16, status_word
from quantized_kv_cache_nvfp4_gb300 import synth
from test_query_attention_gpu import decoded

PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4


def far_case(L, n, H, group, D, bs, fmt, window, slopes=None, softcap=0.0, seed=71, real=4):
    """(out, status, reference, bound) of n query tokens at the end of a sequence of L tokens."""
    # real: the last pages, which the window reaches; page 0 of the pool stands for the others
    mb = -(-L // bs)
    table = torch.zeros((1, mb), dtype=torch.int32)
    table[0, mb - real:] = torch.arange(1, real + 1, dtype=torch.int32)
    pool = kvq.KvPool.empty((real + 1) * bs, H, D, bs, fill=0xFF, fmt=fmt)
    first = (mb - real) * bs
    count = L - first
    k, v = (synth.normal_bf16((count, H, D), seed, st, 0.01, 8.0) for st in (synth.STREAM_K, synth.STREAM_V))
    slots = bs + torch.arange(count)
    kvq.kvq_quant_scatter(k.to(DEV), v.to(DEV), slots.to(DEV), pool)
    q = synth.normal_bf16((n, H * group, D), seed, 9)
    out, st = poison_bf16(tuple(q.shape)), status_word()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    kvq.kvq_attention(pool, table.to(DEV), i32([L]), L, q.to(DEV), i32([0, n]), n, D ** -0.5, out, softcap=softcap, window=window,
                      alibi_slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device=DEV), dev_status=st)
    torch.cuda.synchronize()
    sl = slots.numpy()
    K = decoded(fmt, pool.k_codes, pool.k_bscale, pool.k_rscale, sl, bs)
    V = decoded(fmt, pool.v_codes, pool.v_bscale, pool.v_rscale, sl, bs)
    ref, top = R.attention(q.double().numpy(), [K], [V], [count], [0, n], D ** -0.5, softcap=softcap, slopes=slopes, window=window)
    vmax = np.repeat(np.abs(V).max((0, 2)), group)
    d = 2.0 ** -20 * softcap + 2.0 ** -21 * top + 2.0 ** -22 * math.sqrt(D)
    return out.double().cpu().numpy(), int(st.item()), ref, 2.0 ** -8 * np.abs(ref) + ((2.0 ** -10 + 4 * d) * vmax)[..., None]


@pytest.mark.gpu
@pytest.mark.parametrize("L", [2 ** 24 + 50, 2 ** 24 + 2 ** 23 + 51])
@pytest.mark.parametrize("H,group,D,bs,fmt", [(8, 2, 128, 1024, PG), (2, 4, 64, 512, NV), (3, 4, 128, 1000, F8), (4, 2, 256, 512, PG)])
@pytest.mark.parametrize("n", [1, 3, 60])
def test_bias_at_far_positions(L, H, group, D, bs, fmt, n):
    slopes = np.linspace(0.05, 1.5, H * group).astype(np.float32)
    for cap in (0.0, 20.0):
        got, st, ref, bound = far_case(L, n, H, group, D, bs, fmt, 200, slopes, cap)
        assert st == 0 and (np.abs(got - ref) <= bound).all(), np.nanmax(np.abs(got - ref) / bound)


@pytest.mark.gpu
@pytest.mark.parametrize("H,group,D,fmt", [(8, 2, 128, PG), (2, 4, 64, NV), (3, 4, 128, F8)])
@pytest.mark.parametrize("n", [1, 3, 60])
def test_the_longest_sequences(H, group, D, fmt, n):
    """Every position up to the last one allowed."""
    got, st, ref, bound = far_case(2 ** 31 - 65536, n, H, group, D, 16384, fmt, 300, real=2)
    assert st == 0 and (np.abs(got - ref) <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("H,group,D,bs,fmt", [(8, 2, 128, 16, NV), (8, 2, 128, 16, PG), (3, 2, 64, 16, F8), (2, 2, 256, 8, NV)])
def test_no_limit_given(H, group, D, bs, fmt):
    """max_seq_len of INT_MAX: the block table alone limits the lengths."""
    from test_query_attention_gpu import Case

    for S in (3, 300):
        c = Case([20 + s % 30 for s in range(S)], [1] * S, H, group, D, bs, fmt, seed=72)
        out, st = c.run(max_len=2 ** 31 - 1)
        assert st == 0
        c.check(out, seqs=range(0, S, 17))
        out, st = poison_bf16((S, H * group, D)), status_word()
        ws = torch.empty(max(16, kvq.kvq_decode_attention_workspace(S, H, H * group, D, 2 ** 31 - 1)), dtype=torch.uint8, device=DEV)
        kvq.kvq_decode_attention(c.pool, c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV), 2 ** 31 - 1,
                                 c.q[:S].to(DEV), c.scale, out, ws, st)
        assert int(st.item()) == 0
        c.check(out, seqs=range(0, S, 17))


def test_longer_ones_are_refused(kvq_lib_path):
    import ctypes

    from quantized_kv_cache_nvfp4_gb300 import _abi

    lib = _abi.load()
    q, o = _abi.Bf16In(None, 1024, 128), _abi.Bf16Out(None, 1024, 128)
    for fmt in (PG, F8, NV):
        pool = _abi.Pool(_abi.Plane(), _abi.Plane(), 64, 16, 2, 128, fmt)
        for blocks, most, want in ((1 << 27, 2 ** 31 - 1, 2), (1 << 27, 2 ** 31 - 65535, 2), (1 << 27, 2 ** 31 - 65536, 1), (4, 2 ** 31 - 1, 1)):
            st = lib.kvq_attention(ctypes.byref(pool), None, 1, blocks, None, most, ctypes.byref(q), None, 8, 8, 8, 0.1, None,
                                   ctypes.byref(o), None, 0, None, None)
            assert st == want and (b"tokens" in lib.kvq_last_error()) == (want == 2)
            st = lib.kvq_decode_attention(ctypes.byref(pool), None, 1, blocks, None, most, ctypes.byref(q), 8, 0.1, ctypes.byref(o),
                                          None, 0, None, None)
            assert st == want and (b"tokens" in lib.kvq_last_error()) == (want == 2)
