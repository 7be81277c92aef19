"""The refusals of the paged operators that need no GPU, and the 64-bit definitions the GPU
tests compare with."""

import ctypes

import numpy as np
import torch

import paged_ref as R


def test_e4m3_definition_matches_torch():
    x = np.concatenate([np.linspace(-448, 448, 20001), R.e4m3_value(np.arange(127)),
                        (R.e4m3_value(np.arange(126)) + R.e4m3_value(np.arange(1, 127))) / 2, [-0.0, 2.0 ** -11]])
    want = torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    same = R.e4m3_code(x.astype(np.float32).astype(np.float64))
    np.testing.assert_array_equal(same, want)
    c = np.arange(256, dtype=np.uint8)
    np.testing.assert_array_equal(R.e4m3_value(c), torch.tensor(c).view(torch.float8_e4m3fn).double().numpy())


def test_page_scale_is_the_smallest_power_of_two():
    for a, want in ((448.0, 1.0), (449.0, 2.0), (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (0.0, 2.0 ** -126), (3e38, 2.0 ** 120)):
        assert R.pow2_scale(a) == want


def test_plan_definition():
    t = np.array([[5, 6, 0], [7, 0, 0]])
    table, lens, starts, slots, pos, used, status = R.plan([17, 3], [16, 1], [1, 2], 16, t, 20)
    assert table.tolist() == [[5, 6, 1], [7, 0, 0]] and lens.tolist() == [33, 4] and starts.tolist() == [0, 16, 17]
    assert slots[0] == 97 and slots[15] == 16 and slots[16] == 115 and (slots[17:] == -1).all()
    assert pos[:17].tolist() == list(range(17, 33)) + [3] and used == 1 and status == 0


def test_storage_of_page_scaled_rows(kvq_lib_path):
    import quantized_kv_cache_nvfp4_gb300 as kvq

    assert kvq.kvq_storage_bytes(kvq.FMT_FP8_PAGE, 0, 16, 33, 2, 128) == 33 * 2 * 128 + 3 * 2 * 4
    assert kvq.kvq_storage_bytes(kvq.FMT_FP8_PAGE, 0, 0, 33, 2, 128) == 0
    pool = kvq.KvPool.empty(64, 2, 128, 16, device="cpu", fmt=kvq.FMT_FP8_PAGE)
    assert pool.nbytes() == 2 * kvq.kvq_storage_bytes(kvq.FMT_FP8_PAGE, 0, 16, 64, 2, 128)
    pool.k_rscale = torch.zeros((64, 2))
    try:
        pool._struct()
        raise AssertionError("a row-scale plane was taken for page scales")
    except ValueError as e:
        assert "k_rscale" in str(e)


def test_page_scaled_pools_are_pool_formats_only(kvq_lib_path):
    from quantized_kv_cache_nvfp4_gb300 import _abi

    lib = _abi.load()
    x = _abi.Bf16In(None, 256, 128)
    pool = _abi.Pool(_abi.Plane(), _abi.Plane(), 64, 16, 2, 128, 5)
    assert lib.kvq_quant_scatter(ctypes.byref(x), None, 4, None, ctypes.byref(pool), None, None) == 1
    assert b"slot_ids is NULL" in lib.kvq_last_error()  # the format itself is accepted
    pk = _abi.Packed(5, 0, 16, 4, 2, 128, None, None, None, None)
    assert lib.kvq_pack(ctypes.byref(x), ctypes.byref(pk), None) == 1
    assert b"unknown format" in lib.kvq_last_error()


def test_attention_refusals(kvq_lib_path):
    from quantized_kv_cache_nvfp4_gb300 import _abi

    lib = _abi.load()
    pool = _abi.Pool(_abi.Plane(), _abi.Plane(), 64, 16, 2, 128, 5)
    q, o = _abi.Bf16In(None, 1024, 128), _abi.Bf16Out(None, 1024, 128)

    def call(S=1, mb=4, mlen=64, T=8, mq=8, hq=8, scale=0.1, opt=None, qq=q):
        st = lib.kvq_attention(ctypes.byref(pool), None, S, mb, None, mlen, None if qq is None else ctypes.byref(qq),
                               None, T, mq, hq, scale, None if opt is None else ctypes.byref(opt), ctypes.byref(o),
                               None, 0, None, None)
        return st, lib.kvq_last_error()

    for bad in (dict(S=-1), dict(mb=-1), dict(mlen=-1), dict(T=-1), dict(mq=-1)):
        st, why = call(**bad)
        assert st == 1 and b"negative" in why
    assert call(hq=3)[0] == 1 and call(hq=0)[0] == 1 and call(hq=34)[0] == 2
    for s in (0.0, -1.0, float("inf"), float("nan")):
        st, why = call(scale=s)
        assert st == 1 and b"scale" in why
    for cap in (-1.0, float("inf"), float("nan")):
        st, why = call(opt=_abi.AttnOptions(cap, None, 0, None, None))
        assert st == 1 and b"softcap" in why
    for cap in (2.0 ** -11, 2000.0):
        st, why = call(opt=_abi.AttnOptions(cap, None, 0, None, None))
        assert st == 2 and b"softcap" in why
    st, why = call(opt=_abi.AttnOptions(0.0, None, -1, None, None))
    assert st == 1 and b"window" in why
    assert call(qq=None)[0] == 1
    assert call(S=70000)[0] == 2 and call(T=1 << 30)[0] == 2 and call(mq=1 << 30)[0] == 2
    assert call(S=0)[0] == 0 and call(T=0)[0] == 0 and call(mq=0)[0] == 0  # nothing to do
    st, why = call()
    assert st == 1 and b"NULL" in why  # q's pointer
    for D, want in ((96, 2), (100, 1), (512, 2)):
        pool.head_dim = D
        assert call()[0] == want
    pool.head_dim, pool.fmt = 128, 2
    assert call()[0] == 1
    assert lib.kvq_attention_workspace(0, 8, 2, 8, 128, 8, 64) == 0
    assert lib.kvq_attention_workspace(1, 8, 2, 8, 128, 0, 64) == 0
    assert lib.kvq_attention_workspace(1, 8, 2, 1, 128, 8, 64) == 0


def test_plan_refusals(kvq_lib_path):
    from quantized_kv_cache_nvfp4_gb300 import _abi

    lib = _abi.load()

    def call(S=2, free=4, bs=16, mb=3, T=9):
        return (lib.kvq_plan_pages(None, None, S, None, free, bs, None, mb, None, None, None, None, T, None, None, None),
                lib.kvq_last_error())

    for bad in (dict(S=-1), dict(free=-1), dict(mb=-1), dict(T=-1)):
        st, why = call(**bad)
        assert st == 1 and b"negative" in why
    assert call(bs=0)[0] == 1 and call(bs=-16)[0] == 1
    st, why = call(bs=1 << 20, mb=1 << 20)
    assert st == 2 and b"too large" in why
    st, why = call()
    assert st == 1 and b"query_starts is NULL" in why


def test_binding_checks_types_and_shapes(kvq_lib_path):
    import pytest

    import quantized_kv_cache_nvfp4_gb300 as kvq

    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    pool = kvq.KvPool.empty(64, 2, 128, 16, device="cpu", fmt=kvq.FMT_FP8_PAGE)
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    ok = dict(pool=pool, block_table=i32(2, 4), seq_lens=i32(2), max_seq_len=64, q=q, query_starts=i32(3), max_query_len=2,
              scale=0.1, out=q)
    for change, err in ((dict(block_table=i32(2, 4).long()), TypeError), (dict(block_table=i32(4, 2).T), ValueError),
                        (dict(seq_lens=i32(3)), ValueError), (dict(query_starts=i32(2)), ValueError),
                        (dict(query_starts=i32(3).long()), TypeError), (dict(q=q.float()), TypeError),
                        (dict(out=torch.zeros((5, 8, 128), dtype=torch.bfloat16)), ValueError),
                        (dict(alibi_slopes=torch.zeros(7)), ValueError), (dict(alibi_slopes=torch.zeros(8).double()), TypeError),
                        (dict(prefix_lens=i32(3)), ValueError), (dict(key_starts=i32(5)), ValueError),
                        (dict(key_starts=i32(8)[::2]), ValueError)):
        with pytest.raises(err):
            kvq.kvq_attention(**{**ok, **change})
    plan = [i32(2), i32(2), i32(5), 16, i32(2, 4), i32(2), i32(3), torch.zeros(9, dtype=torch.int64), i32(9), i32(1)]
    for i, bad in ((0, i32(3)), (1, i32(2).long()), (4, i32(2, 4).long()), (5, i32(1)), (6, i32(2)), (7, i32(9)), (8, i32(8)),
                   (9, i32(2))):
        with pytest.raises((TypeError, ValueError)):
            kvq.kvq_plan_pages(*(plan[:i] + [bad] + plan[i + 1:]))
