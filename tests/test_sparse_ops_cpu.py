"""Refusals of the sparse step's operators, before anything touches a GPU, and the host-only
queries; the plain definitions of the tests among themselves."""

import ctypes

import numpy as np
import pytest
import torch

import paged_ref as R
import sparse_ref as X


def _pool(_abi, fmt=5, D=128):
    return _abi.Pool(_abi.Plane(), _abi.Plane(), 64, 16, 2, D, fmt)


def test_append_refusals(kvq_lib_path):
    from quantized_kv_cache_nvfp4_gb300 import _abi

    lib = _abi.load()
    pool = _pool(_abi)
    x, o = _abi.Bf16In(None, 256, 128), _abi.Bf16Out(None, 1024, 128)
    fake = 1 << 20  # never read: the checks before come first

    def call(k=x, v=x, T=8, rot=None, q=None, qo=None, hq=8, bounds=None):
        ref = lambda s: None if s is None else ctypes.byref(s)
        st = lib.kvq_append(ref(k), ref(v), T, None, ctypes.byref(pool), ref(rot), ref(q), ref(qo), hq, bounds, None, None)
        return st, lib.kvq_last_error()

    turn = lambda rot=128, n=10: _abi.Rotation(fake, n, rot, 0, None)
    assert call(k=None, v=None)[0] == 1
    assert call(T=-1)[0] == 1 and call(T=1 << 30)[0] == 2
    assert call(k=None, bounds=fake) == (1, b"key_bounds needs k")
    assert call(q=x)[0] == 1 and call(qo=o)[0] == 1
    st, why = call(q=x, qo=o)
    assert st == 1 and b"rotation" in why
    assert call(q=x, qo=o, rot=turn(), hq=0)[0] == 1 and call(q=x, qo=o, rot=turn(), hq=1 << 29)[0] == 2
    for r in (0, -16, 8, 24, 144):
        st, why = call(rot=turn(r))
        assert st == 1 and b"rot_dim" in why
    assert call(rot=turn(n=-1))[0] == 1
    assert call(T=0)[0] == 0 and call(T=0, rot=turn(), q=x, qo=o)[0] == 0
    assert call() == (1, b"k is NULL")
    pool.head_dim = 100
    assert call()[0] == 1
    pool.head_dim, pool.fmt = 128, 2
    assert call()[0] == 1
    pool.fmt, pool.num_slots = 5, 63
    assert call()[0] == 1
    assert lib.kvq_append(ctypes.byref(x), None, 8, None, None, None, None, None, 0, None, None, None) == 1


def test_select_refusals(kvq_lib_path):
    from quantized_kv_cache_nvfp4_gb300 import _abi

    lib = _abi.load()
    q = _abi.Bf16In(None, 1024, 128)

    def call(nb=10, bs=16, H=2, D=128, S=1, mb=4, mlen=64, T=8, mq=8, hq=8, first=1, last=1, topk=4, qq=q):
        st = lib.kvq_select_blocks(None, nb, bs, H, D, None, S, mb, None, mlen, None if qq is None else ctypes.byref(qq),
                                   None, T, mq, hq, first, last, topk, None, None, 0, None, None)
        return st, lib.kvq_last_error()

    for bad in (dict(S=-1), dict(mb=-1), dict(mlen=-1), dict(T=-1), dict(mq=-1)):
        st, why = call(**bad)
        assert st == 1 and b"negative" in why
    assert call(bs=0)[0] == 1 and call(nb=-1)[0] == 1 and call(topk=0)[0] == 1 and call(topk=-3)[0] == 1
    for bad in (dict(first=-1), dict(last=-1), dict(first=3, last=2), dict(first=2 ** 31 - 1, last=2 ** 31 - 1)):
        assert call(**bad)[0] == 1
    assert call(hq=3)[0] == 1 and call(hq=0)[0] == 1 and call(hq=34)[0] == 2
    for D, want in ((96, 2), (100, 1), (512, 2), (0, 1)):
        assert call(D=D)[0] == want
    assert call(S=70000)[0] == 2 and call(T=1 << 30, mq=1)[0] == 2
    st, why = call(mb=40000, mlen=16 * 40000)
    assert st == 2 and b"32768 blocks" in why
    assert call(mb=1 << 28, mlen=2 ** 31 - 1, topk=1 << 30)[0] == 2  # tokens
    assert call(S=0)[0] == 0 and call(T=0)[0] == 0 and call(mq=0)[0] == 0
    assert call(qq=None)[0] == 1 and call() == (1, b"q is NULL")
    assert lib.kvq_select_blocks_workspace(0, 2, 64, 16) == 0 and lib.kvq_select_blocks_workspace(8, 2, 64, 0) == 0
    assert lib.kvq_select_blocks_workspace(8, 2, 64, 16) >= 8 * 2 * 4 * 4


def test_sparse_attention_refusals(kvq_lib_path):
    from quantized_kv_cache_nvfp4_gb300 import _abi

    lib = _abi.load()
    pool = _pool(_abi)
    q, o = _abi.Bf16In(None, 1024, 128), _abi.Bf16Out(None, 1024, 128)

    def call(S=1, mb=4, mlen=64, T=8, mq=8, hq=8, topk=4, scale=0.1, cap=0.0, qq=q):
        st = lib.kvq_sparse_attention(ctypes.byref(pool), None, S, mb, None, mlen, None if qq is None else ctypes.byref(qq),
                                      None, T, mq, hq, None, topk, scale, cap, ctypes.byref(o), None, 0, None, None)
        return st, lib.kvq_last_error()

    for bad in (dict(S=-1), dict(mb=-1), dict(mlen=-1), dict(T=-1), dict(mq=-1)):
        st, why = call(**bad)
        assert st == 1 and b"negative" in why
    assert call(hq=3)[0] == 1 and call(hq=0)[0] == 1 and call(hq=34)[0] == 2
    assert call(topk=0)[0] == 1 and call(topk=4097)[0] == 2
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=s)[0] == 1
    for cap, want in ((-1.0, 1), (float("inf"), 1), (float("nan"), 1), (2.0 ** -11, 2), (2000.0, 2)):
        st, why = call(cap=cap)
        assert st == want and b"softcap" in why
    assert call(S=70000)[0] == 2 and call(T=1 << 30, mq=1)[0] == 2
    assert call(S=0)[0] == 0 and call(T=0)[0] == 0 and call(mq=0)[0] == 0
    assert call(qq=None)[0] == 1 and call() == (1, b"q is NULL")
    pool.block_size, pool.num_slots = 1 << 20, 1 << 20
    assert call(topk=4096)[0] == 2  # a list of 2^32 tokens
    pool.block_size, pool.num_slots = 16, 64
    for D, want in ((96, 2), (100, 1), (512, 2)):
        pool.head_dim = D
        assert call()[0] == want
    pool.head_dim, pool.fmt = 128, 2
    assert call()[0] == 1
    assert lib.kvq_sparse_attention_workspace(0, 2, 8, 128, 16, 4) == 0
    assert lib.kvq_sparse_attention_workspace(8, 2, 1, 128, 16, 4) == 0


def test_binding_checks_types_and_shapes(kvq_lib_path):
    import quantized_kv_cache_nvfp4_gb300 as kvq

    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    pool = kvq.KvPool.empty(64, 2, 128, 16, device="cpu", fmt=kvq.FMT_FP8_PAGE)
    i64 = torch.zeros(4, dtype=torch.int64)
    ok = dict(k=bf(4, 2, 128), v=bf(4, 2, 128), slot_ids=i64, pool=pool, cos_sin=torch.zeros(9, 64), positions=i32(4),
              q=bf(4, 8, 128), q_out=bf(4, 8, 128), key_bounds=bf(4, 2, 2, 128))
    for change, err in ((dict(k=bf(4, 3, 128)), ValueError), (dict(v=bf(5, 2, 128)), ValueError), (dict(k=bf(4, 2, 64)), ValueError),
                        (dict(k=torch.zeros(4, 2, 128)), TypeError), (dict(slot_ids=i32(4)), TypeError),
                        (dict(slot_ids=i64[:3]), ValueError), (dict(positions=None), ValueError), (dict(positions=i64), TypeError),
                        (dict(positions=i32(3)), ValueError), (dict(cos_sin=torch.zeros(9, 64).double()), ValueError),
                        (dict(cos_sin=torch.zeros(9, 128)[:, ::2]), ValueError), (dict(q_out=None), ValueError),
                        (dict(q=None), ValueError), (dict(q_out=bf(4, 4, 128)), ValueError),
                        (dict(key_bounds=bf(3, 2, 2, 128)), ValueError), (dict(key_bounds=torch.zeros(4, 2, 2, 128)), TypeError),
                        (dict(key_bounds=bf(4, 2, 128, 2).transpose(2, 3)), ValueError),
                        (dict(k=None, v=None, q=None, q_out=None), ValueError)):
        with pytest.raises(err):
            kvq.kvq_append(**{**ok, **change})
    ok = dict(key_bounds=bf(4, 2, 2, 128), block_table=i32(2, 4), seq_lens=i32(2), max_seq_len=64, block_size=16, q=bf(4, 8, 128),
              query_starts=i32(3), max_query_len=2, selected=i32(4, 2, 3))
    for change, err in ((dict(block_table=i32(2, 4).long()), TypeError), (dict(block_table=i32(4, 2).T), ValueError),
                        (dict(seq_lens=i32(3)), ValueError), (dict(query_starts=i32(2)), ValueError),
                        (dict(selected=i32(4, 3, 3)), ValueError), (dict(selected=i32(4, 2, 6)[..., ::2]), ValueError),
                        (dict(selected=i32(4, 2, 3).long()), TypeError), (dict(key_bounds=bf(4, 2, 2, 64)), ValueError),
                        (dict(q=torch.zeros(4, 8, 128)), TypeError)):
        with pytest.raises(err):
            kvq.kvq_select_blocks(**{**ok, **change})
    ok = dict(pool=pool, block_table=i32(2, 4), seq_lens=i32(2), max_seq_len=64, q=bf(4, 8, 128), query_starts=i32(3),
              max_query_len=2, selected=i32(4, 2, 3), scale=0.1, out=bf(4, 8, 128))
    for change, err in ((dict(block_table=i32(2, 4).long()), TypeError), (dict(seq_lens=i32(3)), ValueError),
                        (dict(selected=i32(5, 2, 3)), ValueError), (dict(out=bf(4, 4, 128)), ValueError),
                        (dict(q=bf(4, 8, 64), out=bf(4, 8, 64)), ValueError), (dict(query_starts=i32(3).long()), TypeError)):
        with pytest.raises(err):
            kvq.kvq_sparse_attention(**{**ok, **change})


def test_plain_selection_bounds_the_scores():
    """The bound that the selection ranks by is one: no key of a block exceeds it."""
    r = np.random.RandomState(0)
    H, g, D, bs = 2, 3, 32, 8
    k = r.randn(5 * bs, H, D)
    b = np.stack([np.stack((k[i * bs:(i + 1) * bs].min(0), k[i * bs:(i + 1) * bs].max(0)), 1) for i in range(5)])
    q = r.randn(H * g, D)
    x, ok = X.scores(q, b, np.arange(5), 5, H)
    dots = np.einsum("hgd,thd->ht", q.reshape(H, g, D), k)
    assert ok.all() and (x >= dots.reshape(H, 5, bs).max(2) - 1e-12).all()


def test_plain_codecs_agree_with_the_oracle():
    """The tests' own row codecs, on bf16 rows, against the oracle's."""
    import oracle as O
    from quantized_kv_cache_nvfp4_gb300 import synth

    x = synth.normal_bf16((200, 2, 64), 1, synth.STREAM_K, 0.02, 30.0)
    x[5], x[6] = 0, (x[6].float() * 2.0 ** -126).to(torch.bfloat16)
    c, b, s = X.row_codes(x.float().numpy(), X.NVFP4)
    oc, ob, os_ = O.nvfp4_encode_rows(synth.bf16_bits(x))
    np.testing.assert_array_equal(c, oc)
    np.testing.assert_array_equal(b, ob)
    np.testing.assert_array_equal(s, os_)
    c, _, s = X.row_codes(x.float().numpy(), X.ROW8)
    oc, os_ = O.fp8_encode_rows(synth.bf16_bits(x))
    np.testing.assert_array_equal(c, oc)
    np.testing.assert_array_equal(s, os_)
    assert R.e4m3_value(R.e4m3_code(np.array([448.0])))[0] == 448
