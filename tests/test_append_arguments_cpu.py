"""Arguments of kvq_append that would leave K unturned without a word are refused, before anything
touches a GPU."""

import ctypes

import pytest
import torch


def test_a_rotation_without_angles_is_refused(kvq_lib_path):
    from quantized_kv_cache_nvfp4_gb300 import _abi

    lib = _abi.load()
    pool, x = _abi.Pool(_abi.Plane(), _abi.Plane(), 64, 16, 2, 128, 5), _abi.Bf16In(None, 256, 128)
    fake = 1 << 20  # never read: the checks before come first

    def call(rot, T=8):
        st = lib.kvq_append(ctypes.byref(x), None, T, None, ctypes.byref(pool), ctypes.byref(rot), None, None, 0, None, None, None)
        return st, lib.kvq_last_error()

    for fields in ((None, 0, 128, 0, fake), (None, 10, 128, 0, fake), (None, 0, 0, 0, fake), (None, 0, 64, 0, None), (None, 5, 0, 1, None)):
        for T in (8, 0):
            st, why = call(_abi.Rotation(*fields), T)
            assert st == 1 and b"without cos_sin" in why
    assert call(_abi.Rotation(None, 0, 0, 0, None)) == (1, b"k is NULL")  # nothing to turn: on to the next check
    assert call(_abi.Rotation(fake, 0, 128, 0, fake)) == (1, b"k is NULL")  # every token is past the angles


def test_binding_refuses_empty_angles_and_positions_alone(kvq_lib_path):
    import quantized_kv_cache_nvfp4_gb300 as kvq

    pool = kvq.KvPool.empty(64, 2, 128, 16, device="cpu", fmt=kvq.FMT_FP8_PAGE)
    k, slots, pos = torch.zeros((4, 2, 128), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="no positions"):
        kvq.kvq_append(k, k, slots, pool, cos_sin=torch.zeros(0, 64), positions=pos)
    with pytest.raises(ValueError, match="positions need cos_sin"):
        kvq.kvq_append(k, k, slots, pool, positions=pos)
