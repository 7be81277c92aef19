"""The workspace that the binding allocates belongs to the stream that the call runs on: a block
from the current stream's pool may still be in use by kernels queued there."""

import contextlib

import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq


def test_scratch_is_allocated_under_the_given_stream(monkeypatch):
    now, seen = [None], []

    @contextlib.contextmanager
    def under(stream):
        now[0], before = stream, now[0]
        yield
        now[0] = before

    real = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (seen.append(now[0]), real(*a, **k))[1])
    side = object()
    assert kvq._workspace(64, "cpu", side).numel() == 64 and kvq._workspace(32, "cpu", None).numel() == 32
    assert seen == [side, None] and now == [None]


@pytest.mark.gpu
@pytest.mark.parametrize("decode", [False, True])
def test_calls_on_a_side_stream_beside_freed_blocks_in_use(decode):
    """A block of the workspace's size, freed while kernels queued on the current stream still
    write and read it; the call on the side stream must neither change nor be changed by them."""
    from kvq_testutil import DEV
    from test_query_attention_gpu import Case

    c = Case([4000, 700], [1, 1], 2, 4, 128, seed=31)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    table, lens, q, starts = c.table.to(DEV), i32(c.lens), c.q[:2].to(DEV), i32([0, 1, 2])
    need = max(kvq.kvq_attention_workspace(2, 2, 2, 8, 128, 1, 4000), kvq.kvq_decode_attention_workspace(2, 2, 8, 128, 4000))
    assert need > 0

    def call(out, stream):
        if decode:
            kvq.kvq_decode_attention(c.pool, table, lens, 4000, q, c.scale, out, stream=stream)
        else:
            kvq.kvq_attention(c.pool, table, lens, 4000, q, starts, 1, c.scale, out, stream=stream)

    want = torch.zeros_like(q)
    call(want, None)
    side = torch.cuda.Stream()
    big = torch.randn((4096, 4096), device=DEV)
    sums = []
    torch.cuda.synchronize()
    outs = [torch.zeros_like(q) for _ in range(30)]
    torch.cuda.synchronize()
    for out in outs:
        busy = torch.empty(need, dtype=torch.uint8, device=DEV)
        big = torch.tanh(big @ big)  # the current stream is busy
        for _ in range(4):
            busy.fill_(7)
            sums.append(busy.sum(dtype=torch.int64))
        del busy
        call(out, side)
    torch.cuda.synchronize()
    assert all(int(s) == 7 * need for s in sums)
    assert all(torch.equal(o, want) for o in outs)
