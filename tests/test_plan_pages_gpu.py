"""kvq_plan_pages against a plain loop: every output entry equal, nothing else written."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
import paged_ref as R
from kvq_testutil import DEV, status_word

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _run(cached, new, free, bs, table, max_tokens, positions=True, stream=None):
    S = len(cached)
    d = dict(table=_i32(table).view(table.shape), lens=_i32(np.full(S, -7)), starts=_i32(np.full(S + 1, -7)),
             slots=torch.full((max_tokens,), -7, dtype=torch.int64, device=DEV),
             pos=_i32(np.full(max_tokens, -7)), used=_i32([-7]), st=status_word())
    kvq.kvq_plan_pages(_i32(cached), _i32(new), _i32(free), bs, d["table"], d["lens"], d["starts"], d["slots"],
                       d["pos"] if positions else None, d["used"], d["st"], stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in d.items()}


def _same(got, want, positions=True):
    table, lens, starts, slots, pos, used, status = want
    np.testing.assert_array_equal(got["table"], table)
    np.testing.assert_array_equal(got["lens"], lens)
    np.testing.assert_array_equal(got["starts"], starts)
    np.testing.assert_array_equal(got["slots"], slots)
    np.testing.assert_array_equal(got["pos"], pos if positions else np.full_like(pos, -7))
    assert got["used"][0] == used and int(got["st"][0]) == status


@pytest.mark.parametrize("S,bs,most,cap", [(1, 16, 1, 40), (3, 16, 50, 100), (64, 16, 1, 900), (257, 1, 9, 30),
                                           (1024, 32, 40, 500), (1025, 7, 12, 200), (5000, 64, 3, 300), (2, 16, 30000, 9)])
def test_matches_the_plain_loop(S, bs, most, cap):
    r = np.random.RandomState(S + bs)
    cached, new = r.randint(0, cap + 1, S), r.randint(0, most + 1, S)
    mb = int((cached + new + bs - 1).max() // bs) + 1
    need = int(((cached + new + bs - 1) // bs - (cached + bs - 1) // bs).sum())
    perm = r.permutation(S * mb + need)
    table, free = perm[:S * mb].reshape(S, mb), perm[S * mb:]
    T = int(new.sum()) + 3
    for positions in (True, False):
        _same(_run(cached, new, free, bs, table, T, positions), R.plan(cached, new, free, bs, table, T), positions)


def test_nothing_to_do():
    t = np.zeros((0, 4), np.int32)
    _same(_run([], [], [1], 16, t, 5), R.plan([], [], [1], 16, t, 5))
    t = np.arange(8).reshape(2, 4)
    _same(_run([0, 17], [0, 0], [], 16, t, 0), R.plan([0, 17], [0, 0], [], 16, t, 0))


@pytest.mark.parametrize("cached,new,free,tokens", [
    ([5, -1, 3], [2, 4, 2], 9, 30),           # a negative length
    ([5, 60, 3], [2, 5, 2], 9, 30),           # past the table
    ([5, 2147483647, 3], [2, 2147483647, 2], 9, 30),
    ([5, 16, 3, 1], [2, -3, 2, 1], 9, 30),
    ([16, 16, 5, 16], [17, 40, 3, 1], 3, 90),  # the free list runs out at the second request
    ([16, 16, 5, 16], [1, 1, 1, 1], 0, 90),
    ([0, 0, 0], [10, 10, 10], 9, 25),          # the token arrays run out
])
def test_refused_requests(cached, new, free, tokens):
    table = np.arange(100, 100 + 4 * len(cached)).reshape(len(cached), 4)
    fb = np.arange(free)
    _same(_run(cached, new, fb, 16, table, tokens), R.plan(cached, new, fb, 16, table, tokens))


def test_negative_blocks_give_no_slot():
    table = np.array([[3, -1, 9]])
    _same(_run([20], [20], [-5, 6], 16, table, 20), R.plan([20], [20], [-5, 6], 16, table, 20))


def test_replayed_graph_follows_its_inputs_and_runs_on_its_stream():
    bs, T = 16, 64
    cached, new, free = _i32([3, 15, 40]), _i32([1, 1, 1]), _i32(np.arange(50, 90))
    table = _i32(np.arange(30)).view(3, 10).contiguous()
    lens, starts, pos, used = _i32([0] * 3), _i32([0] * 4), _i32([0] * T), _i32([0])
    slots = torch.zeros(T, dtype=torch.int64, device=DEV)
    s = torch.cuda.Stream()
    call = lambda: kvq.kvq_plan_pages(cached, new, free, bs, table, lens, starts, slots, pos, used)
    with torch.cuda.stream(s):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    t0 = np.arange(30).reshape(3, 10)
    for c, n in (([3, 15, 40], [1, 1, 1]), ([16, 0, 31], [20, 1, 2])):
        table.copy_(_i32(t0))
        cached.copy_(_i32(c))
        new.copy_(_i32(n))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = R.plan(c, n, np.arange(50, 90), bs, t0, T)
        got = [x.cpu().numpy() for x in (table, lens, starts, slots, pos)]
        for a, b in zip(got, want):
            np.testing.assert_array_equal(a, b)
        assert int(used) == want[5]


def test_host_tensors_and_overlapping_lengths_are_refused():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    args = [i32(2), i32(2), i32(5), 16, i32(2, 4), i32(2), i32(3), torch.zeros(9, dtype=torch.int64, device=DEV), i32(9), i32(1)]
    for i in (0, 1, 2, 4, 5, 6, 7, 8, 9):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_plan_pages(*(args[:i] + [args[i].cpu()] + args[i + 1:]))
    for i in (0, 1):  # the lengths in place
        with pytest.raises(kvq.KvqError, match="overlap"):
            kvq.kvq_plan_pages(*(args[:5] + [args[i]] + args[6:]))
