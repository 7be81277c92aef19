"""kvq_select_blocks against a sort of the scores in 64 bits: every list equal.  Inputs of the near
ties are integers and powers of two whose scores binary64 holds exactly."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
import sparse_ref as X
from kvq_testutil import DEV, status_word

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, lens, new, H, g, D, bs, seed=0, spare=2, shared=False):
        r = np.random.RandomState(seed)
        self.lens, self.new, self.H, self.D, self.bs = lens, new, H, D, bs
        S = len(lens)
        self.mb = max(1, -(-max(lens) // bs)) + 1
        nb = (1 if shared else S) * self.mb + 3  # shared: all sequences over the same blocks
        self.table = (np.stack([r.permutation(nb)[:self.mb] for _ in lens]) if shared else
                      r.permutation(nb)[:S * self.mb].reshape(S, self.mb)).astype(np.int32)
        self.starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        self.T = int(self.starts[-1]) + spare
        mean, half = r.randn(nb, H, D) * 0.5, 0.3 + r.rand(nb, H, D)
        self.bounds = torch.tensor(np.stack((mean - half, mean + half), 2)).to(torch.bfloat16)
        self.q = torch.tensor(r.randn(self.T, H * g, D)).to(torch.bfloat16)

    def run(self, topk, first=1, last=1, out=None, stream=None, max_len=None, max_q=None, lens=None, q=None):
        i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)
        st = status_word()
        out = torch.full((self.T, self.H, topk), -7, dtype=torch.int32, device=DEV) if out is None else out
        kvq.kvq_select_blocks(self.bounds.to(DEV), i32(self.table), i32(self.lens if lens is None else lens),
                              max_len or max(self.lens), self.bs, self.q.to(DEV) if q is None else q, i32(self.starts),
                              max_q or max(self.new), out, first_blocks=first, last_blocks=last, dev_status=st, stream=stream)
        torch.cuda.synchronize()
        return out.cpu().numpy(), int(st.item())

    def want(self, topk, first=1, last=1):
        out = np.full((self.T, self.H, topk), -7, np.int32)
        return X.select(self.q.float().numpy(), self.bounds.float().numpy(), self.table, self.lens, self.starts, self.bs, topk,
                        first, last, out)

    def check(self, topk, first=1, last=1, status=0):
        got, st = self.run(topk, first, last)
        assert st == status
        np.testing.assert_array_equal(got, self.want(topk, first, last))


@pytest.mark.parametrize("lens,new", [([1], [1]), ([800, 90], [3, 4]), ([800, 90], [2, 1]), ([1600, 40], [8, 5]), ([16, 17, 700], [1, 1, 1]), ([900, 0, 333], [4, 0, 7]), ([500], [300]),
                                      ([64, 2000], [64, 9])])
@pytest.mark.parametrize("H,g,D,bs", [(2, 4, 128, 16), (1, 16, 64, 8), (3, 7, 256, 32), (8, 1, 128, 64), (2, 3, 64, 1),
                                      (12, 2, 64, 16), (11, 1, 128, 16), (5, 2, 256, 16)])
def test_lists(lens, new, H, g, D, bs):
    c = Case(lens, new, H, g, D, bs, seed=D + bs)
    for topk, first, last in ((5, 1, 2), (16, 0, 0), (1, 1, 0), (40, 20, 20)):
        c.check(topk, first, last)


@pytest.mark.parametrize("blocks,topk", [(512, 100), (513, 100), (4096, 64), (4097, 64), (8193, 64), (16384, 100),
                                         (16385, 100), (20000, 300), (32768, 2000)])
def test_many_blocks(blocks, topk):
    """At and past the sizes at which a wider thread block takes over."""
    bs = 16 if blocks < 20000 else 2
    c = Case([bs * blocks, bs * blocks - 1], [1, 2], 1, 4, 64, bs, seed=blocks, shared=True)
    c.check(topk)


def test_a_list_for_all_needs_no_scores():
    """More than 32768 blocks, all of them listed; and the refusal where they are not."""
    c = Case([40000], [1], 1, 1, 64, 1, seed=3)
    got, st = c.run(40000)
    assert st == 0 and (got[0, 0] == np.arange(40000)).all() and (got[1:] == -7).all()
    with pytest.raises(kvq.KvqError, match="32768"):
        c.run(39999)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("blocks", [60, 700, 1500, 5000])
@pytest.mark.parametrize("new", [1, 12])
def test_near_ties(D, blocks, new):
    """Scores that differ by less than binary32 resolves: one channel adds 2^20 to all, another
    tells the blocks apart by multiples of 2^-8; then by differences that only the last bits of binary64 show."""
    c = Case([16 * blocks], [new], 2, 2, D, 16, seed=D)
    r = np.random.RandomState(blocks)
    for step, count in ((2.0 ** -8, 200), (2.0 ** -26, 250)):
        b = np.zeros(c.bounds.shape, np.float32)
        b[..., 1, 0] = 256.0
        b[..., 1, 1] = r.randint(0, count, b.shape[:2])
        b[..., 0, 2] = -r.randint(0, count, b.shape[:2])
        c.bounds = torch.tensor(b).to(torch.bfloat16)
        q = np.zeros(c.q.shape, np.float32)
        q[..., 0], q[..., 1], q[..., 2] = 2048.0, step, -step
        c.q = torch.tensor(q).to(torch.bfloat16)
        for topk in (3, 17, 50):
            c.check(topk, 1, 1)


@pytest.mark.parametrize("blocks,new", [(300, 2), (300, 70), (2000, 3), (5000, 9)])
def test_equal_scores_go_by_index(blocks, new):
    c = Case([16 * blocks], [new], 2, 4, 128, 16)
    c.bounds[:] = c.bounds[0]
    c.check(40)
    c.bounds[::3] = c.bounds[0] * 1.5
    c.check(40)
    c.q[:] = 0
    c.check(40, 0, 0)
    c.bounds[:] = 0
    c.check(7)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [3, 20])
def test_large_small_and_absent_numbers(D, new):
    """Sums that overflow binary32 and cancel in binary64, subnormal ones, infinities and NaN."""
    c = Case([16 * 90], [new], 2, 2, D, 16, seed=1)
    c.q[0] = (c.q[0].float() * 2.0 ** 100).to(torch.bfloat16)
    c.q[1] = (c.q[1].float() * 2.0 ** -126).to(torch.bfloat16)
    for f in (1.0, 2.0 ** 100, 2.0 ** -100, 2.0 ** -126):
        c.bounds = (c.bounds.float() * f).to(torch.bfloat16)
        c.check(12)
    c = Case([16 * 90], [new], 2, 2, D, 16, seed=2)
    c.bounds[c.table[0, 10], 0, 1, 3] = float("inf")
    c.bounds[c.table[0, 11], 0, 0, 3] = float("-inf")
    c.bounds[c.table[0, 12], 0, 1, 3] = float("nan")
    c.bounds[c.table[0, 20:50], 1, 0, 5] = float("nan")
    c.q[:, :, 3] = c.q[:, :, 3].abs() + 0.5  # no product of 0 and infinity
    c.q[:, 1, 3] *= -1
    c.q[2, 3, 8] = float("nan")
    for topk in (12, 75, 88):
        c.check(topk)


@pytest.mark.parametrize("new", [[1, 2], [30, 2]])
def test_blocks_outside_the_pool_come_last(new):
    c = Case([16 * 50, 16 * 30], new, 2, 4, 128, 16)
    c.table[0, 5], c.table[0, 49], c.table[1, 7] = -1, c.bounds.size(0), 10 ** 9
    c.check(10, status=kvq.DEV_BAD_BLOCK)
    c.check(49, status=kvq.DEV_BAD_BLOCK)
    c.check(50)


def test_refused_sequences_and_spare_rows():
    c = Case([800, 700, 600], [1, 2, 1], 2, 4, 64, 16)
    want = c.want(9)
    for lens, bad in (([800, -1, 600], 1), ([900, 700, 600], 0), ([800, 1, 600], 1)):
        got, st = c.run(9, lens=lens, max_len=800)
        assert st == kvq.DEV_BAD_SEQLEN
        mine = slice(c.starts[bad], c.starts[bad + 1])
        assert (got[mine] == -7).all()
        want_here = want.copy()
        want_here[mine] = -7
        np.testing.assert_array_equal(got, want_here)
    got, st = c.run(9, max_q=1)  # sequence 1 has more queries than announced
    assert st == kvq.DEV_BAD_SEQLEN and (got[1:3] == -7).all()


def test_views_graph_and_streams():
    """Queries out of a fused projection; two captured graphs with scratch of their own; a side stream."""
    c = Case([1600, 900], [2, 1], 2, 4, 128, 16)
    wide = torch.zeros((c.T, 20, 128), dtype=torch.bfloat16, device=DEV)
    wide[:, 5:13] = c.q.to(DEV)
    want = c.want(20)
    got, _ = c.run(20, q=wide[:, 5:13])
    np.testing.assert_array_equal(got, want)
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)
    bounds, table, lens, starts, q = c.bounds.to(DEV), i32(c.table), i32(c.lens), i32(c.starts), c.q.to(DEV)
    outs = [torch.full((c.T, 2, 20), -7, dtype=torch.int32, device=DEV) for _ in range(2)]
    graphs = []
    size = kvq.kvq_select_blocks_workspace(c.T, 2, 1600, 16)
    for o in outs:
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvq.kvq_select_blocks(bounds, table, lens, 1600, 16, q, starts, 2, o, workspace=ws)
        graphs.append((g, ws))
    for g, _ in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        np.testing.assert_array_equal(o.cpu().numpy(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = c.run(20, stream=side)
    np.testing.assert_array_equal(got, want)
