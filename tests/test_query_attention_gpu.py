"""kvq_attention against attention in 64 bits over the decoded rows.

Tolerance, as for decode attention (K, V and Q enter exactly, P rounded once to f16, the
output once to bf16): 2^-9 |o| + 2^-11 vmax, twice that in the test; plus what an error d
of the logits does to the weights, at most 4 d vmax, with d = 2^-20 softcap (the cap's own
bound) + 2^-21 max|logit| (a handful of binary32 roundings of values of that size) +
2^-22 sqrt(D) (the products' binary32 sums, of terms near 1 / sqrt(D))."""

import math

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
import paged_ref as R
from quantized_kv_cache_nvfp4_gb300 import synth
from kvq_testutil import DEV, poison_bf16, status_word

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def decoded(fmt, codes, bscale, scale, slots, bs):
    """float64 rows [n, H, D] of the given slots."""
    codes, scale = codes.cpu().numpy()[slots], scale.cpu().numpy().astype(np.float64)
    if fmt == NV:
        x = E2M1[np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:2], 2 * codes.shape[2])]
        return x * np.repeat(R.e4m3_value(bscale.cpu().numpy()[slots]) * scale[slots][..., None], 16, -1)
    return R.e4m3_value(codes) * scale[slots // bs if fmt == PG else slots][..., None]


class Case:
    """Sequences of `lens` tokens, the last `new` of each as queries, in a pool whose unused
    rows are NaN."""

    def __init__(self, lens, new, H, group, D, bs=16, fmt_k=PG, fmt_v=None, seed=0, spare=2):
        S, self.bs, self.D, self.H, self.group = len(lens), bs, D, H, group
        mb = max(1, -(-max(lens) // bs)) + 1
        nb = S * mb + 3
        self.table = synth.block_permutation(nb, seed)[:S * mb].view(S, mb).contiguous()
        self.pool = kvq.KvPool.empty(nb * bs, H, D, bs, fill=0xFF, fmt=fmt_k, v_fmt=fmt_v)
        self.lens, self.new = lens, new
        k = synth.normal_bf16((sum(lens), H, D), seed, synth.STREAM_K, 0.01, 8.0)
        v = synth.normal_bf16((sum(lens), H, D), seed, synth.STREAM_V, 0.01, 8.0)
        self.slots, at = [], 0
        for s, n in enumerate(lens):
            p = torch.arange(n)
            sl = self.table[s, p // bs].long() * bs + p % bs
            self.slots.append(sl.numpy())
            if n:
                kvq.kvq_quant_scatter(k[at:at + n].to(DEV), v[at:at + n].to(DEV), sl.to(DEV), self.pool)
            at += n
        self.starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        self.T = int(self.starts[-1]) + spare
        self.q = synth.normal_bf16((self.T, H * group, D), seed, 9)
        self.scale = 1.0 / math.sqrt(D)

    def run(self, max_q=None, max_len=None, out=None, q=None, lens=None, starts=None, table=None, **opts):
        dev = lambda a, t: None if a is None else torch.tensor(np.asarray(a), dtype=t, device=DEV)
        st = status_word()
        out = poison_bf16(tuple(self.q.shape)) if out is None else out
        kvq.kvq_attention(self.pool, (self.table if table is None else table).to(DEV),
                          dev(self.lens if lens is None else lens, torch.int32), max_len or max(self.lens),
                          self.q.to(DEV) if q is None else q,
                          dev(self.starts if starts is None else starts, torch.int32), max_q or max(self.new),
                          self.scale, out, softcap=opts.get("softcap", 0.0),
                          alibi_slopes=dev(opts.get("slopes"), torch.float32), window=opts.get("window", 0),
                          prefix_lens=dev(opts.get("prefix"), torch.int32),
                          key_starts=dev(opts.get("key_starts"), torch.int32), dev_status=st)
        torch.cuda.synchronize()
        return out, int(st.item())

    def check(self, out, seqs=None, **opts):
        p = self.pool
        K = [decoded(p.fmt, p.k_codes, p.k_bscale, p.k_rscale, sl, self.bs) for sl in self.slots]
        V = [decoded(p.fmt if p.v_fmt is None else p.v_fmt, p.v_codes, p.v_bscale, p.v_rscale, sl, self.bs)
             for sl in self.slots]
        ref, top = R.attention(self.q.double().numpy(), K, V, self.lens, self.starts, self.scale, **opts)
        got = out.double().cpu().numpy()
        for s in range(len(self.lens)) if seqs is None else seqs:
            if not self.new[s]:
                continue
            rows = slice(self.starts[s], self.starts[s + 1])
            vmax = np.repeat(np.abs(V[s]).max((0, 2)), self.group)
            d = 2.0 ** -20 * opts.get("softcap", 0.0) + 2.0 ** -21 * top[rows] + 2.0 ** -22 * math.sqrt(self.D)
            bound = 2.0 ** -8 * np.abs(ref[rows]) + ((2.0 ** -10 + 4 * d) * vmax)[..., None]
            err = np.abs(got[rows] - ref[rows])
            assert (err <= bound).all(), (s, np.nanmax(err / np.maximum(bound, 1e-30)))
        return ref

    def untouched(self, out, rows):
        return (out[rows].contiguous().view(torch.uint8) == 0xA5).all().item()


SHAPES = [
    # lens, new: single tokens; drafts; prompts; whole sequences, empty ones, odd ends
    ([1, 17, 300, 16], [1, 1, 1, 1]),
    ([40, 5, 333, 64], [4, 5, 1, 3]),
    ([130, 0, 257, 20], [130, 0, 31, 0]),
    ([400, 129], [260, 128]),
]


@pytest.mark.parametrize("lens,new", SHAPES)
@pytest.mark.parametrize("H,group,D", [(2, 4, 128), (1, 8, 64), (3, 7, 64), (2, 1, 256), (1, 16, 128)])
def test_causal(lens, new, H, group, D):
    c = Case(lens, new, H, group, D, seed=D + group)
    out, st = c.run()
    assert st == 0 and c.untouched(out, slice(c.starts[-1], c.T))
    c.check(out)


@pytest.mark.parametrize("fmt_k,fmt_v", [(NV, NV), (F8, F8), (PG, NV), (NV, PG), (F8, PG)])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 8), (128, 33), (256, 16)])
@pytest.mark.parametrize("new", [[1, 1], [5, 2], [150, 90]])
def test_formats(fmt_k, fmt_v, D, bs, new):
    c = Case([170, 260], new, 2, 4, D, bs, fmt_k, fmt_v, seed=bs)
    out, st = c.run()
    assert st == 0
    c.check(out)


OPTIONS = ["cap", "alibi", "window", "prefix", "docs", "cap+alibi", "cap+window+prefix", "alibi+docs+window"]


@pytest.mark.parametrize("which", OPTIONS)
@pytest.mark.parametrize("lens,new,H,group,D", [([300, 41, 16], [1, 1, 1], 2, 4, 128), ([300, 41, 16], [6, 3, 16], 2, 4, 64),
                                                ([420, 150, 9], [200, 150, 9], 2, 3, 128), ([300, 200], [90, 64], 1, 2, 256)])
def test_options(which, lens, new, H, group, D):
    c = Case(lens, new, H, group, D, seed=len(which))
    c.q = (c.q.float() * 4).to(torch.bfloat16)  # logits that the cap bends
    r = np.random.RandomState(5)
    opts = {}
    if "cap" in which:
        opts["softcap"] = 5.0
    if "alibi" in which:
        opts["slopes"] = (2.0 ** -np.arange(1, H * group + 1)).astype(np.float32)
    if "window" in which:
        opts["window"] = 33
    if "prefix" in which:
        opts["prefix"] = [lens[0] // 2, 10 ** 9, -3][:len(lens)]
    if "docs" in which:  # boundaries every 50 tokens
        opts["key_starts"] = np.concatenate([(np.arange(n - m, n) // 50) * 50 for n, m in zip(lens, new)] + [[0, 0]])
    out, st = c.run(**opts)
    assert st == 0 and c.untouched(out, slice(c.starts[-1], c.T))
    c.check(out, **opts)


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 30, 70]])
def test_rows_that_see_nothing_are_zero(new):
    """key_starts behind the query (and far out of range) leave a row without keys."""
    c = Case([90, 30, 200], new, 2, 4, 128, seed=3)
    ks = np.zeros(c.T, np.int64)
    ks[::2] = 10 ** 6
    ks[1::4] = -5
    out, st = c.run(key_starts=ks)
    assert st == 0
    c.check(out, key_starts=ks)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("n", [1, 60])
def test_left_padding_is_never_read(n):
    """Rows before key_starts hold NaN codes and scales in every format."""
    for f in (PG, F8, NV):
        c = Case([150], [n], 2, 4, 128, fmt_k=f, seed=4)
        ref_out, _ = c.run(key_starts=np.full(c.T, 32))
        c.check(ref_out, key_starts=np.full(c.T, 32))
        slots = torch.tensor(c.slots[0][:32], device=DEV)
        p = c.pool
        for t in (p.k_codes, p.v_codes, p.k_bscale, p.v_bscale):
            if t is not None:
                t[slots] = 0xFF
        for t in (p.k_rscale, p.v_rscale):
            t[slots // 16 if f == PG else slots] = float("nan")
        out, st = c.run(key_starts=np.full(c.T, 32))
        assert st == 0 and torch.equal(out[:n], ref_out[:n])


@pytest.mark.parametrize("lens,new", [([6000], [1]), ([6000, 300], [3, 2]), ([5000], [300]), ([3000, 7], [64, 7])])
def test_long_sequences_split(lens, new):
    c = Case(lens, new, 1, 4, 128, seed=8)
    for opts in ({}, {"window": 700}, {"softcap": 20.0}):
        out, st = c.run(**opts)
        assert st == 0
        c.check(out, **opts)


@pytest.mark.parametrize("S,longest,new,H,group,D", [
    (40, 1500, 1, 2, 4, 128), (90, 1100, 1, 8, 1, 64), (33, 1300, 4, 4, 4, 128), (40, 1200, 1, 4, 2, 256),
    (2, 20000, 3, 1, 4, 64), (90, 4200, 1, 2, 1, 64), (230, 1030, 1, 4, 1, 64), (20, 900, 1, 4, 16, 128)])
def test_ragged_batches(S, longest, new, H, group, D):
    """Sequences of very different lengths, one of them alone the longest, empty and refused ones
    among them: however the work is shared, every row is whole."""
    rng = np.random.default_rng(S)
    lens = rng.integers(1, longest // 8, S) + new
    lens[S // 2:] //= 4
    lens[-1], lens[0] = longest, new
    n = np.minimum(rng.integers(0, new + 1, S) if new > 1 else np.ones(S, int), lens)
    n[-1] = new
    c = Case([int(x) for x in lens], [int(x) for x in n], H, group, D, seed=S)
    for opts in ({}, {"window": 333}, {"slopes": np.linspace(0.001, 0.1, H * group).astype(np.float32), "softcap": 30.0}):
        out, st = c.run(**opts)
        assert st == 0 and c.untouched(out, slice(c.starts[-1], c.T))
        c.check(out, **opts)
        again, _ = c.run(**opts)
        assert torch.equal(out, again)
    if S > 2:
        wrong = list(c.lens)
        wrong[S // 3] = wrong[-2] = -1
        out, st = c.run(lens=wrong, max_len=longest)
        assert st == 8 and c.untouched(out, slice(c.starts[S - 2], c.starts[S - 1]))
        assert c.untouched(out, slice(c.starts[S // 3], c.starts[S // 3 + 1]))
        c.check(out, seqs=[s for s in range(S - 2) if s != S // 3] + [S - 1])
    if max(c.new) == min(c.new) == 1:
        st, out = status_word(), poison_bf16((S, H * group, D))
        kvq.kvq_decode_attention(c.pool, c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV), longest,
                                 c.q[:S].to(DEV), c.scale, out, dev_status=st)
        assert int(st.item()) == 0
        c.check(out)


@pytest.mark.parametrize("new", [[1, 1, 1], [70, 40, 50]])
def test_bad_sequences_keep_their_rows(new):
    c = Case([100, 80, 60], new, 2, 4, 128, seed=6)
    for lens, status in (([100, -1, 60], 8), ([100, 5000, 60], 8), ([100, new[1] - 1, 60], 8)):
        out, st = c.run(lens=lens, max_len=100)
        assert st == status and c.untouched(out, slice(c.starts[1], c.starts[2]))
        c.check(out, seqs=[0, 2])
    for starts in ([0, new[0], c.T + 9, c.T + 9], [0, new[0], new[0] - 1, c.starts[3]], [0, new[0], -4, c.starts[3]]):
        out, st = c.run(starts=starts)
        assert st == 8 and c.untouched(out, slice(c.starts[-1], c.T))
        c.check(out, seqs=[0])
    if max(new) > 1:
        out, st = c.run(max_q=50)
        assert st == 8 and c.untouched(out, slice(0, c.starts[1]))
        c.check(out, seqs=[1, 2])
    for blk in (-1, 10 ** 6):
        t = c.table.clone()
        t[1, 0] = blk
        out, st = c.run(table=t)
        assert st == 2 and c.untouched(out, slice(c.starts[1], c.starts[2]))
        c.check(out, seqs=[0, 2])


def test_pitches_and_views():
    """q a slice of a fused projection, out a slice of a wider buffer, heads outside tokens."""
    c = Case([90, 200], [33, 70], 2, 4, 64, seed=9)
    Hq = 8
    ref, _ = c.run()
    wide = torch.zeros((c.T, Hq + 8, 64), dtype=torch.bfloat16, device=DEV)
    wide[:, 4:4 + Hq] = c.q.to(DEV)
    big = poison_bf16((c.T, Hq + 2, 64))
    c.run(q=wide[:, 4:4 + Hq], out=big[:, 1:1 + Hq])
    assert torch.equal(big[:c.starts[-1], 1:1 + Hq], ref[:c.starts[-1]])
    assert (big[:, 0].contiguous().view(torch.uint8) == 0xA5).all() and (big[:, -1].contiguous().view(torch.uint8) == 0xA5).all()
    heads_first = c.q.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
    o2 = poison_bf16((Hq, c.T, 64)).transpose(0, 1)
    c.run(q=heads_first, out=o2)
    assert torch.equal(o2[:c.starts[-1]], ref[:c.starts[-1]])


@pytest.mark.parametrize("new", [1, 3, 120])
@pytest.mark.parametrize("q_scale,cap", [(1.0, 50.0), (1.0, 2.0), (6.0, 8.0), (30.0, 1.0)])
def test_cap_from_nearly_linear_to_saturated(new, q_scale, cap):
    """Scores far below the cap, around 3/4 of it (where the tile kernel changes its tanh) and far
    above it."""
    for f in (PG, NV):
        c = Case([333], [new], 2, 4, 128, fmt_k=f, seed=12)
        c.q = (c.q.float() * q_scale).to(torch.bfloat16)
        out, st = c.run(softcap=cap)
        assert st == 0
        c.check(out, softcap=cap)


def test_stored_scales_that_are_no_powers_of_two_and_zero_pages():
    for new in (1, 90):
        c = Case([150], [new], 2, 4, 128, seed=13)
        for t in (c.pool.k_rscale, c.pool.v_rscale):
            t.mul_(1.37)
        first = int(c.table[0, 0])
        c.pool.v_rscale[first] = 0.0  # a page of zeros that still takes its part of the sum
        c.pool.k_rscale[int(c.table[0, 3])] = 0.0
        out, st = c.run()
        assert st == 0
        c.check(out)


@pytest.mark.parametrize("bs,H", [(16, 8), (16, 1), (8, 8), (64, 4)])
@pytest.mark.parametrize("new", [1, 5])
def test_few_rows_by_pages_and_by_rows(bs, H, new):
    for fmts in ((PG, PG), (F8, NV), (NV, F8), (NV, NV)):
        c = Case([70, 1000, new, 0], [new, new, new, 0], H, 2, 128, bs, *fmts, seed=14)
        for opts in ({}, {"window": 90}, {"slopes": np.linspace(0.01, 0.5, 2 * H).astype(np.float32)}):
            out, st = c.run(**opts)
            assert st == 0
            c.check(out, **opts)


def test_large_values():
    """Scores and rows far from 1: scales near the ends of what V's scales allow."""
    for f in (PG, F8, NV):
        for factor in (2.0 ** -60, 2.0 ** 60):
            c = Case([100], [40], 1, 4, 128, fmt_k=f, seed=2)
            c.pool.v_rscale.mul_(factor)
            out, st = c.run()
            assert st == 0
            c.check(out)


def test_calls_on_two_streams_and_two_graphs_with_their_own_workspaces():
    a, b = Case([3000], [2], 2, 4, 128, seed=1), Case([2500, 900], [40, 64], 2, 4, 128, seed=2)
    want = [x.run()[0] for x in (a, b)]
    dev = []
    for x in (a, b):
        need = kvq.kvq_attention_workspace(len(x.lens), x.T, x.H, x.H * x.group, x.D, max(x.new), max(x.lens))
        dev.append(dict(table=x.table.to(DEV), lens=torch.tensor(x.lens, dtype=torch.int32, device=DEV), q=x.q.to(DEV),
                        starts=torch.tensor(x.starts, device=DEV), out=poison_bf16(tuple(x.q.shape)),
                        ws=torch.empty(max(16, need), dtype=torch.uint8, device=DEV), stream=torch.cuda.Stream()))
    call = lambda x, d: kvq.kvq_attention(x.pool, d["table"], d["lens"], max(x.lens), d["q"], d["starts"], max(x.new),
                                          x.scale, d["out"], workspace=d["ws"], stream=d["stream"])
    torch.cuda.synchronize()
    for _ in range(20):
        for x, d in zip((a, b), dev):
            call(x, d)
    torch.cuda.synchronize()
    for x, d, w in zip((a, b), dev, want):
        assert torch.equal(d["out"][:x.starts[-1]], w[:x.starts[-1]])
        d["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(d["graph"], stream=d["stream"]):
            call(x, d)
    for d in dev:
        d["out"].zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for d in dev:
            with torch.cuda.stream(d["stream"]):
                d["graph"].replay()
    torch.cuda.synchronize()
    for x, d, w in zip((a, b), dev, want):
        assert torch.equal(d["out"][:x.starts[-1]], w[:x.starts[-1]])


def test_a_serving_loop():
    """Plan, scatter and attention as a server runs them: prompts in chunks, then single
    tokens, two requests that come and go; every step against the rows stored so far."""
    H, group, D, bs, nb = 2, 4, 128, 16, 64
    pool = kvq.KvPool.empty(nb * bs, H, D, bs, fill=0xFF, fmt=PG, v_fmt=NV)
    S, mb, T = 3, 16, 160
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    table, lens, starts, pos, used, st = i32(S, mb), i32(S), i32(S + 1), i32(T), i32(1), status_word()
    slots = torch.zeros(T, dtype=torch.int64, device=DEV)
    free = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV)
    cached, held = [0, 0, 0], [[], [], []]
    for step, new in enumerate(([50, 7, 0], [33, 1, 20], [1, 1, 1], [4, 1, 90], [1, 1, 1])):
        q, k, v = (synth.normal_bf16((T, h, D), 10 * step + j, 1) for j, h in ((1, H * group), (2, H), (3, H)))
        kvq.kvq_plan_pages(torch.tensor(cached, dtype=torch.int32, device=DEV), torch.tensor(new, dtype=torch.int32, device=DEV),
                           free, bs, table, lens, starts, slots, pos, used, st)
        kvq.kvq_quant_scatter(k.to(DEV), v.to(DEV), slots, pool, st)
        out = poison_bf16((T, H * group, D))
        kvq.kvq_attention(pool, table, lens, mb * bs, q.to(DEV), starts, max(new), D ** -0.5, out, softcap=30.0, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        free = free[int(used):].contiguous()
        host, at = slots.cpu().numpy(), 0
        for s, n in enumerate(new):
            held[s] += list(host[at:at + n])
            at += n
            cached[s] += n
        assert lens.tolist() == cached and (host[at:] == -1).all() and len(set(sum(held, []))) == sum(cached)
        rows = lambda f, c, b, sc: [decoded(f, c, b, sc, np.array(h, np.int64), bs) for h in held]
        K = rows(PG, pool.k_codes, None, pool.k_rscale)
        V = rows(NV, pool.v_codes, pool.v_bscale, pool.v_rscale)
        ref, top = R.attention(q.double().numpy(), K, V, cached, starts.tolist(), D ** -0.5, softcap=30.0)
        vmax = max(np.abs(x).max() for x in V if x.size)
        bound = 2.0 ** -8 * np.abs(ref[:at]) + (2.0 ** -10 + 4 * (30 * 2.0 ** -20 + 2.0 ** -21 * 30 + 2.0 ** -18)) * vmax
        assert (np.abs(out[:at].double().cpu().numpy() - ref[:at]) <= bound).all()
