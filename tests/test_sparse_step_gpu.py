"""The sparse step as a server runs it: page plan, append, selection and attention over the listed
blocks, prompts first, then captured steps of single tokens; each part against its definition."""

import numpy as np
import pytest
import torch

import quantized_kv_cache_nvfp4_gb300 as kvq
import paged_ref as R
import sparse_ref as X
from quantized_kv_cache_nvfp4_gb300 import synth
from kvq_testutil import DEV, status_word
from test_query_attention_gpu import decoded

pytestmark = pytest.mark.gpu
PG, F8, NV = kvq.FMT_FP8_PAGE, kvq.FMT_FP8, kvq.FMT_NVFP4


@pytest.mark.parametrize("fk,fv,D,bs,rot,pairs", [(PG, PG, 128, 16, 128, False), (NV, NV, 64, 8, 32, True), (F8, NV, 256, 16, 256, False)])
def test_prompts_then_captured_steps(fk, fv, D, bs, rot, pairs):
    S, H, g, mb, topk, cap = 3, 2, 4, 40, 6, 30.0
    Hq, nb, most = H * g, S * 40 + 5, 40 * bs
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)
    pool = kvq.KvPool.empty(nb * bs, H, D, bs, fill=0xFF, fmt=fk, v_fmt=fv)
    bounds = torch.full((nb, H, 2, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    cs = X.angles(most, rot)
    cs_on, free = cs.to(DEV), synth.block_permutation(nb, 1).to(DEV)
    table, used, st = torch.full((S, mb), -1, dtype=torch.int32, device=DEV), i32([0]), status_word()
    cached = i32([0] * S)
    host = {s: (np.zeros((0, H, D), np.float32), np.zeros((0, H, D), np.float32)) for s in range(S)}
    taken = 0

    def make(T):
        return dict(T=T, new=i32([0] * S), lens=i32([0] * S), starts=i32([0] * (S + 1)),
                    slots=torch.zeros(T, dtype=torch.int64, device=DEV), pos=i32([0] * T),
                    qkv=torch.zeros((T, Hq + 2 * H, D), dtype=torch.bfloat16, device=DEV),
                    sel=i32(np.full((T, H, topk), -7)), out=torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV),
                    ws=[torch.empty(max(16, n), dtype=torch.uint8, device=DEV) for n in
                        (kvq.kvq_select_blocks_workspace(T, H, most, bs), kvq.kvq_sparse_attention_workspace(T, H, Hq, D, bs, topk))])

    def step(b, max_q):
        q, k, v = b["qkv"][:, :Hq], b["qkv"][:, Hq:Hq + H], b["qkv"][:, Hq + H:]
        kvq.kvq_plan_pages(cached, b["new"], free_now, bs, table, b["lens"], b["starts"], b["slots"], b["pos"], used, st)
        kvq.kvq_append(k, v, b["slots"], pool, cos_sin=cs_on, positions=b["pos"], interleaved=pairs, q=q, q_out=q,
                       key_bounds=bounds, dev_status=st)
        kvq.kvq_select_blocks(bounds, table, b["lens"], most, bs, q, b["starts"], max_q, b["sel"], first_blocks=1,
                              last_blocks=1, workspace=b["ws"][0], dev_status=st)
        kvq.kvq_sparse_attention(pool, table, b["lens"], most, q, b["starts"], max_q, b["sel"], D ** -0.5, b["out"],
                                 softcap=cap, workspace=b["ws"][1], dev_status=st)
        cached.copy_(b["lens"])

    def check(b, new, raw):
        assert int(st.item()) == 0
        lens = b["lens"].cpu().numpy()
        starts = np.concatenate(([0], np.cumsum(new)))
        np.testing.assert_array_equal(b["starts"].cpu().numpy(), starts)
        n, x, tab = starts[-1], raw.float().numpy(), table.cpu().numpy()
        pos = np.concatenate([np.arange(l - m, l) for l, m in zip(lens, new)]) if n else np.zeros(0, np.int64)
        rows = cs.numpy()[pos]
        q = torch.tensor(X.turned(x[:n, :Hq], rows, pairs)).to(torch.bfloat16)
        assert torch.equal(b["qkv"][:n, :Hq].cpu(), q)
        assert torch.equal(b["qkv"][n:, :Hq].cpu(), raw[n:, :Hq])  # padding stays
        turned = X.turned(x[:n, Hq:Hq + H], rows, pairs)
        bnd = bounds.float().cpu().numpy()
        for s in range(S):
            k, v = host[s]
            a = starts[s]
            host[s] = (np.concatenate((k, turned[a:a + new[s]])), np.concatenate((v, x[a:a + new[s], Hq + H:])))
            kb = X.bf16(host[s][0])
            for blk in range(-(-lens[s] // bs)):
                mine = kb[blk * bs:(blk + 1) * bs]
                np.testing.assert_array_equal(bnd[tab[s, blk], :, 0], mine.min(0))
                np.testing.assert_array_equal(bnd[tab[s, blk], :, 1], mine.max(0))
        sel = b["sel"].cpu().numpy()
        want = X.select(q.float().numpy(), bnd, tab, lens, starts, bs, topk, 1, 1, np.full((b["T"], H, topk), -7, np.int32))
        np.testing.assert_array_equal(sel[:n], want[:n])
        K, V = [], []
        for s in range(S):
            p = np.arange(lens[s])
            slots = tab[s, p // bs].astype(np.int64) * bs + p % bs
            K.append(decoded(fk, pool.k_codes, pool.k_bscale, pool.k_rscale, slots, bs))
            V.append(decoded(fv, pool.v_codes, pool.v_bscale, pool.v_rscale, slots, bs))
            # what the pool holds is what was appended, within the format's rounding of the block's largest
            for got, ref, f in ((K[s], host[s][0], fk), (V[s], host[s][1], fv)):
                if len(ref):
                    top = np.abs(ref).max((0, 2), keepdims=True)
                    assert (np.abs(got - ref) <= (0.27 if f == NV else 0.07) * top).all()
        ref, top, vmax = X.sparse_attention(q.double().numpy(), K, V, lens, starts, sel[:n], bs, D ** -0.5, cap)
        X.close(b["out"][:n].double().cpu().numpy(), ref, top, vmax, D, cap)

    def load(b, new, seed):
        raw = synth.normal_bf16((b["T"], Hq + 2 * H, D), seed, 3, 0.01, 8.0)
        b["qkv"].copy_(raw), b["new"].copy_(i32(new))
        return raw

    free_now = free
    new = [9 * bs + 3, 1, 12 * bs]
    b = make(sum(new) + 4)
    raw = load(b, new, 1)
    step(b, max(new))
    torch.cuda.synchronize()
    check(b, new, raw)
    taken = int(used.item())
    # the captured step takes its blocks off a list of its own, refreshed before each replay
    b, free_now = make(7), torch.zeros(S, dtype=torch.int32, device=DEV)
    free_now.copy_(free[taken:taken + S])
    keep = cached.clone(), table.clone(), pool, bounds.clone(), [t.clone() for t in pool._planes()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # lazy set-up outside of the capture, undone below
        step(b, 2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b, 2)
    cached.copy_(keep[0]), table.copy_(keep[1]), bounds.copy_(keep[3])
    for t, was in zip(pool._planes(), keep[4]):
        t.copy_(was)
    r = np.random.RandomState(2)
    for i in range(2 * bs + 3):
        new = r.randint(0, 3, S).tolist()
        raw = load(b, new, 10 + i)
        free_now.copy_(free[taken:taken + S])
        graph.replay()
        torch.cuda.synchronize()
        check(b, new, raw)
        taken += int(used.item())
