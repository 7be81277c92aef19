"""Operators of a sparse serving step over the paged cache, as calls and in plain form.

Three operators that a step of a server with long contexts runs one after the other:

  append  K and V of a step or a prompt written into the cache in its format, K turned by
          its position's angles on the way and Q turned beside it, with the least and the
          largest key of each block of tokens kept for the next operator;
  select  for each query token and KV head, the blocks of the cache with the highest bound
          on a score, the first and the last ones always among them;
  attend  attention of the query tokens over the listed blocks alone.

``run`` computes them with elementary torch operations, or, where ``own`` is true, by the
package's entry points.  Request lengths and block lists follow from the case alone,
values, block tables and slots from the seed.
"""

import functools
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
#: where the nearest E2M1 value changes; a tie goes to the even code
E2M1_STEPS = tuple(np.nextafter(np.float32(m), np.float32(0)) if i % 2 else m
                   for i, m in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _append(name, S, L, n, H, g, D, bs, k, v, rot, pairs=False):
    return {"name": name, "op": "append", "S": S, "L": L, "n": n, "H": H, "g": g, "D": D, "bs": bs, "k": k, "v": v,
            "rot": rot, "pairs": pairs}


def _select(name, S, L, n, H, g, D, bs, top, first=1, last=2, even=False):
    return {"name": name, "op": "select", "S": S, "L": L, "n": n, "H": H, "g": g, "D": D, "bs": bs, "top": top,
            "first": first, "last": last, "even": even}


def _attend(name, S, L, n, H, g, D, bs, top, k, v, cap=0.0, even=False):
    return {"name": name, "op": "attend", "S": S, "L": L, "n": n, "H": H, "g": g, "D": D, "bs": bs, "top": top,
            "k": k, "v": v, "cap": cap, "even": even}


def listed():
    return [
        # one decode step of an ordinary batch, written into half-filled pages
        _append("append_step", 64, 8192, 1, 8, 4, 128, 16, "page8", "page8", 128),
        # prompts of several requests, none a whole number of pages
        _append("append_prompts", 24, 300, 2500, 8, 4, 128, 16, "row8", "page8", 128),
        # a small model whose heads turn a part of their channels, neighbours in pairs; 4-bit keys
        _append("append_partial", 9, 50, 700, 2, 7, 64, 32, "nvfp4", "row8", 32, pairs=True),
        # a few chats of middling length: the call's latency
        _select("select_chats", 4, 6000, 1, 8, 4, 128, 16, 32),
        # the ordinary batch of long contexts
        _select("select_batch", 32, 32768, 1, 8, 4, 128, 16, 128, even=True),
        # draft tokens to verify in one step, wide heads
        _select("select_drafts", 8, 40000, 4, 4, 8, 256, 32, 64),
        # a chunk of a very long prompt
        _select("select_chunk", 1, 65536, 1024, 8, 4, 128, 64, 32, even=True),
        # the same few chats
        _attend("attend_chats", 4, 6000, 1, 8, 4, 128, 16, 32, "page8", "page8"),
        # the same batch, a sixteenth of each context
        _attend("attend_batch", 32, 32768, 1, 8, 4, 128, 16, 128, "page8", "page8", even=True),
        # many query heads over a 4-bit cache, capped scores, ragged lengths (some below the list's reach)
        _attend("attend_4bit", 16, 20000, 1, 8, 8, 128, 32, 48, "nvfp4", "nvfp4", cap=50.0),
        # draft tokens to verify in one step, wide heads, 8-bit keys beside 4-bit values
        _attend("attend_drafts", 8, 30000, 4, 4, 4, 256, 16, 64, "row8", "nvfp4"),
        # a chunk of a long prompt
        _attend("attend_chunk", 1, 32768, 512, 8, 4, 128, 64, 32, "page8", "page8", even=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) if hi > lo else lo


FORMATS = [("page8", "page8"), ("page8", "page8"), ("row8", "row8"), ("nvfp4", "nvfp4"), ("row8", "nvfp4"), ("page8", "nvfp4")]


def draw(rng):
    op = rng.choice(["append", "select", "attend"])
    H, D, g = rng.choice([1, 2, 3, 4, 8, 8]), rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 4, 7, 8, 16])
    bs = rng.choice([8, 16, 16, 32, 64])
    if op == "append":
        S = _log(rng, 1, 200)
        n = rng.choice([1, _log(rng, 1, max(1, min(3000, 50000000 // (S * H * D * (g + 2)))))])
        k, v = rng.choice(FORMATS)
        return dict(_append("", S, rng.choice([0, _log(rng, 16, 8192)]), n, H, g, D, bs, k, v,
                            rng.choice([D, D, D // 2, 32]), rng.random() < 0.4), name="draw")
    S = _log(rng, 1, 64)
    n = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, max(9, 400 // S))])
    if op == "select":
        most = max(32 * bs, min(60000, 500000000 // (S * H * D * (1 + n // 8))))
        top = _log(rng, 8, min(200, most // bs // 4))
        L = n + _log(rng, 4 * top * bs, most)
        first = rng.randint(0, 2)
        return dict(_select("", S, L, n, H, g, D, bs, top, first, rng.randint(0, 2)), name="draw")
    top = _log(rng, 1, max(1, min(4096 // bs, 100000000 // (S * n * H * D * bs) + 1)))
    L = n + _log(rng, 1, max(1, min(40000, 500000000 // (S * H * D))))
    k, v = rng.choice(FORMATS)
    return dict(_attend("", S, L, n, H, g, D, bs, top, k, v, cap=rng.choice([0.0, 0.0, 30.0])), name="draw")


# ---------------------------------------------------------------------------
# request lengths, block lists, values and caches
# ---------------------------------------------------------------------------
def _lens(c):
    """(cached, new) tokens of each request, from the case alone."""
    r = random.Random("%s %s %s %s" % (c["op"], c["S"], c["L"], c["n"]))
    cached, new = [], []
    for s in range(c["S"]):
        if c["op"] == "append":
            n = 1 if c["n"] == 1 else r.randint(1, c["n"])
            cached.append(r.randint(0, c["L"]))
        else:  # c["L"]: tokens after the step
            n = c["n"] if s == 0 or c["even"] else r.randint(1, c["n"])
            cached.append((c["L"] if s == 0 or c["even"] else r.randint(n, c["L"])) - n)
        new.append(n)
    return cached, new


@functools.lru_cache(maxsize=2)
def _block_lists(key):
    """Listed blocks [T, H, top] in ascending order, -1 behind the last, as a selection gives
    them: each (request, head) has blocks that most of its queries want, and each query some
    of its own; the query's own block and the first one are always listed."""
    c = dict(key)
    cached, new = _lens(c)
    r = np.random.RandomState(c["S"] * 7919 + c["top"])
    H, bs, top = c["H"], c["bs"], c["top"]
    out = np.full((sum(new), H, top), -1, np.int32)
    at = 0
    for a, n in zip(cached, new):
        blocks = (a + n - 1) // bs + 1
        want = r.rand(H, blocks)
        for i in range(n):
            vis = (a + i) // bs + 1
            x = want[:, :vis] + 0.3 * r.rand(H, vis)
            x[:, 0] = 4
            x[:, vis - 1] = 5
            m = min(top, vis)
            out[at + i, :, :m] = np.sort(np.argpartition(-x, m - 1, axis=1)[:, :m], axis=1)
        at += n
    return out


def _lists(c):
    return _block_lists(tuple(sorted((k, v) for k, v in c.items() if k != "name")))


def _normal(gen, *shape):
    """N(0, 1) values, 1 of 200 channels ten times as large, as K and V rows have them."""
    x = torch.randn(shape, generator=gen, device=DEV)
    return x * (1 + 9 * (torch.rand(shape[-2:], generator=gen, device=DEV) < 0.005).float())


def _power_of_two(amax):
    """The smallest power of two s with amax <= 448 s (at least 2^-126)."""
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), torch.clamp(e - 8 - (m <= 0.875).int(), min=-126))


def _e2m1_codes(q):
    """Nearest 4-bit codes, two to a byte."""
    steps = torch.tensor(E2M1_STEPS, device=DEV)
    code = (torch.bucketize(q.abs().contiguous(), steps) + 8 * torch.signbit(q)).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _quantised_rows(x, fmt):
    """Codes, block scales and row scales of rows x [..., D] in 32 bits."""
    amax = x.abs().amax(-1)
    if fmt == "row8":
        s = amax / 448
        q = torch.clamp(x * torch.where(s > 0, 1 / s, 0.0)[..., None], -448, 448)
        return q.to(torch.float8_e4m3fn).view(torch.uint8), None, s
    s = amax / 2688
    b = x.unflatten(-1, (-1, 16))
    t = torch.clamp(torch.where(s[..., None] > 0, b.abs().amax(-1) / 6 / s[..., None], 0.0), max=448)
    bsc = t.to(torch.float8_e4m3fn)
    f = bsc.float() * s[..., None]
    return _e2m1_codes((b * torch.where(f > 0, 1 / f, 0.0)[..., None]).flatten(-2)), bsc.view(torch.uint8), s


def _plane(x, fmt):
    """One tensor's cache planes (codes, block scales, scales) of values x [blocks, bs, H, D]."""
    nb, bs, H, D = x.shape
    if fmt == "page8":
        s = _power_of_two(x.abs().amax((1, 3)))
        return (x / s[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(nb * bs, H, D), None, s
    return _quantised_rows(x.view(nb * bs, H, D), fmt)


def _tables(gen, c, total, spare):
    """A block table for `total` tokens a request through shuffled blocks, and the number of blocks."""
    bs = c["bs"]
    need = [-(-t // bs) for t in total]
    mb = max(max(need), 1)
    perm = torch.randperm(sum(need) + spare, generator=gen, device=DEV).to(torch.int32)
    col = torch.arange(mb, device=DEV)
    need = torch.tensor(need, device=DEV)
    first = torch.cumsum(need, 0) - need
    table = torch.where(col < need[:, None], perm[torch.clamp(first[:, None] + col, max=perm.numel() - 1)], 0)
    return table.to(torch.int32).contiguous(), perm.numel()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _angles(rot, positions):
    """A model's table of cosines and sines, [positions, rot], in 32 bits from 64-bit angles."""
    a = (torch.arange(positions, device=DEV, dtype=torch.float64)[:, None]
         * 500000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot))
    return torch.cat((torch.cos(a), torch.sin(a)), 1).float().contiguous()


FMT = {"page8": "FMT_FP8_PAGE", "row8": "FMT_FP8", "nvfp4": "FMT_NVFP4"}


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    cached, new = _lens(c)
    S, bs, H, D, T = c["S"], c["bs"], c["H"], c["D"], sum(new)
    Hq = H * c["g"]
    st = dict(c)
    total = [a + n for a, n in zip(cached, new)]
    table, nb = _tables(gen, c, total, 3)
    st.update(table=table, nb=nb, max_len=max(total), max_new=max(new), seq_lens=_i32(total),
              starts=_i32([sum(new[:i]) for i in range(S + 1)]))
    if c["op"] == "append":
        held = _normal(gen, nb, bs, H, D).to(torch.bfloat16).float()
        st["bounds"] = torch.stack((held.amin(1), held.amax(1)), 2).to(torch.bfloat16)
        planes = {"k": _plane(held, c["k"]), "v": _plane(_normal(gen, nb, bs, H, D), c["v"])}
        rows = [(s, p) for s in range(S) for p in range(cached[s], total[s])]
        s, p = (torch.tensor(v, device=DEV) for v in zip(*rows))
        st["slots"] = table[s, p // bs].long() * bs + p % bs
        st["positions"] = p.to(torch.int32)
        st["cos_sin"] = _angles(c["rot"], max(total))
        # Q, K and V are views of a fused projection's output
        qkv = (_normal(gen, T, Hq + 2 * H, D) * 1.5).to(torch.bfloat16)
        st["q"], st["x_k"], st["x_v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        st["q_out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "select":
        # least and largest keys of a block: a block's keys lie around a mean of its own
        mean = torch.randn((nb, H, D), generator=gen, device=DEV) * 0.6
        wide = (1 + 9 * (torch.rand((H, D), generator=gen, device=DEV) < 0.005).float())
        half = 0.5 + torch.rand((nb, H, D), generator=gen, device=DEV)
        st["bounds"] = torch.stack(((mean - half) * wide, (mean + half) * wide), 2).to(torch.bfloat16)
        st["selected"] = torch.full((T, H, c["top"]), -1, dtype=torch.int32, device=DEV)
        planes = {}
    else:
        planes = {j: _plane(_normal(gen, nb, bs, H, D), c[j]) for j in ("k", "v")}
        st["selected"] = torch.tensor(_lists(c), device=DEV)
        st["out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    if c["op"] != "append":
        st["q"] = torch.randn((T, Hq, D), generator=gen, device=DEV).to(torch.bfloat16)
    for j, p in planes.items():
        st[j + "_planes"] = p
    if c["op"] == "append" and "nvfp4" in (c["k"], c["v"]):  # a byte's two 4-bit values, as E4M3 bytes
        val = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV).to(torch.float8_e4m3fn).view(torch.uint8).int()
        byte = torch.arange(256, device=DEV)
        st["pairs_of"] = (val[byte & 15] | (val[byte >> 4] << 8)).to(torch.int16)
    if own:  # the handles and scratch that a server keeps
        import quantized_kv_cache_nvfp4_gb300 as kvq
        if c["op"] == "select":
            st["geometry"] = (bs, nb)
            size = kvq.kvq_select_blocks_workspace(T, H, st["max_len"], bs)
        else:
            st["pool"] = kvq.KvPool(*planes["k"], *planes["v"], bs, *(getattr(kvq, FMT[c[j]]) for j in ("k", "v")))
            size = 0 if c["op"] == "append" else kvq.kvq_sparse_attention_workspace(T, H, Hq, D, bs, c["top"])
        st["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _run_own(st):
    import quantized_kv_cache_nvfp4_gb300 as kvq
    op = st["op"]
    if op == "append":
        kvq.kvq_append(st["x_k"], st["x_v"], st["slots"], st["pool"], cos_sin=st["cos_sin"], positions=st["positions"],
                       interleaved=st["pairs"], q=st["q"], q_out=st["q_out"], key_bounds=st["bounds"])
        return _append_out(st)
    if op == "select":
        return kvq.kvq_select_blocks(st["bounds"], st["table"], st["seq_lens"], st["max_len"], st["bs"], st["q"],
                                     st["starts"], st["max_new"], st["selected"], first_blocks=st["first"],
                                     last_blocks=st["last"], workspace=st["ws"])
    return kvq.kvq_sparse_attention(st["pool"], st["table"], st["seq_lens"], st["max_len"], st["q"], st["starts"],
                                    st["max_new"], st["selected"], st["D"] ** -0.5, st["out"], softcap=st["cap"],
                                    workspace=st["ws"])


def _append_out(st):
    out = {"q": st["q_out"], "bounds": st["bounds"]}
    for j in ("k", "v"):
        codes, bsc, s = st[j + "_planes"]
        out[j + "_scale"] = s
        if bsc is None:
            out[j] = codes.view(torch.float8_e4m3fn)
        else:
            out[j] = st["pairs_of"][codes.int()].view(torch.float8_e4m3fn)
            out[j + "_block_scale"] = bsc.view(torch.float8_e4m3fn)
    return out


def _turned(x, cos_sin, pairs):
    """Rows x [T, heads, D] with their first channels turned by the angles of cos_sin [T, rot]."""
    rot = cos_sin.size(1)
    c, s = (t[:, None] for t in cos_sin.chunk(2, 1))
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = (a * c - b * s, b * c + a * s)
    y = torch.stack(y, -1).flatten(-2) if pairs else torch.cat(y, -1)
    return torch.cat((y, x[..., rot:]), -1)


def _store_pages(x, slots, bs, codes, scale):
    """A page that gets its first row starts over; a page whose scale grows has its rows
    rounded again under the new one."""
    nb, H = scale.shape
    page, off = slots // bs, slots % bs
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(2), "amax")
    hit = torch.zeros(nb, dtype=torch.bool, device=DEV).index_fill_(0, page, True)
    fresh = torch.zeros(nb, dtype=torch.int64, device=DEV).index_add_(0, page, (off == 0).long()) > 0
    kept = torch.where(fresh[:, None], 0.0, scale)
    s = torch.where(hit[:, None], torch.maximum(kept, _power_of_two(amax)), scale)
    ratio = torch.where(kept > 0, kept / s, 1.0)
    held = codes.view(torch.float8_e4m3fn).view(nb, bs, H, -1).float() * ratio[:, None, :, None]
    held = held.to(torch.float8_e4m3fn).view(torch.uint8)
    held[page, off] = (x / s[page][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes.copy_(held.view(codes.shape))
    scale.copy_(s)


def _run_append(st):
    bs, slots = st["bs"], st["slots"]
    cs = st["cos_sin"][st["positions"].long()]
    st["q_out"].copy_(_turned(st["q"].float(), cs, st["pairs"]).to(torch.bfloat16))
    k = _turned(st["x_k"].float(), cs, st["pairs"])
    page = slots // bs
    fresh = torch.zeros(st["nb"], dtype=torch.int64, device=DEV).index_add_(0, page, (slots % bs == 0).long()) > 0
    held = st["bounds"].float()
    low = torch.where(fresh[:, None, None], math.inf, held[:, :, 0]).index_reduce_(0, page, k, "amin")
    high = torch.where(fresh[:, None, None], -math.inf, held[:, :, 1]).index_reduce_(0, page, k, "amax")
    st["bounds"].copy_(torch.stack((low, high), 2).to(torch.bfloat16))
    for j, x in (("k", k), ("v", st["x_v"].float())):
        codes, bsc, s = st[j + "_planes"]
        if st[j] == "page8":
            _store_pages(x, slots, bs, codes, s)
            continue
        for plane, new in zip((codes, bsc, s), _quantised_rows(x, st[j])):
            if plane is not None:
                plane[slots] = new
    return _append_out(st)


def _rows(st):
    """(token, live) of each request's query rows [S, N] and their positions."""
    starts, lens = st["starts"].long(), st["seq_lens"].long()
    i = torch.arange(st["max_new"], device=DEV)
    count = starts[1:] - starts[:-1]
    tok = torch.clamp(starts[:-1, None] + i, max=st["q"].size(0) - 1)
    return tok, i < count[:, None], (lens - count)[:, None] + i


def _run_select(st):
    """Scores in 64 bits: which of two near blocks is listed must not hang on the order of a sum."""
    S, H, g, D, bs, top = (st[k] for k in ("S", "H", "g", "D", "bs", "top"))
    tok, live, pos = _rows(st)
    q = st["q"].double().view(-1, H, g, D)
    q = torch.cat((torch.clamp(q, max=0).sum(2), torch.clamp(q, min=0).sum(2)), -1)  # meets the least, the largest keys
    b = st["bounds"][st["table"].long()].flatten(3).double()  # [S, blocks, H, 2 D]
    score = q[tok].transpose(1, 2) @ b.permute(0, 2, 3, 1)  # [S, H, N, blocks]
    blk = torch.arange(b.size(1), device=DEV)
    own_blk = (pos // bs)[:, None, :, None]
    score = torch.where((blk < st["first"]) | (blk > own_blk - st["last"]), math.inf, score)
    score = torch.where(blk <= own_blk, score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True)
    few = min(top, b.size(1))
    picked = torch.where(order.values[..., :few] > -math.inf, order.indices[..., :few], 1 << 30)
    picked = torch.sort(picked, dim=-1).values.transpose(1, 2)  # [S, N, H, few]
    picked = torch.where(picked < 1 << 30, picked, -1).to(torch.int32)
    st["selected"].fill_(-1)
    st["selected"][tok[live], :, :few] = picked[live]
    return st["selected"]


def _decoded(planes, fmt, bs, at):
    """The cache's values in 32 bits at (slots, heads) `at`."""
    codes, bsc, s = planes
    if fmt == "nvfp4":
        val = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
        codes = codes[at]
        x = torch.stack((val[(codes & 15).int()], val[(codes >> 4).int()]), -1).flatten(-2).unflatten(-1, (-1, 16))
        return (x * (bsc.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s[at][..., None])[..., None]).flatten(-2)
    x = codes[at].view(torch.float8_e4m3fn).float()
    return x * (s[at] if fmt == "row8" else s[at[0] // bs, at[1]])[..., None]


def _run_attend(st):
    S, H, g, D, bs, top = (st[k] for k in ("S", "H", "g", "D", "bs", "top"))
    tok, live, pos = _rows(st)
    T = st["q"].size(0)
    seq = torch.zeros(T, dtype=torch.int64, device=DEV)
    seq[tok[live]] = torch.arange(S, device=DEV)[:, None].expand_as(tok)[live]
    at = torch.zeros(T, dtype=torch.int64, device=DEV)
    at[tok[live]] = pos[live]
    sel = st["selected"].long()
    t = (sel[..., None] * bs + torch.arange(bs, device=DEV)).flatten(2)  # [T, H, top bs]
    seen = (t >= 0) & (t <= at[:, None, None])
    t = torch.where(seen, t, 0)
    slot = st["table"].long()[seq[:, None, None], t // bs] * bs + t % bs
    where = (slot, torch.arange(H, device=DEV)[:, None].expand_as(slot))
    K, V = (_decoded(st[j + "_planes"], st[j], bs, where) for j in "kv")  # [T, H, top bs, D]
    x = st["q"].float().view(T, H, g, D) @ K.transpose(2, 3) * D ** -0.5
    if st["cap"]:
        x = st["cap"] * torch.tanh(x / st["cap"])
    x = torch.where(seen[:, :, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    st["out"].copy_((p @ V / torch.where(total > 0, total, 1.0)).view(T, H * g, D).to(torch.bfloat16))
    return st["out"]


def run(st):
    if own:
        return _run_own(st)
    return {"append": _run_append, "select": _run_select, "attend": _run_attend}[st["op"]](st)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _row_bytes(c, j):
    return {"page8": c["D"] + 4 / c["bs"], "row8": c["D"] + 4, "nvfp4": c["D"] / 2 + c["D"] / 16 + 4}[c[j]]


def work(c):
    cached, new = _lens(c)
    bs, H, D, T = c["bs"], c["H"], c["D"], sum(new)
    Hq = H * c["g"]
    if c["op"] == "append":
        first = [a // bs for a in cached]
        pages = sum((a + n - 1) // bs - f + 1 for a, n, f in zip(cached, new, first))
        begun = sum((a + n - 1) // bs - (a - 1) // bs for a, n in zip(cached, new))
        turns = len({p for a, n in zip(cached, new) for p in range(a, a + n)})
        # Q read and written, K and V read, their codes and scales written, slots and positions read,
        # each position's angles read once, bounds of the pages written, of those held before read
        moved = 4 * T * Hq * D + T * H * (4 * D + _row_bytes(c, "k") + _row_bytes(c, "v")) + 12 * T + 4 * turns * c["rot"]
        moved += (2 * pages - begun) * H * 4 * D
        return {"bytes": moved, "flops": 3 * T * (Hq + H) * c["rot"] + 6 * T * H * D}
    if c["op"] == "select":
        blocks = sum((a + n - 1) // bs + 1 for a, n in zip(cached, new))
        pairs = sum((a + i) // bs + 1 for a, n in zip(cached, new) for i in range(n))
        return {"bytes": blocks * (H * 4 * D + 4) + 2 * T * Hq * D + 4 * T * H * c["top"] + 8 * c["S"],
                "flops": 4 * pairs * H * D + T * Hq * D}
    lists, at, rows, pairs, listed_blocks = _lists(c), 0, 0, 0, 0
    for a, n in zip(cached, new):
        mine = lists[at:at + n]
        pos = np.arange(a, a + n)[:, None, None]
        keys = np.where(mine >= 0, np.clip(pos + 1 - mine.astype(np.int64) * bs, 0, bs), 0)
        pairs += int(keys.sum())
        for h in range(H):  # each listed block's rows once, up to the last query that sees it
            uniq = np.unique(mine[:, h][mine[:, h] >= 0]).astype(np.int64)
            rows += int(np.minimum(bs, a + n - uniq * bs).sum())
            listed_blocks += len(uniq)
        at += n
    moved = rows * (_row_bytes(c, "k") + _row_bytes(c, "v")) + 4 * listed_blocks + 4 * lists.size + 4 * T * Hq * D + 8 * c["S"]
    return {"bytes": moved, "flops": 4 * pairs * Hq // H * D}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_64(q):
    """Nearest E4M3 value (ties to even) of |q| <= 448, in 64 bits."""
    e = torch.floor(torch.log2(torch.clamp(q.abs(), min=2.0 ** -6)))
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return torch.round(q / step) * step


def _e2m1_64(q):
    """Nearest E2M1 value (ties to even) of |q| <= 6, in 64 bits."""
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(q.abs(), min=1.0))), max=2.0) - 1)
    return torch.clamp(torch.round(q / step) * step, -6, 6)


def _exact_append(c, st):
    bs, slots, D = c["bs"], st["slots"], c["D"]
    page, off = slots // bs, slots % bs
    half = c["rot"] // 2
    j = torch.arange(half, device=DEV)
    one, two = (2 * j, 2 * j + 1) if c["pairs"] else (j, j + half)
    cs = st["cos_sin"].double()[st["positions"].long()][:, None]

    def turn(x):
        x, y = x.double(), x.double().clone()
        y[..., one] = x[..., one] * cs[..., :half] - x[..., two] * cs[..., half:]
        y[..., two] = x[..., one] * cs[..., half:] + x[..., two] * cs[..., :half]
        return y

    out = {"q": turn(st["q"])}
    k = turn(st["x_k"])
    begun = torch.zeros(st["nb"], dtype=torch.bool, device=DEV)
    begun[page[off == 0]] = True
    idx = page[:, None, None].expand_as(k)
    b = st["bounds"].double()
    b[begun, :, 0], b[begun, :, 1] = math.inf, -math.inf
    low, high = b[:, :, 0].contiguous(), b[:, :, 1].contiguous()
    out["bounds"] = torch.stack((low.scatter_reduce_(0, idx, k, "amin"), high.scatter_reduce_(0, idx, k, "amax")), 2)
    for name, x in (("k", k), ("v", st["x_v"].double())):
        codes, bsc, scale = st[name + "_planes"]
        if c[name] == "nvfp4":
            s = x.abs().amax(-1) / 2688
            blocks = x.unflatten(-1, (D // 16, 16))
            f = _e4m3_64(torch.clamp(blocks.abs().amax(-1) / 6 / s[..., None], max=448))
            val = st["pairs_of"][codes.int()].view(torch.float8_e4m3fn).double()
            val[slots] = _e2m1_64(blocks / torch.clamp(f * s[..., None], min=1e-30)[..., None]).flatten(-2)
            planes = (val, bsc.view(torch.float8_e4m3fn).double(), scale.double())
            planes[1][slots], planes[2][slots] = f, s
            out[name], out[name + "_block_scale"], out[name + "_scale"] = planes
            continue
        val = codes.view(torch.float8_e4m3fn).double()
        if c[name] == "row8":
            s = scale.double()
            s[slots] = x.abs().amax(-1) / 448
            val[slots] = _e4m3_64(x / s[slots][..., None])
        else:
            val, old = val.view(st["nb"], bs, -1, D), scale.double()
            big = torch.zeros_like(old).scatter_reduce_(0, page[:, None].expand(-1, old.size(1)), x.abs().amax(2), "amax")
            want = torch.exp2(torch.ceil(torch.log2(torch.clamp(big / 448, min=2.0 ** -126))))
            want = torch.where(big <= 448 * want / 2, want / 2, want)
            want = torch.clamp(torch.where(big > 448 * want, want * 2, want), min=2.0 ** -126)
            hit = torch.zeros(st["nb"], dtype=torch.bool, device=DEV)
            hit[page] = True
            base = torch.where(begun[:, None], torch.zeros_like(old), old)
            s = torch.where(hit[:, None], torch.maximum(base, want), old)
            grown = hit[:, None] & (base > 0) & (s > base)
            val = torch.where(grown[:, None, :, None], _e4m3_64(val * (old / s)[:, None, :, None]), val)
            val[page, off] = _e4m3_64(x / s[page][..., None])
        out[name], out[name + "_scale"] = val.view(codes.shape), s
    return out


def _exact_attend(c, st):
    if work(c)["flops"] > 4e11:
        return None
    cached, new = _lens(c)
    H, g, bs = c["H"], c["g"], c["bs"]
    lists = _lists(c)
    y = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    half = torch.tensor(E2M1, dtype=torch.float64, device=DEV)

    def values(j, slot, h):
        codes, bsc, sc = st[j + "_planes"]
        if c[j] != "nvfp4":
            return codes[slot, h].view(torch.float8_e4m3fn).double() * sc[slot if c[j] == "row8" else slot // bs, h].double()[:, None]
        w = codes[slot, h].long()
        w = torch.stack((w % 16, w // 16), -1).flatten(-2)
        x = torch.where(w >= 8, -half[w % 8], half[w % 8])
        f = bsc[slot, h].view(torch.float8_e4m3fn).double() * sc[slot, h].double()[:, None]
        return (x.view(*f.shape, 16) * f[..., None]).flatten(-2)

    at = 0
    for s, (a, n) in enumerate(zip(cached, new)):
        for h in range(H):
            # the keys of every block that a query of this request lists, then each query's share of them
            blocks, place = np.unique(np.where(lists[at:at + n, h] >= 0, lists[at:at + n, h], lists[at, h, 0]), return_inverse=True)
            count = np.zeros((n, len(blocks)))
            np.add.at(count, (np.arange(n)[:, None], place.reshape(n, -1)), lists[at:at + n, h] >= 0)
            blocks = torch.tensor(blocks, device=DEV).long()
            t = (blocks[:, None] * bs + torch.arange(bs, device=DEV)).flatten()
            tt = torch.clamp(t, max=a + n - 1)
            slot = st["table"][s].long()[tt // bs] * bs + tt % bs
            K, V = values("k", slot, h), values("v", slot, h)
            x = torch.einsum("ngd,td->ngt", st["q"][at:at + n, h * g:h * g + g].double(), K) / math.sqrt(c["D"])
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            pos = torch.arange(a, a + n, device=DEV)[:, None]
            seen = torch.repeat_interleave(torch.tensor(count, device=DEV) > 0, bs, 1) & (t <= pos)
            x = torch.nan_to_num(torch.softmax(x.masked_fill(~seen[:, None], -math.inf), -1), nan=0.0)
            y[at:at + n, h * g:h * g + g] = torch.einsum("ngt,td->ngd", x, V)
        at += n
    return y


def exact(c, seed):
    if c["op"] == "select":  # whole numbers
        return None
    st = prepare(dict(c), seed)
    return _exact_append(c, st) if c["op"] == "append" else _exact_attend(c, st)
