"""Paged-cache operators of an LLM server, as calls and in plain form.

Four operators around one paged K/V cache:

  plan    block tables and slot maps built on the GPU from request lengths;
  store   a step's or a prompt's K and V rows written into a cache held in 8 bits (E4M3),
          with one power-of-two scale for each block of tokens and head;
  decode  attention of one new token a sequence over that cache;
  attend  attention of several query tokens a sequence (prompt chunks, draft tokens) over
          the cache, with a tanh cap on the scores, a bias by distance, a window, a prefix
          mask and a document mask.

``run`` computes them with elementary torch operations, or, where ``own`` is true, by the
package's entry points.  Request lengths follow from the case alone, values, tables and
slots from the seed.
"""

import math
import random

import torch

own = False
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _plan(name, S, L, n, bs, prompts):
    return {"name": name, "op": "plan", "S": S, "L": L, "n": n, "bs": bs, "prompts": prompts}


def _store(name, S, L, n, H, D, bs):
    return {"name": name, "op": "store", "S": S, "L": L, "n": n, "H": H, "D": D, "bs": bs}


def _decode(name, S, L, H, g, D, bs, even=False):
    return {"name": name, "op": "decode", "S": S, "L": L, "n": 1, "H": H, "g": g, "D": D, "bs": bs, "even": even,
            "k": "page8", "v": "page8", "cap": 0.0, "alibi": False, "window": 0, "prefix": False, "docs": False}


def _attend(name, S, L, n, H, g, D, bs, k, v, cap=0.0, alibi=False, window=0, prefix=False, docs=False, even=False):
    return {"name": name, "op": "attend", "S": S, "L": L, "n": n, "H": H, "g": g, "D": D, "bs": bs, "even": even,
            "k": k, "v": v, "cap": cap, "alibi": alibi, "window": window, "prefix": prefix, "docs": docs}


def listed():
    return [
        # one decode step of a small server: every request gets one token
        _plan("plan_step", 64, 8192, 1, 16, 0.0),
        # a step that mixes decoding requests with the prompts of new ones
        _plan("plan_prompts", 1000, 16384, 700, 32, 0.25),
        # one decode step written into half-filled pages
        _store("store_step", 64, 4096, 1, 8, 128, 16),
        # prompts of several requests, none a whole number of pages
        _store("store_prompts", 37, 0, 3001, 8, 128, 32),
        # a few short chats: the call's latency
        _decode("decode_chats", 4, 700, 8, 4, 128, 16),
        # the ordinary serving batch
        _decode("decode_batch", 32, 8192, 8, 4, 128, 16, even=True),
        # two very long contexts, wide heads
        _decode("decode_long", 2, 65536, 4, 4, 256, 32, even=True),
        # short prompts behind a shared, fully visible prefix
        _attend("attend_prefix", 5, 333, 77, 2, 7, 64, 16, "page8", "page8", prefix=True),
        # draft tokens to verify in one step, scores capped, local layers' window
        _attend("attend_drafts", 32, 4096, 4, 8, 4, 128, 16, "page8", "page8", cap=30.0, window=1024),
        # single tokens with a bias by distance over a 4-bit cache
        _attend("attend_bias_step", 16, 5000, 1, 8, 8, 128, 16, "nvfp4", "nvfp4", alibi=True),
        # whole prompts made of packed documents, 4-bit cache
        _attend("attend_documents", 2, 2500, 2500, 8, 4, 128, 16, "nvfp4", "nvfp4", docs=True),
        # a chunk of a long prompt, scores capped
        _attend("attend_chunk", 1, 12288, 4096, 8, 4, 128, 32, "page8", "page8", cap=50.0, even=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "decode", "attend", "attend"])
    bs = rng.choice([8, 16, 16, 32, 64])
    if op == "plan":
        S = _log(rng, 1, 2000)
        n = min(_log(rng, 1, 4000), 400000 // S)
        return dict(_plan("", S, _log(rng, 64, 32768), max(1, n), bs, rng.choice([0.0, 0.25, 1.0])), name="draw")
    H, D = rng.choice([1, 2, 3, 4, 8, 8]), rng.choice([64, 128, 128, 256])
    if op == "store":
        S = _log(rng, 1, 256)
        n = rng.choice([1, _log(rng, 1, max(1, min(4000, 60000000 // (S * H * D))))])
        return dict(_store("", S, rng.choice([0, _log(rng, 16, 4096)]), n, H, D, bs), name="draw")
    g = rng.choice([1, 2, 4, 4, 7, 8])
    if op == "decode":
        S = _log(rng, 1, 64)
        L = _log(rng, 1, max(1, min(32768, 100000000 // (S * H * D))))
        return dict(_decode("", S, L, H, g, D, bs), name="draw")
    n = rng.choice([1, rng.randint(2, 8), _log(rng, 9, 2000)])
    S = _log(rng, 1, max(1, min(32, 4000 // n)))
    L = n + rng.choice([0, _log(rng, 1, max(1, min(12000, 60000000 // (S * n * H * g) + 200)))])
    fmts = rng.choice([("page8", "page8"), ("page8", "page8"), ("row8", "row8"), ("nvfp4", "nvfp4"), ("page8", "nvfp4")])
    return dict(_attend("", S, L, n, H, g, D, bs, *fmts, cap=rng.choice([0.0, 20.0, 50.0]),
                        alibi=rng.random() < 0.3, window=rng.choice([0, 0, 0, rng.randint(1, 600)]),
                        prefix=rng.random() < 0.25, docs=rng.random() < 0.25), name="draw")


# ---------------------------------------------------------------------------
# request lengths, values and caches
# ---------------------------------------------------------------------------
def _lens(c):
    """(cached, new) tokens of each request, from the case alone."""
    r = random.Random("%s %s %s %s" % (c["op"], c["S"], c["L"], c["n"]))
    cached, new = [], []
    for s in range(c["S"]):
        if c["op"] == "plan":
            n = r.randint(1, c["n"]) if r.random() < c["prompts"] else 1
            cached.append(0 if n > 1 and r.random() < 0.7 else r.randint(0, c["L"]))
        elif c["op"] == "store":
            n = 1 if c["n"] == 1 else r.randint(1, c["n"])
            cached.append(r.randint(0, c["L"]))
        else:  # c["L"]: tokens after the step
            n = c["n"] if s == 0 or c["even"] else r.randint(1, c["n"])
            cached.append((c["L"] if s == 0 or c["even"] else r.randint(n, c["L"])) - n)
        new.append(n)
    return cached, new


def _normal(gen, *shape):
    """N(0, 1) values, 1 of 200 channels ten times as large, as K and V rows have them."""
    x = torch.randn(shape, generator=gen, device=DEV)
    return x * (1 + 9 * (torch.rand(shape[-2:], generator=gen, device=DEV) < 0.005).float())


def _power_of_two(amax):
    """The smallest power of two s with amax <= 448 s (at least 2^-126)."""
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), torch.clamp(e - 8 - (m <= 0.875).int(), min=-126))


def _plane(gen, fmt, nb, bs, H, D):
    """One tensor's cache planes (codes, block scales, scales) with quantised N(0, 1) rows."""
    x = _normal(gen, nb, bs, H, D).to(torch.bfloat16).float()
    if fmt == "page8":
        s = _power_of_two(x.abs().amax((1, 3)))
        return (x / s[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(nb * bs, H, D), None, s
    x = x.view(nb * bs, H, D)
    amax = x.abs().amax(2)
    if fmt == "row8":
        s = amax / 448
        q = torch.clamp(x / s[..., None], -448, 448)
        return q.to(torch.float8_e4m3fn).view(torch.uint8), None, s
    s = amax / 2688
    b = x.view(nb * bs, H, D // 16, 16)
    bsc = torch.clamp(b.abs().amax(3) / 6 / s[..., None], max=448).to(torch.float8_e4m3fn)
    q = b / torch.clamp(bsc.float() * s[..., None], min=1e-30)[..., None]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = (torch.bucketize(q.abs().contiguous(), mids) + 8 * (q < 0)).view(nb * bs, H, D // 2, 2).to(torch.uint8)
    return code[..., 0] | (code[..., 1] << 4), bsc.view(torch.uint8), s


def _tables(gen, c, total, spare):
    """A block table for `total` tokens a request through shuffled blocks, and the rest."""
    bs = c["bs"]
    need = [-(-t // bs) for t in total]
    mb = max(max(need), 1)
    perm = torch.randperm(sum(need) + spare, generator=gen, device=DEV).to(torch.int32)
    col = torch.arange(mb, device=DEV)
    need = torch.tensor(need, device=DEV)
    first = torch.cumsum(need, 0) - need
    table = torch.where(col < need[:, None], perm[torch.clamp(first[:, None] + col, max=perm.numel() - 1)], 0)
    return table.to(torch.int32).contiguous(), perm[int(need.sum()):].contiguous(), perm.numel()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


FMT = {"page8": "FMT_FP8_PAGE", "row8": "FMT_FP8", "nvfp4": "FMT_NVFP4"}


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    cached, new = _lens(c)
    S, bs, T = c["S"], c["bs"], sum(new)
    st = dict(c)
    if c["op"] == "plan":
        used = sum(-(-(a + n) // bs) - -(-a // bs) for a, n in zip(cached, new))
        mb = max(-(-(a + n) // bs) for a, n in zip(cached, new))
        table, free, _ = _tables(gen, c, cached, used + 40)
        st["table"] = torch.zeros((S, mb), dtype=torch.int32, device=DEV)
        st["table"][:, :table.size(1)] = table[:, :mb]
        st.update(free=free, cached=_i32(cached), new=_i32(new), seq_lens=_i32([0] * S), starts=_i32([0] * (S + 1)),
                  slots=torch.zeros(T + 5, dtype=torch.int64, device=DEV), positions=_i32([0] * (T + 5)), used=_i32([0]))
        return st
    H, D = c["H"], c["D"]
    table, _, nb = _tables(gen, c, [a + n for a, n in zip(cached, new)], 3)
    planes = {j: _plane(gen, c.get(j, "page8"), nb, bs, H, D) for j in ("k", "v")}
    for j, p in planes.items():
        st[j + "_planes"] = p
    st["table"] = table
    if own:  # the handle of the cache, as a server keeps it
        import quantized_kv_cache_nvfp4_gb300 as kvq
        f = {j: getattr(kvq, FMT[c.get(j, "page8")]) for j in ("k", "v")}
        st["pool"] = kvq.KvPool(*planes["k"], *planes["v"], bs, f["k"], f["v"])
    if c["op"] == "store":
        rows = [(s, p) for s in range(S) for p in range(cached[s], cached[s] + new[s])]
        s, p = (torch.tensor(v, device=DEV) for v in zip(*rows))
        st["slots"] = table[s, p // bs].long() * bs + p % bs
        # K is a view of a fused projection's output, V has its own tensor
        st["qkv"] = (_normal(gen, T, 2 * H, D) * 1.5).to(torch.bfloat16)
        st["x_k"] = st["qkv"][:, H:]
        st["x_v"] = (_normal(gen, T, H, D) * 1.5).to(torch.bfloat16)
        return st
    Hq = H * c["g"]
    st["max_len"] = max(a + n for a, n in zip(cached, new))
    st["max_new"] = max(new)
    st["seq_lens"] = _i32([a + n for a, n in zip(cached, new)])
    starts = [sum(new[:i]) for i in range(S + 1)]
    st["starts"] = _i32(starts)
    st["q"] = torch.randn((T, Hq, D), generator=gen, device=DEV).to(torch.bfloat16)
    st["out"] = torch.zeros_like(st["q"])
    st["slopes"] = torch.exp2(-8 * torch.arange(1, Hq + 1, device=DEV).float() / Hq) if c["alibi"] else None
    r = random.Random("%d" % c["L"])
    st["prefix"] = _i32([r.randint(0, a + n) for a, n in zip(cached, new)]) if c["prefix"] else None
    st["key_starts"] = None
    if c["docs"]:  # each query's document begins at the last boundary up to its position
        firsts = []
        for a, n in zip(cached, new):
            cuts = sorted({0} | {r.randint(0, a + n) for _ in range((a + n) // 400 + 1)})
            at = 0
            for p in range(a, a + n):
                while at + 1 < len(cuts) and cuts[at + 1] <= p:
                    at += 1
                firsts.append(cuts[at])
        st["key_starts"] = _i32(firsts)
    if own:
        size = (kvq.kvq_decode_attention_workspace(S, H, Hq, D, st["max_len"]) if c["op"] == "decode" else
                kvq.kvq_attention_workspace(S, T, H, Hq, D, st["max_new"], st["max_len"]))
        st["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _run_own(st):
    import quantized_kv_cache_nvfp4_gb300 as kvq
    op = st["op"]
    if op == "plan":
        kvq.kvq_plan_pages(st["cached"], st["new"], st["free"], st["bs"], st["table"], st["seq_lens"], st["starts"],
                           st["slots"], st["positions"], st["used"])
        return _plan_out(st)
    if op == "store":
        kvq.kvq_quant_scatter(st["x_k"], st["x_v"], st["slots"], st["pool"])
        return _store_out(st)
    scale = st["D"] ** -0.5
    if op == "decode":
        return kvq.kvq_decode_attention(st["pool"], st["table"], st["seq_lens"], st["max_len"], st["q"], scale,
                                        st["out"], st["ws"])
    return kvq.kvq_attention(st["pool"], st["table"], st["seq_lens"], st["max_len"], st["q"], st["starts"],
                             st["max_new"], scale, st["out"], softcap=st["cap"], alibi_slopes=st["slopes"],
                             window=st["window"], prefix_lens=st["prefix"], key_starts=st["key_starts"],
                             workspace=st["ws"])


def _plan_out(st):
    return {k: st[k] for k in ("table", "seq_lens", "starts", "slots", "positions", "used")}


def _store_out(st):
    return {"k": st["k_planes"][0].view(torch.float8_e4m3fn), "k_scale": st["k_planes"][2],
            "v": st["v_planes"][0].view(torch.float8_e4m3fn), "v_scale": st["v_planes"][2]}


def _run_plan(st):
    """Request s takes ceil((c + n) / bs) - ceil(c / bs) blocks off the free list, in order;
    its token i sits at position c + i, in slot table[s][pos / bs] * bs + pos % bs."""
    c, n, bs = st["cached"].long(), st["new"].long(), st["bs"]
    old, all_ = (c + bs - 1) // bs, (c + n + bs - 1) // bs
    last = torch.cumsum(all_ - old, 0)
    first = last - (all_ - old)
    ends = torch.cumsum(n, 0)
    col = torch.arange(st["table"].size(1), device=DEV)
    taken = st["free"][torch.clamp(first[:, None] + col - old[:, None], 0, st["free"].numel() - 1)]
    is_new = (col >= old[:, None]) & (col < all_[:, None])
    st["table"].copy_(torch.where(is_new, taken, st["table"]))
    st["seq_lens"].copy_(c + n)
    st["starts"][1:].copy_(ends)
    t = torch.arange(st["slots"].numel(), device=DEV)
    s = torch.clamp(torch.searchsorted(ends, t, right=True), max=c.numel() - 1)
    pos = c[s] + t - (ends - n)[s]
    live = t < ends[-1]
    page = torch.clamp(pos // bs, max=col.numel() - 1)
    st["slots"].copy_(torch.where(live, st["table"][s, page].long() * bs + pos % bs, -1))
    st["positions"].copy_(torch.where(live, pos, -1))
    st["used"].copy_(last[-1:])
    return _plan_out(st)


def _store_plane(x, slots, bs, codes, scale):
    """A page that gets its first row starts over; a page whose scale grows has its rows
    rounded again under the new one."""
    nb, H = scale.shape
    page, off = slots // bs, slots % bs
    x = x.float()
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


def _decoded(planes, fmt, bs):
    """The cache's values in 32 bits, [blocks, bs, H, D]."""
    codes, bsc, s = planes
    if fmt == "nvfp4":
        val = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
        x = torch.stack((val[(codes & 15).long()], val[(codes >> 4).long()]), 3).flatten(2)
        x = x * torch.repeat_interleave(bsc.view(torch.float8_e4m3fn).float() * s[..., None], 16, 2)
    else:
        x = codes.view(torch.float8_e4m3fn).float()
        x = x * (s[..., None] if fmt == "row8" else torch.repeat_interleave(s, bs, 0)[..., None])
    return x.view(-1, bs, *x.shape[1:])


def _visible(st, pos, tok):
    """The keys [lo, hi) that a query at position pos sees."""
    lo, hi = torch.zeros_like(pos), pos + 1
    if st["prefix"] is not None:
        hi = torch.maximum(hi, torch.minimum(st["prefix"], st["seq_lens"])[:, None].long())
    if st["window"]:
        lo = torch.clamp(pos + 1 - st["window"], min=0)
    if st["key_starts"] is not None:
        lo = torch.maximum(lo, st["key_starts"][tok].long())
    return lo, hi


def _run_attend(st):
    S, H, g, D = st["S"], st["H"], st["g"], st["D"]
    L, N = st["max_len"], st["max_new"]
    live = st["table"][:, :-(-L // st["bs"])].long()
    K, V = (_decoded(st[j + "_planes"], st[j], st["bs"])[live].flatten(1, 2)[:, :L].transpose(1, 2) for j in "kv")
    starts, lens = st["starts"].long(), st["seq_lens"].long()
    i = torch.arange(N, device=DEV)
    count = starts[1:] - starts[:-1]
    tok = torch.clamp(starts[:-1, None] + i, max=st["q"].size(0) - 1)
    pos = (lens - count)[:, None] + i
    q = st["q"][tok].float().view(S, N, H, g, D).permute(0, 2, 3, 1, 4).reshape(S, H, g * N, D)
    x = (q @ K.transpose(2, 3)).view(S, H, g, N, L) * D ** -0.5
    if st["cap"]:
        x = st["cap"] * torch.tanh(x / st["cap"])
    t = torch.arange(L, device=DEV)
    if st["slopes"] is not None:
        x = x + st["slopes"].view(1, H, g, 1, 1) * (t - pos[..., None])[:, None, None]
    lo, hi = _visible(st, pos, tok)
    seen = ((t >= lo[..., None]) & (t < hi[..., None]))[:, None, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    p = (p / torch.where(total > 0, total, 1.0)).view(S, H, g * N, L)
    y = (p @ V).view(S, H, g, N, D).permute(0, 3, 1, 2, 4).reshape(S, N, H * g, D)
    st["out"].copy_(y[i < count[:, None]].to(torch.bfloat16))
    return st["out"]


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "plan":
        return _run_plan(st)
    if st["op"] == "store":
        _store_plane(st["x_k"], st["slots"], st["bs"], st["k_planes"][0], st["k_planes"][2])
        _store_plane(st["x_v"], st["slots"], st["bs"], st["v_planes"][0], st["v_planes"][2])
        return _store_out(st)
    return _run_attend(st)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(c):
    cached, new = _lens(c)
    S, bs, T = c["S"], c["bs"], sum(new)
    if c["op"] == "plan":
        taken = sum(-(-(a + n) // bs) - -(-a // bs) for a, n in zip(cached, new))
        # lengths read, lengths, starts and tables written, slots and positions written,
        # the half-filled page of each request looked up
        return {"bytes": 8 * S + 4 * S + 4 * (S + 1) + 8 * taken + 12 * (T + 5) + 4 * S + 4, "flops": 0}
    H, D = c["H"], c["D"]
    if c["op"] == "store":
        pages = sum((a + n - 1) // bs - a // bs + 1 for a, n in zip(cached, new))
        return {"bytes": 2 * T * H * D * 3 + 8 * T + 2 * pages * H * 4, "flops": 2 * T * H * D * 2}
    row = {"page8": D + 4 / bs, "row8": D + 4, "nvfp4": D / 2 + D / 16 + 4}
    Hq, keys, pairs = H * c["g"], 0, 0
    st = prepare_masks(c)
    at = 0
    for s, (a, n) in enumerate(zip(cached, new)):
        lo, hi = st[0][at:at + n], st[1][at:at + n]
        pairs += sum(max(0, h - l) for l, h in zip(lo, hi))
        keys += max(0, max(hi) - min(lo))
        at += n
    moved = keys * H * (row[c["k"]] + row[c["v"]]) + 4 * keys / bs + 4 * T * Hq * D + 8 * S
    return {"bytes": moved, "flops": 4 * pairs * Hq * D}


def prepare_masks(c):
    """The visible range of every query, as prepare's masks give it."""
    cached, new = _lens(c)
    r = random.Random("%d" % c["L"])
    prefix = [r.randint(0, a + n) for a, n in zip(cached, new)] if c["prefix"] else [0] * len(new)
    lo, hi = [], []
    for a, n, pre in zip(cached, new, prefix):
        cuts, at = [0], 0
        if c["docs"]:
            cuts = sorted({0} | {r.randint(0, a + n) for _ in range((a + n) // 400 + 1)})
        for p in range(a, a + n):
            while at + 1 < len(cuts) and cuts[at + 1] <= p:
                at += 1
            lo.append(max(cuts[at], p + 1 - c["window"] if c["window"] else 0, 0))
            hi.append(max(p + 1, min(pre, a + n)))
    return lo, hi


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_64(q):
    """Nearest E4M3 value (ties to even) of |q| <= 448, in 64 bits."""
    e = torch.floor(torch.log2(torch.clamp(q.abs(), min=2.0 ** -6)))
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return torch.round(q / step) * step


def exact(c, seed):
    if c["op"] == "plan":
        return None
    st = prepare(dict(c), seed)
    if c["op"] == "store":
        out, bs = {}, c["bs"]
        for j in ("k", "v"):
            codes, _, scale = st[j + "_planes"]
            nb, H = scale.shape
            x, slots = st["x_" + j].double(), st["slots"]
            page = slots // bs
            val = codes.view(torch.float8_e4m3fn).double().view(nb, bs, H, -1)
            s_old = scale.double()
            begun = torch.zeros(nb, dtype=torch.bool, device=DEV)
            begun[page[slots % bs == 0]] = True
            big = torch.zeros_like(s_old).scatter_reduce_(0, page[:, None].expand(-1, H), x.abs().amax(2), "amax")
            want = torch.exp2(torch.ceil(torch.log2(torch.clamp(big / 448, min=2.0 ** -126))))
            want = torch.where(big <= 448 * want / 2, want / 2, want)
            want = torch.clamp(torch.where(big > 448 * want, want * 2, want), min=2.0 ** -126)
            hit = torch.zeros(nb, dtype=torch.bool, device=DEV)
            hit[page] = True
            base = torch.where(begun[:, None], torch.zeros_like(s_old), s_old)
            s = torch.where(hit[:, None], torch.maximum(base, want), s_old)
            grown = hit[:, None] & (base > 0) & (s > base)
            val = torch.where(grown[:, None, :, None], _e4m3_64(val * (s_old / s)[:, None, :, None]), val)
            val[page, slots % bs] = _e4m3_64(x / s[page][..., None])
            out[j], out[j + "_scale"] = val.view(codes.shape), s
        return out
    if work(c)["flops"] > 4e12:
        return None
    cached, new = _lens(c)
    lo, hi = prepare_masks(c)
    H, g, D, bs = c["H"], c["g"], c["D"], c["bs"]
    y = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    half = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    at = 0
    for s, (a, n) in enumerate(zip(cached, new)):
        t = torch.arange(a + n, device=DEV)
        slot = st["table"][s].long()[t // bs] * bs + t % bs
        kv = []
        for j in ("k", "v"):
            codes, bsc, sc = st[j + "_planes"]
            if c[j] == "nvfp4":
                w = codes[slot].long()
                w = torch.stack((w % 16, w // 16), -1).flatten(-2)
                x = torch.where(w >= 8, -half[w % 8], half[w % 8])
                b = bsc[slot].view(torch.float8_e4m3fn).double() * sc[slot].double()[..., None]
                x = (x.view(*b.shape, 16) * b[..., None]).flatten(-2)
            else:
                x = codes[slot].view(torch.float8_e4m3fn).double()
                x = x * sc[slot if c[j] == "row8" else slot // bs].double()[..., None]
            kv.append(x)
        low, high = (torch.tensor(v[at:at + n], device=DEV)[:, None] for v in (lo, hi))
        seen = (t >= low) & (t < high)
        p = torch.arange(a, a + n, device=DEV)[:, None]
        for h in range(H * g):
            x = st["q"][at:at + n, h].double() @ kv[0][:, h // g].T / math.sqrt(D)
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if c["alibi"]:
                x = x + st["slopes"][h].double() * (t - p)
            x = x.masked_fill(~seen, -math.inf)
            x = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
            y[at:at + n, h] = x @ kv[1][:, h // g]
        at += n
    return y
